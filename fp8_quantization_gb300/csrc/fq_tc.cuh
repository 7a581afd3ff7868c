// Tensor-core (tcgen05 / TMEM) and ragged-group helpers shared by the FP8
// matrix products of libfq.so.
#pragma once

#include "fq_common.cuh"

namespace fq {

// ---------------------------------------------------------------- bounded waits

// A whole converged warp waits for phase `parity` of the mbarrier at shared
// address `bar`, at most about kWaitLimitNs; a wait that runs out raises the
// CTA's shared `abort` flag, at which every other wait of the CTA gives up too,
// so that all roles reach the kernel's end.  Every branch is on a vote of the
// warp: branches on which the lanes could part cost about 100 cycles here.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, volatile int32_t *abort)
{
    auto done = [&]() {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        return __all_sync(0xffffffffu, ok);
    };
    uint64_t t0 = 0;
    for (uint32_t n = 1; !done(); n++) {
        if (n % 64 == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0)
                t0 = now;
            if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > kWaitLimitNs)) {
                *abort = 1;
                return;
            }
        }
    }
}

// One lane of the converged warp, always the same.  The tensor copies and
// tcgen05 instructions take their operands from the warp's uniform registers:
// behind this predicate the compiler knows that one thread issues them, behind
// a comparison of lane numbers it does not.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- tcgen05

// kCtas = 1: the CTA alone; kCtas = 2: a cluster of two CTAs whose tensor cores
// work on one tile (each CTA holds its half of both operands and of the
// accumulator rows; the CTA of even rank issues).

// Columns of TMEM for the CTA (a power of two, 32..512); the base address is
// written to shared memory.  One full warp (of each CTA) allocates and frees.
template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols)
{
    if (kCtas == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(dst)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(dst)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}

template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if (kCtas == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptor of a K-major tile of 128-byte rows in the
// 128-byte swizzle (8-row atoms of 1024 bytes, the tile 1024-byte aligned):
// start address / 16, atom pitch / 16 in bits 32-45, the fixed 001 of bits
// 46-48, swizzle mode 2 (128 bytes) in bits 61-63.
__device__ __forceinline__ uint64_t smem_desc_sw128(const void *tile)
{
    return static_cast<uint64_t>((smem_u32(tile) & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f8f6f4: E4M3 x E4M3 -> FP32, both operands
// K-major, an M x N tile.
constexpr uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(m / 16) << 24);
}

// D (+)= A B^T over 32 elements of K, issued by one thread; `accumulate`
// false starts a new sum.
template <int kCtas>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate)
{
    const uint32_t acc = accumulate;
    if (kCtas == 1)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc)
                     : "memory");
}

// One arrival on the barrier at shared address `bar` (kCtas = 2: on the barrier
// at that place in both CTAs) once every tcgen05.mma this thread issued is done.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if (kCtas == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Address, in the cluster's shared memory, of CTA `rank`'s object at the place
// of this CTA's `own`.
__device__ __forceinline__ uint32_t cluster_addr(const void *own, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(own)), "r"(rank));
    return a;
}

// FP32 of the cluster's shared memory (address by cluster_addr).
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// An arrival by the lanes with `pred`, on a barrier of this CTA or its pair's
// (released to the CTA only: a cluster-wide release costs the length of a block,
// and what it would order, the TMEM reads, has its own fences).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar, bool pred)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(static_cast<uint32_t>(pred))
                 : "memory");
}

// 2D tensor copy into this CTA's shared memory that completes on the barrier
// at `bar`, this CTA's or its pair's.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int32_t x,
                                                 int32_t y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// 2D tensor copy from shared memory to global memory (rows and columns outside
// the tensor are not written), in the thread's current group of such copies.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int32_t x,
                                             int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                     "l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit()
{
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the thread's last `kPending` groups have been read from shared memory.
template <int kPending>
__device__ __forceinline__ void tma_store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
// All of the thread's groups are done.
__device__ __forceinline__ void tma_store_wait()
{
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Makes the thread's shared-memory writes visible to tensor copies.
__device__ __forceinline__ void fence_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- TMEM reads

// 32 consecutive FP32 columns of the warp's 32 TMEM lanes (lane i of the warp
// reads lane 32 (warp mod 4) + i); valid after tmem_wait_ld().
#define FQ_R8(r, i) "=r"((r)[i]), "=r"((r)[i + 1]), "=r"((r)[i + 2]), "=r"((r)[i + 3]), \
                    "=r"((r)[i + 4]), "=r"((r)[i + 5]), "=r"((r)[i + 6]), "=r"((r)[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : FQ_R8(r, 0), FQ_R8(r, 8), FQ_R8(r, 16), FQ_R8(r, 24)
        : "r"(addr));
}
// 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : FQ_R8(r, 0), FQ_R8(r, 8)
        : "r"(addr));
}
#undef FQ_R8

// Waits for the warp's TMEM loads.  Their registers may be used after it only,
// by volatile statements, which stay behind it (passing 32 registers through
// the wait instead costs as many moves).
__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Registers a thread of the warpgroup may use from here on (the block keeps
// the registers it was launched with: the shares add up to them).
template <int kRegs>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The same where plain C++ uses the registers: they pass through the wait, so
// that no use of them is moved ahead of it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// Packed pairs of FP32 (lower half first).
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// acc += {lo, hi} * s, a pair of FMAs.
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t s)
{
    asm volatile("{\n\t.reg .b64 v;\n\t"
                 "mov.b64 v, {%1, %2};\n\t"
                 "fma.rn.f32x2 %0, v, %3, %0;\n\t}"
                 : "+l"(acc)
                 : "r"(lo), "r"(hi), "l"(s));
}
// acc += ({lo, hi} * {c0, c1}) * s.
__device__ __forceinline__ void mul_fma2(uint64_t &acc, uint32_t lo, uint32_t hi, uint32_t c0,
                                         uint32_t c1, uint64_t s)
{
    asm volatile("{\n\t.reg .b64 v, c;\n\t"
                 "mov.b64 v, {%1, %2};\n\t"
                 "mov.b64 c, {%3, %4};\n\t"
                 "mul.rn.f32x2 v, v, c;\n\t"
                 "fma.rn.f32x2 %0, v, %5, %0;\n\t}"
                 : "+l"(acc)
                 : "r"(lo), "r"(hi), "r"(c0), "r"(c1), "l"(s));
}

// Two FP32 -> packed BF16 (round to nearest even, lo in the low half).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- ragged groups

// The group structure of the offsets, in shared memory, by one warp:
// off[0..G] clamped into [0, M] and non-decreasing, off[0] = 0, off[G+1] = M;
// first[g] = number of `unit`-row tiles of the groups before g, a group's
// tiles starting at its first row; index G counts the rows that belong to no
// group (off[G]..M), first[G+1] is the total.  With offs == nullptr there is
// one group of all M rows (G = 1).  Returns (in every lane) whether the
// offsets given were malformed: off[0] != 0, decreasing, or outside [0, M].
__device__ inline bool load_row_groups(const int64_t *__restrict__ offs, int32_t G, int32_t M,
                                       int32_t unit, int32_t *off, int32_t *first)
{
    const int lane = threadIdx.x & 31;
    const int per = (G + 32) / 32;  // G + 1 entries over 32 lanes
    const int lo = min(lane * per, G + 1), hi = min(lo + per, G + 1);
    int32_t run = 0;
    for (int i = lo; i < hi; i++) {
        const int64_t v = offs ? offs[i] : (i == 0 ? 0 : M);
        run = max(run, i == 0 || v < 0 ? 0 : static_cast<int32_t>(v < M ? v : M));
        off[i] = run;
    }
    int32_t before = run;
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d)
            before = max(before, u);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (lane == 0)
        before = 0;
    bool bad = false;
    for (int i = lo; i < hi; i++) {
        off[i] = max(off[i], before);
        bad |= offs && offs[i] != off[i];
    }
    if (lane == 31)
        off[G + 1] = M;
    __syncwarp();
    int32_t sum = 0;
    for (int i = lo; i < hi; i++) {
        first[i] = sum;
        sum += (off[i + 1] - off[i] + unit - 1) / unit;
    }
    int32_t incl = sum;
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d)
            incl += u;
    }
    for (int i = lo; i < hi; i++)
        first[i] += incl - sum;
    if (lane == 31)
        first[G + 1] = incl;
    __syncwarp();
    return __any_sync(0xffffffffu, bad);
}

// Group of tile t: the last g in [0, n) with first[g] <= t.
__device__ __forceinline__ int group_of_tile(const int32_t *first, int n, int32_t t)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

}  // namespace fq
