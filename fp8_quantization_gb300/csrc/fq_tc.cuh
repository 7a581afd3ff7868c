// Tensor-core (tcgen05 / TMEM) and ragged-group helpers shared by the FP8
// matrix products of libfq.so.
#pragma once

#include "fq_common.cuh"

namespace fq {

// ---------------------------------------------------------------- bounded waits

// Waits for phase `parity` of `bar` at most kWaitLimitNs; a wait that runs out
// raises the CTA's shared `abort` flag, at which every other wait of the CTA
// gives up too, so that all roles reach the kernel's end.
__device__ __forceinline__ bool mbar_wait_or_abort(uint64_t *bar, uint32_t parity,
                                                   volatile int32_t *abort)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort)
            return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// ---------------------------------------------------------------- tcgen05

// Columns of TMEM for the CTA (a power of two, 32..512); the base address is
// written to shared memory.  One full warp allocates and later frees.
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
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
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
                 : "memory");
}

// One arrival on `bar` once every tcgen05.mma this thread issued has finished.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

// 16 consecutive FP32 columns of the warp's 32 TMEM lanes (lane i of the warp
// reads lane 32 (warp mod 4) + i); valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// Waits for the warp's TMEM loads; the loaded registers pass through it so
// that no use of them is scheduled ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16])
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
