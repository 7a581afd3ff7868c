// Block-scaled FP8 matrix product, dense and per expert on ragged row groups.
//
// Source: "Practical FP4 Training for Large-Scale MoE Models on Hopper GPUs",
// technical overview section 2 (items 1-3): E4M3 operands with 128-element
// blocks and FP32 block scales feed the expert products, whose token groups
// are ragged and unpadded.
//
//   C[m, n] = sum_b sa[m, b] * sb[n, b] * ( sum_{k in block b} A[m, k] B[n, k] )
//
// b runs over the 128-element blocks of K.  The inner sums are tensor-core
// products (kind::f8f6f4, FP32 accumulation); the outer sum is kept in FP32
// registers: one multiply sa * sb per row and block and one FMA per element.
#include "fq_tc.cuh"

namespace fq {

namespace {

constexpr int kRowsM = 128;       // rows of c of a CTA (its TMEM lanes)
constexpr int kBlockK = 128;      // one scale block, one pipeline stage
constexpr int kPromoteWarps = 8;  // two warpgroups
constexpr int kMmThreads = (kPromoteWarps + 4) * 32;
// Registers of a promoting and of another thread: 384 threads x 168 at launch =
// 64512 = 256 x 200 + 128 x 104 = 256 x 208 + 128 x 88.  The other roles' spills
// cost 10 to 20 % (at 56); with a scale per column the promoting warps need more.
constexpr int promote_regs(bool col_scale) { return col_scale ? 208 : 200; }
constexpr int other_regs(bool col_scale) { return col_scale ? 88 : 104; }
constexpr int kRaster = 8;        // row tiles walked together over the columns
constexpr int kScaleBlocks = 4;   // blocks whose scales are fetched together
constexpr int kBoxCols = 32;      // columns of c that a warp writes at once

// kCtas CTAs work on a tile of 128 kCtas rows.  Columns of the tile: 256 for a
// pair, 128 for one CTA.
template <int kCtas>
struct Shape {
    static constexpr int bn = 128 * kCtas;
    static constexpr int cols = bn / 2;               // of a promoting thread
    static constexpr int a_bytes = kRowsM * kBlockK;  // of a stage of a CTA
    static constexpr int b_rows = bn / kCtas;
    static constexpr int b_bytes = b_rows * kBlockK;
    static constexpr int stages = 5;
};

// Boxes of 32 rows x kBoxCols columns of c, staged by a warp.
template <bool kF32>
struct Box {
    static constexpr int row = kBoxCols * (kF32 ? 4 : 2);
    static constexpr int bytes = 32 * row;
    static constexpr int count = kF32 ? 1 : 2;
};

// What the second operand's scales and the tiles are:
//   kTileScale  forward, one scale per 128x128 weight tile
//   kRowScale   forward, one scale per weight row and block
//   kWgrad      weight gradient: per group, sum over its 128-token blocks of
//               products of transposed operands, both with a scale per row
//               and block
enum Mode { kTileScale, kRowScale, kWgrad };

// Shared memory behind the operand stages and the staged output.
template <int kCtas>
struct MmTail {
    using S = Shape<kCtas>;
    uint64_t full[S::stages], empty[S::stages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t scale_full[2], scale_empty[2];
    uint32_t tmem;
    int32_t abort;
    // column scales of two groups of kScaleBlocks blocks
    alignas(16) float col_scale[2][kScaleBlocks][S::bn];
    // int32 off[G + 2], first[G + 2] follow
};

struct MmArgs {
    const float *sa, *sb;
    const int64_t *offs;
    void *c;
    int32_t *dev_status;
    int32_t G;
    int32_t M;        // tokens
    int32_t R, N;     // rows (weight gradient only) and columns of c
    int32_t KB;       // 128-element blocks of K (forward only)
    int32_t sb_rows;  // rows of sb per group (forward only)
    int32_t add;      // weight gradient: c += instead of c =
};

// One output tile.
struct Tile {
    int32_t g;          // group
    int32_t row, n0;    // first row and column in c (row: in the group's matrix for kWgrad)
    int32_t end;        // rows of c end here
    int32_t blocks;     // blocks to add up
    int32_t xblk;       // first block's index along K
    int32_t arow, brow; // operand rows
};

// Row tile, column tile of the tile index: kRaster row tiles share a walk over
// the columns, so that the operands of the tiles in flight stay in L2.
__device__ __forceinline__ void tile_coords(int32_t idx, int32_t mt, int32_t nt, int32_t &i,
                                            int32_t &j)
{
    const int32_t band = idx / (kRaster * nt);
    const int32_t rows = min(kRaster, mt - band * kRaster);
    const int32_t r = idx - band * kRaster * nt;
    j = r / rows;
    i = band * kRaster + r - j * rows;
}

template <Mode kMode, int kCtas>
__device__ __forceinline__ Tile tile_at(int32_t idx, const MmArgs &p, const int32_t *off,
                                        const int32_t *first, int32_t mt, int32_t nt)
{
    constexpr int kRows = kCtas * kRowsM, BN = Shape<kCtas>::bn;
    Tile t;
    int32_t i, j;
    if (kMode == kWgrad) {
        t.g = idx / (mt * nt);
        tile_coords(idx - t.g * mt * nt, mt, nt, i, j);
        t.row = t.arow = i * kRows;
        t.n0 = t.brow = j * BN;
        t.end = p.R;
        t.blocks = first[t.g + 1] - first[t.g];
        t.xblk = first[t.g];
    } else {
        tile_coords(idx, mt, nt, i, j);
        t.g = group_of_tile(first, p.G + 1, i);
        t.row = t.arow = off[t.g] + (i - first[t.g]) * kRows;
        t.n0 = j * BN;
        t.brow = t.g * p.N + t.n0;
        t.end = off[t.g + 1];
        t.blocks = t.g < p.G ? p.KB : 0;  // rows of no group are 0
        t.xblk = 0;
    }
    return t;
}

// Byte of 16-byte piece i of row r in a box: the swizzle of a tensor copy of
// rows of 64 (BF16) or 128 (FP32) bytes.
template <bool kF32>
__device__ __forceinline__ int box_at(int r, int i)
{
    return Box<kF32>::row * r + 16 * (kF32 ? i ^ (r & 7) : i ^ ((r >> 1) & 3));
}

// A warp's box, from registers (lane l holds row l, packed pairs of columns).
template <bool kF32>
__device__ __forceinline__ void stage_box(uint8_t *box, const uint64_t *acc)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < Box<kF32>::row / 16; i++) {
        uint4 *to = reinterpret_cast<uint4 *>(box + box_at<kF32>(lane, i));
        float v[8];
        if (kF32) {
            unpack2(acc[2 * i], v[0], v[1]);
            unpack2(acc[2 * i + 1], v[2], v[3]);
            *to = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                             __float_as_uint(v[3]));
        } else {
#pragma unroll
            for (int h = 0; h < 4; h++)
                unpack2(acc[4 * i + h], v[2 * h], v[2 * h + 1]);
            *to = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                             cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
        }
    }
}

// The staged box by ordinary stores, a row at a time: where the group's rows end
// inside the box, where rows of c are not 16-byte aligned, and for c += box, whose
// loads are waited for one by one (65536 tokens, 32 x 2048 x 7168: 1511 -> 7075 us).
template <bool kF32, bool kAdd>
__device__ __forceinline__ void store_box(void *c, const uint8_t *box, int64_t row0, int32_t rows,
                                          int32_t col, int32_t N)
{
    const int e = threadIdx.x & 31, b = e * (kF32 ? 4 : 2);
    if (col + e >= N)
        return;
    for (int r = 0; r < rows; r++) {
        const uint8_t *from = box + box_at<kF32>(r, b >> 4) + (b & 15);
        const int64_t at = (row0 + r) * N + col + e;
        if (kF32) {
            float v = *reinterpret_cast<const float *>(from);
            if (kAdd)
                v += static_cast<float *>(c)[at];
            static_cast<float *>(c)[at] = v;
        } else {
            static_cast<uint16_t *>(c)[at] = *reinterpret_cast<const uint16_t *>(from);
        }
    }
}

// acc += the BF16 values c holds (before the one rounding).  Two bytes a lane from
// as many rows (the case above: 1460 -> 3431 us).
template <int kCols>
__device__ __forceinline__ void add_bf16(const void *c, int64_t row_off, int32_t col, int32_t N,
                                         uint64_t *acc)
{
#pragma unroll
    for (int i = 0; i < kCols / 2; i++) {
        float v[2];
        unpack2(acc[i], v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; h++)
            if (col + 2 * i + h < N)
                v[h] += bf16_lo(static_cast<const uint16_t *>(c)[row_off + col + 2 * i + h]);
        acc[i] = pack2(__float_as_uint(v[0]), __float_as_uint(v[1]));
    }
}

// The tiles of a cluster, in order: a lane works out one of the next 32, a
// shuffle hands the next one to the warp (the divisions and the search for the
// group take longer than a block).
template <Mode kMode, int kCtas>
struct TileWalk {
    Tile mine;
    int32_t idx, step, ntiles, mt, nt;
    int32_t n;

    __device__ __forceinline__ TileWalk(int32_t idx0, int32_t stride, int32_t rows, int32_t cols,
                                        int32_t total)
        : idx(idx0), step(stride), ntiles(total), mt(rows), nt(cols), n(0)
    {
    }
    // Whether there is another tile; next() then returns it.
    __device__ __forceinline__ bool more() const { return idx < ntiles; }
    __device__ __forceinline__ Tile next(const MmArgs &p, const int32_t *off, const int32_t *first)
    {
        if ((n & 31) == 0) {
            const int64_t at = idx + static_cast<int64_t>(threadIdx.x & 31) * step;
            mine = tile_at<kMode, kCtas>(static_cast<int32_t>(min(at, static_cast<int64_t>(ntiles - 1))),
                                         p, off, first, mt, nt);
        }
        Tile t;
        const int src = n & 31;
        t.g = __shfl_sync(0xffffffffu, mine.g, src);
        t.row = __shfl_sync(0xffffffffu, mine.row, src);
        t.n0 = __shfl_sync(0xffffffffu, mine.n0, src);
        t.end = __shfl_sync(0xffffffffu, mine.end, src);
        t.blocks = __shfl_sync(0xffffffffu, mine.blocks, src);
        t.xblk = __shfl_sync(0xffffffffu, mine.xblk, src);
        t.arow = __shfl_sync(0xffffffffu, mine.arow, src);
        t.brow = __shfl_sync(0xffffffffu, mine.brow, src);
        n++;
        idx = idx > ntiles - step ? ntiles : idx + step;
        return t;
    }
};

// The scales of one line (a row of c, a column or a weight tile) for up to
// kScaleBlocks consecutive blocks, `step` floats apart, from `s` on; `vec`: the
// four are one aligned vector.
__device__ __forceinline__ float4 load_scales(const float *s, int64_t step, int32_t n, bool vec)
{
    if (vec)
        return __ldg(reinterpret_cast<const float4 *>(s));
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n > 0)
        v.x = __ldg(s);
    if (n > 1)
        v.y = __ldg(s + step);
    if (n > 2)
        v.z = __ldg(s + 2 * step);
    if (n > 3)
        v.w = __ldg(s + 3 * step);
    return v;
}

// Persistent: one CTA per SM, in clusters of kCtas.  Every CTA loads 128 rows of
// a and its share of the rows of b per block and owns 128 rows of the
// accumulator.  Warps 0-7 add up the scaled blocks (warp w: TMEM lanes 32 (w mod
// 4).., half w / 4 of the columns), warp 8 issues the tensor copies, warp 9 of
// the cluster's first CTA the MMAs, warp 10 fetches the scales of the columns
// where every column has its own.  Two TMEM buffers: the MMAs of block b + 1 run
// while block b is scaled and added.
//
// What bounds it.  A block of a 256 x 256 tile takes the tensor cores 512 cycles
// and its operands 64 KB of shared-memory traffic per SM (512 cycles as well), but
// the warps 0-7 about 820: the TMEM loads, 64 packed FMAs a thread (256 cycles for
// the two warps of a scheduler) and about 20 more instructions a warp at their full
// latency, which two warps a scheduler do not hide.  16384 x 4096 x 7168: 337 us
// (2.86 PFLOP/s) with the L2 flushed, 375 us back to back at the lower clocks that
// this draws; without scaling and adding the same loop takes 285 us.  With a scale
// per column it is twice the FMAs and a shared load per four columns: 540 us.
// Why so: pairs of CTAs halve the traffic of b (one CTA a tile: 415 us before the
// rest); 256 accumulator columns need 128 registers a thread, so the other roles
// give theirs up, down to 104 (at 56 they spill, and the kernel takes 10 to 20 %
// longer); 192-column tiles wait more often per column (410
// us); half-tile MMAs read a twice (500 us); 16 adding warps have too few registers
// (414 us and more).
template <int kCtas, Mode kMode, bool kF32>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                      const __grid_constant__ CUtensorMap tc, const MmArgs p)
{
    using S = Shape<kCtas>;
    using B = Box<kF32>;
    constexpr int BN = S::bn, kCols = S::cols, kStages = S::stages;
    constexpr int kTmemCols = 256 * kCtas, kBufCols = kTmemCols / 2;
    constexpr bool kColScale = kMode != kTileScale;
    constexpr int kCopyWarp = kPromoteWarps, kMmaWarp = kCopyWarp + 1, kColWarp = kMmaWarp + 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sA = smem, *sB = sA + kStages * S::a_bytes, *sC = sB + kStages * S::b_bytes;
    MmTail<kCtas> &t =
        *reinterpret_cast<MmTail<kCtas> *>(sC + kPromoteWarps * B::count * B::bytes);
    int32_t *off = reinterpret_cast<int32_t *>(&t + 1), *first = off + p.G + 2;

    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 1 ? 0 : cluster_rank();
    if (wid == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; i++) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < 2; i++) {
                mbar_init(&t.acc_full[i], 1);
                mbar_init(&t.acc_empty[i], kCtas * kPromoteWarps);
                mbar_init(&t.scale_full[i], 1);
                mbar_init(&t.scale_empty[i], kPromoteWarps);
            }
            t.abort = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc<kCtas>(&t.tmem, kTmemCols);
    }
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    if (wid == 0) {
        const bool bad = load_row_groups(p.offs, p.G, p.M, kMode == kWgrad ? 128 : kCtas * kRowsM,
                                         off, first);
        if (bad && p.dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(p.dev_status, 1);
    }
    tc_fence_before();
    __syncthreads();
    if (kCtas > 1) {  // the barriers of both CTAs are set up
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    const uint32_t tmem = t.tmem;
    volatile int32_t *abort = &t.abort;
    const int32_t mt = kMode == kWgrad ? (p.R + kCtas * kRowsM - 1) / (kCtas * kRowsM)
                                       : first[p.G + 1];
    const int32_t nt = (p.N + BN - 1) / BN;
    const int32_t ntiles = mt * nt * (kMode == kWgrad ? p.G : 1);
    TileWalk<kMode, kCtas> walk(blockIdx.x / kCtas, gridDim.x / kCtas, mt, nt, ntiles);

    if (wid >= kPromoteWarps) {
        regs_down<other_regs(kColScale)>();
        if (wid == kCopyWarp) {
            const uint32_t full0 = smem_u32(t.full), empty0 = smem_u32(t.empty);
            const uint32_t fill0 = kCtas == 1 ? full0 : cluster_addr(t.full, 0);
            const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
            uint32_t s = 0, ph = 1;
            while (!*abort && walk.more()) {
                const Tile tl = walk.next(p, off, first);
                const int32_t arow = tl.arow + rank * kRowsM, brow = tl.brow + rank * S::b_rows;
                int32_t x = tl.xblk * kBlockK;
                for (int32_t b = 0; b < tl.blocks; b++, x += kBlockK) {
                    warp_wait(empty0 + 8 * s, ph, abort);
                    if (*abort)
                        break;
                    if (elect_one()) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&t.full[s], kCtas * (S::a_bytes + S::b_bytes));
                        if (kCtas == 1) {
                            tma_load_2d(sA + s * S::a_bytes, &ta, x, arow, &t.full[s]);
                            tma_load_2d(sB + s * S::b_bytes, &tb, x, brow, &t.full[s]);
                        } else {
                            tma_load_2d_pair(a0 + s * S::a_bytes, &ta, x, arow, fill0 + 8 * s);
                            tma_load_2d_pair(b0 + s * S::b_bytes, &tb, x, brow, fill0 + 8 * s);
                        }
                    }
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // every stage has been consumed: the last arrivals of the MMAs, which
            // come from the pair's first CTA, find this CTA's barriers
            for (int k = 0; k < kStages; k++) {
                warp_wait(empty0 + 8 * s, ph, abort);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (*abort) {  // no copy may land after the CTA is gone: a millisecond is plenty
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000)
                    ;
            }
        } else if (wid == kMmaWarp && rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kCtas * kRowsM, BN);
            const uint64_t da0 = smem_desc_sw128(sA), db0 = smem_desc_sw128(sB);
            const uint32_t full0 = smem_u32(t.full), empty0 = smem_u32(t.empty);
            const uint32_t acc_full0 = smem_u32(t.acc_full), acc_empty0 = smem_u32(t.acc_empty);
            uint32_t s = 0, ph = 0, it = 0;
            uint64_t da = da0, db = db0;
            while (!*abort && walk.more()) {
                const int32_t blocks = walk.next(p, off, first).blocks;
                for (int32_t b = 0; b < blocks; b++, it++) {
                    const uint32_t buf = it & 1;
                    warp_wait(full0 + 8 * s, ph, abort);
                    warp_wait(acc_empty0 + 8 * buf, ((it >> 1) & 1) ^ 1, abort);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBlockK / 32; k++)
                            mma_e4m3<kCtas>(tmem + buf * kBufCols, da + 2 * k, db + 2 * k, idesc, k > 0);
                        mma_commit<kCtas>(acc_full0 + 8 * buf);
                        mma_commit<kCtas>(empty0 + 8 * s);
                    }
                    s++;
                    da += S::a_bytes >> 4;
                    db += S::b_bytes >> 4;
                    if (s == kStages) {
                        s = 0;
                        ph ^= 1;
                        da = da0;
                        db = db0;
                    }
                }
            }
            if (*abort) {  // no MMA may be in flight when TMEM is freed
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000)
                    ;
            }
        } else if (kColScale && wid == kColWarp) {
            constexpr int kPer = BN / 32;  // columns of a lane
            const bool vec = kMode == kRowScale && p.KB % 4 == 0;
            uint32_t gq = 0;
            while (!*abort && walk.more()) {
                const Tile tl = walk.next(p, off, first);
                for (int32_t b = 0; b < tl.blocks; b += kScaleBlocks, gq++) {
                    const uint32_t slot = gq & 1;
                    warp_wait(smem_u32(&t.scale_empty[slot]), ((gq >> 1) & 1) ^ 1, abort);
#pragma unroll
                    for (int i = 0; i < kPer; i += 2) {
                        float4 v[2];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int32_t col = min(tl.n0 + lane + 32 * (i + h), p.N - 1);
                            const float *s =
                                kMode == kWgrad
                                    ? p.sb + static_cast<int64_t>(tl.xblk + b) * p.N + col
                                    : p.sb + (static_cast<int64_t>(tl.g) * p.N + col) * p.KB + b;
                            v[h] = load_scales(s, kMode == kWgrad ? p.N : 1, tl.blocks - b, vec);
                        }
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            float *to = &t.col_scale[slot][0][lane + 32 * (i + h)];
                            to[0] = v[h].x;
                            to[BN] = v[h].y;
                            to[2 * BN] = v[h].z;
                            to[3 * BN] = v[h].w;
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&t.scale_full[slot]);
                }
            }
        }
        __syncwarp();
    } else {
        regs_up<promote_regs(kColScale)>();
        const int half = wid >> 2;
        const uint32_t lane_base =
            tmem + (static_cast<uint32_t>(32 * (wid & 3)) << 16) + half * kCols;
        const bool aligned = static_cast<int64_t>(p.N) * (kF32 ? 4 : 2) % 16 == 0;
        uint8_t *stage = sC + wid * B::count * B::bytes;
        const bool leader = lane == 0;
        const uint32_t acc_full0 = smem_u32(t.acc_full);
        const uint32_t read0 = kCtas == 1 ? smem_u32(t.acc_empty) : cluster_addr(t.acc_empty, 0);
        const uint32_t scale_full0 = smem_u32(t.scale_full), scale_empty0 = smem_u32(t.scale_empty);
        uint32_t it = 0, gq = 0, nbox = 0;
        // The scales of the row and (kTileScale) of the weight tile that the columns
        // lie in, fetched two blocks ahead: those of a tile's first blocks before the
        // output of the tile before.
        const int64_t step = kMode == kWgrad ? p.R : 1;
        const float *sa = nullptr, *sb = nullptr;
        float a0 = 0.0f, a1 = 0.0f, b0 = 1.0f, b1 = 1.0f;
        auto open_tile = [&](const Tile &t) {
            const int32_t row = t.row + rank * kRowsM + 32 * (wid & 3) + lane;
            if (kMode == kWgrad)
                sa = p.sa + static_cast<int64_t>(t.xblk) * p.R + min(row, p.R - 1);
            else
                sa = p.sa + static_cast<int64_t>(min(row, p.M - 1)) * p.KB;
            if (!kColScale)
                sb = p.sb + (static_cast<int64_t>(t.g) * p.sb_rows +
                             min((t.n0 + half * kCols) / 128, p.sb_rows - 1)) * p.KB;
            if (t.blocks > 0) {
                a0 = __ldg(sa);
                if (!kColScale)
                    b0 = __ldg(sb);
            }
            if (t.blocks > 1) {
                a1 = __ldg(sa + step);
                if (!kColScale)
                    b1 = __ldg(sb + 1);
            }
            sa += 2 * step;
            sb += 2;
        };
        bool more = walk.more();
        Tile next = {};
        if (more) {
            next = walk.next(p, off, first);
            open_tile(next);
        }
        while (more && !*abort) {
            const Tile tl = next;
            const int32_t blocks = tl.blocks;
            const int32_t col0 = tl.n0 + half * kCols;
            const int32_t row0 = tl.row + rank * kRowsM + 32 * (wid & 3);
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int e = 0; e < kCols / 2; e++)
                acc[e] = 0;
            // A wait that gives up does not leave the loop (the other warps' waits
            // end soon as well); the flag is looked at behind it.
#pragma unroll 1
            for (int32_t b = 0; b < blocks; b++, it++) {
                const float s = kColScale ? a0 : a0 * b0;
                a0 = a1;
                b0 = b1;
                if (b + 2 < blocks) {
                    a1 = __ldg(sa);
                    sa += step;
                    if (!kColScale)
                        b1 = __ldg(sb++);
                }
                const uint32_t buf = it & 1, slot = gq & 1;
                const float *cols = &t.col_scale[slot][b % kScaleBlocks][half * kCols];
                if (kColScale && b % kScaleBlocks == 0)
                    warp_wait(scale_full0 + 8 * slot, (gq >> 1) & 1, abort);
                warp_wait(acc_full0 + 8 * buf, (it >> 1) & 1, abort);
                tc_fence_after();
                const uint64_t sc = pack2(__float_as_uint(s), __float_as_uint(s));
                const uint32_t addr = lane_base + buf * kBufCols;
                // kChunk columns at a time; with a scale per column, those of the
                // chunk are fetched while it is on its way (16 columns: registers)
                constexpr int kChunk = kColScale ? 16 : 32;
#pragma unroll
                for (int c = 0; c < kCols / kChunk; c++) {
                    uint32_t r[kChunk];
                    uint4 cs[kColScale ? 4 : 1];
                    if (kColScale) {
                        tmem_ld16(addr + kChunk * c, r);
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            cs[kColScale ? q : 0] =
                                *reinterpret_cast<const uint4 *>(cols + kChunk * c + 4 * q);
                    } else {
                        tmem_ld32(addr + kChunk * c, r);
                    }
                    tmem_wait_ld();
                    if (c + 1 == kCols / kChunk) {  // the buffer has been read
                        tc_fence_before();
                        mbar_arrive_cluster(read0 + 8 * buf, leader);
                    }
                    uint64_t *o = acc + kChunk / 2 * c;
#pragma unroll
                    for (int e = 0; e < kChunk; e += 4) {
                        if (kColScale) {
                            const uint4 q = cs[kColScale ? e / 4 : 0];
                            mul_fma2(o[e / 2], r[e], r[e + 1], q.x, q.y, sc);
                            mul_fma2(o[e / 2 + 1], r[e + 2], r[e + 3], q.z, q.w, sc);
                        } else {
                            fma2(o[e / 2], r[e], r[e + 1], sc);
                            fma2(o[e / 2 + 1], r[e + 2], r[e + 3], sc);
                        }
                    }
                }
                if (kColScale && (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks)) {
                    __syncwarp();
                    mbar_arrive_cluster(scale_empty0 + 8 * slot, leader);
                    gq++;
                }
            }
            more = walk.more();
            if (more) {
                next = walk.next(p, off, first);
                open_tile(next);
            }
            const bool ok = __all_sync(0xffffffffu, *abort == 0);
            const int32_t rows = min(32, tl.end - row0);
            if (ok && rows > 0) {
                const int64_t out0 = (kMode == kWgrad ? static_cast<int64_t>(tl.g) * p.R : 0) + row0;
                const bool add = kMode == kWgrad && p.add;
                const bool bulk = aligned && rows == 32 && !add;
                if (!kF32 && add && lane < rows)
                    add_bf16<kCols>(p.c, (out0 + lane) * p.N, col0, p.N, acc);
#pragma unroll
                for (int x = 0; x < kCols / kBoxCols; x++) {
                    const int32_t col = col0 + kBoxCols * x;
                    if (col >= p.N)
                        continue;
                    // the box used B::count boxes ago has been read
                    uint8_t *box = stage + nbox % B::count * B::bytes;
                    nbox++;
                    if (lane == 0)
                        tma_store_wait_read<B::count - 1>();
                    __syncwarp();
                    stage_box<kF32>(box, acc + kBoxCols / 2 * x);
                    fence_async_shared();
                    __syncwarp();
                    if (!bulk) {
                        if (add)
                            store_box<kF32, true>(p.c, box, out0, rows, col, p.N);
                        else
                            store_box<kF32, false>(p.c, box, out0, rows, col, p.N);
                        __syncwarp();
                    }
                    if (lane == 0) {
                        if (bulk)
                            tma_store_2d(&tc, box, col, static_cast<int32_t>(out0));
                        tma_store_commit();  // a group for every box
                    }
                }
            }
        }
        if (lane == 0)
            tma_store_wait();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (kCtas > 1) {  // nothing of the pair reaches into this CTA any more
        cluster_arrive();
        cluster_wait();
    }
    if (wid == kMmaWarp)
        tmem_free<kCtas>(tmem, kTmemCols);
    if (threadIdx.x == 0 && t.abort && p.dev_status)
        atomicOr(p.dev_status, 2);
}

// Both operands: [rows, K bytes] matrices cut into 128-byte blocks along K.
template <int kCtas, Mode kMode, bool kF32>
fq_status launch_matmul(const uint8_t *a, int64_t a_rows, const uint8_t *b, int64_t b_rows,
                        int64_t K, int64_t c_rows, const MmArgs &p, cudaStream_t st)
{
    using S = Shape<kCtas>;
    using B = Box<kF32>;
    constexpr int kSize = kF32 ? 4 : 2;
    CUtensorMap ta, tb, tc = {};
    bool ok = encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, a_rows, K, kBlockK,
                                   kRowsM, CU_TENSOR_MAP_SWIZZLE_128B, true) &&
              encode_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K, b_rows, K, kBlockK,
                                   S::b_rows, CU_TENSOR_MAP_SWIZZLE_128B, true);
    if (static_cast<int64_t>(p.N) * kSize % 16 == 0)  // otherwise c is not written by tensor copies
        ok = ok && encode_tensor_map_2d(&tc, kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                        p.c, p.N, c_rows, static_cast<uint64_t>(p.N) * kSize,
                                        kBoxCols, 32, kF32 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                           : CU_TENSOR_MAP_SWIZZLE_64B, false);
    if (!ok) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    const auto kern = fp8_matmul_kernel<kCtas, kMode, kF32>;
    const size_t dyn = 1024 + S::stages * (S::a_bytes + S::b_bytes) +
                       kPromoteWarps * B::count * B::bytes + sizeof(MmTail<kCtas>) +
                       2 * (p.G + 2) * sizeof(int32_t);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int64_t rows = kCtas * kRowsM, nt = (p.N + S::bn - 1) / S::bn;
    const int64_t tiles = kMode == kWgrad ? (p.R + rows - 1) / rows * nt * p.G
                                          : ((p.M + rows - 1) / rows + p.G + 1) * nt;
    const int64_t most = sm_count() / kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kCtas * (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, ta, tb, tc, p) != cudaSuccess)
        return launch_status();
    return launch_status();
}

// ---------------------------------------------------------------- few rows

// The product for few rows per group (a decode step): the weights are read once
// and bound the time, so the roles are swapped.  The 128 rows of the MMA are
// weight rows (columns of c), its columns kT rows of a, and what is in flight is
// weights: 2 CTAs per SM with 4 to 6 stages of 16 KB of them (3 CTAs with 4 stages
// were 8 % slower, 1 CTA with 11 stages 5 %).  A lane of the
// accumulator is a column of c; a block's products are scaled by the row's scale,
// which a shuffle hands round.  With few tiles the blocks of K are split over a
// cluster of S CTAs, whose sums are added through shared memory in rank order.
// Bound by HBM: 512 rows over 32 experts of 4096 x 7168 in 152 to 163 us, 5.8 to 6.2
// TB/s; one row through 14336 x 4096 in 15.6 us, 3.8 TB/s, of which the launch, the
// set-up and the first and last bytes' latency are about 6 us.
template <int kT>
struct Few {
    // CTAs per SM and their stages: about 200 KB of weights in flight per SM
    static constexpr int per_sm = 2;
    static constexpr int stages = kT == 16 ? 6 : (kT == 32 ? 5 : 4);
    static constexpr int w_bytes = 128 * kBlockK, x_bytes = kT * kBlockK;
    static constexpr int tmem_cols = 128, bufs = tmem_cols / kT;
    static constexpr int threads = 6 * 32;
};

template <int kT>
struct FewTail {
    uint64_t full[Few<kT>::stages], empty[Few<kT>::stages];
    uint64_t acc_full[Few<kT>::bufs], acc_empty[Few<kT>::bufs];
    uint32_t tmem;
    int32_t abort;
    // int32 off[G + 2], first[G + 2] follow
};

// Warps 0-3 add up the blocks, warp 4 issues the tensor copies, warp 5 the MMAs.
template <int kT, Mode kMode, bool kF32>
__global__ void __launch_bounds__(Few<kT>::threads, Few<kT>::per_sm)
    fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                          const MmArgs p, const int32_t S)
{
    using F = Few<kT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem, *sX = sW + F::stages * F::w_bytes;
    FewTail<kT> &t = *reinterpret_cast<FewTail<kT> *>(sX + F::stages * F::x_bytes);
    int32_t *off = reinterpret_cast<int32_t *>(&t + 1), *first = off + p.G + 2;
    volatile int32_t *abort = &t.abort;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t rank = S > 1 ? static_cast<int32_t>(cluster_rank()) : 0;

    if (wid == 5) {
        if (lane == 0) {
            for (int i = 0; i < F::stages; i++) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < F::bufs; i++) {
                mbar_init(&t.acc_full[i], 1);
                mbar_init(&t.acc_empty[i], 4);
            }
            t.abort = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc<1>(&t.tmem, F::tmem_cols);
    }
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();  // the next kernel may start its set-up
    if (wid == 0) {
        const bool bad = load_row_groups(p.offs, p.G, p.M, kT, off, first);
        if (bad && p.dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(p.dev_status, 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = t.tmem;
    // row tiles of all groups run fastest: tiles in flight share weights
    const int32_t mt = first[p.G + 1], nt = (p.N + 127) / 128, ntiles = mt * nt;
    const int32_t b_lo = static_cast<int32_t>(static_cast<int64_t>(p.KB) * rank / S);
    const int32_t b_hi = static_cast<int32_t>(static_cast<int64_t>(p.KB) * (rank + 1) / S);
    const int32_t idx0 = blockIdx.x / S, step = gridDim.x / S;

    if (wid == 4) {
        uint32_t s = 0, ph = 1;
        for (int32_t idx = idx0; idx < ntiles && !*abort; idx += step) {
            const int32_t j = idx / mt, i = idx - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            if (g == p.G)
                continue;
            const int32_t row = off[g] + (i - first[g]) * kT, wrow = g * p.N + j * 128;
            for (int32_t b = b_lo; b < b_hi; b++) {
                warp_wait(smem_u32(&t.empty[s]), ph, abort);
                if (*abort)
                    break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&t.full[s], F::w_bytes + F::x_bytes);
                    tma_load_2d(sW + s * F::w_bytes, &tw, b * kBlockK, wrow, &t.full[s]);
                    tma_load_2d(sX + s * F::x_bytes, &tx, b * kBlockK, row, &t.full[s]);
                }
                if (++s == F::stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (*abort) {  // no copy may land after the CTA is gone: a millisecond is plenty
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000)
                ;
        }
    } else if (wid == 5) {
        constexpr uint32_t idesc = idesc_e4m3(128, kT);
        const uint64_t dw0 = smem_desc_sw128(sW), dx0 = smem_desc_sw128(sX);
        uint32_t s = 0, ph = 0, it = 0;
        for (int32_t idx = idx0; idx < ntiles && !*abort; idx += step) {
            if (group_of_tile(first, p.G + 1, idx % mt) == p.G)
                continue;
            for (int32_t b = b_lo; b < b_hi; b++, it++) {
                const uint32_t buf = it % F::bufs, bph = (it / F::bufs) & 1;
                warp_wait(smem_u32(&t.full[s]), ph, abort);
                warp_wait(smem_u32(&t.acc_empty[buf]), bph ^ 1, abort);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dw = dw0 + s * (F::w_bytes >> 4), dx = dx0 + s * (F::x_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < kBlockK / 32; k++)
                        mma_e4m3<1>(tmem + buf * kT, dw + 2 * k, dx + 2 * k, idesc, k > 0);
                    mma_commit<1>(smem_u32(&t.acc_full[buf]));
                    mma_commit<1>(smem_u32(&t.empty[s]));
                }
                if (++s == F::stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (*abort) {  // no MMA may be in flight when TMEM is freed
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000)
                ;
        }
    } else {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wid) << 16);
        constexpr int kHold = (kT + 31) / 32;  // rows' scales of a lane
        uint32_t it = 0;
        for (int32_t idx = idx0; idx < ntiles && !*abort; idx += step) {
            const int32_t j = idx / mt, i = idx - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            const int32_t row0 = off[g] + (i - first[g]) * kT;
            const int32_t rows = min(kT, off[g + 1] - row0);
            const int32_t n = j * 128 + 32 * wid + lane;
            float acc[kT];
#pragma unroll
            for (int e = 0; e < kT; e++)
                acc[e] = 0.0f;
            if (g < p.G) {
                const float *sa[kHold];
                float a[kHold], an[kHold];
#pragma unroll
                for (int h = 0; h < kHold; h++) {
                    sa[h] = p.sa + static_cast<int64_t>(
                                       min(row0 + min(lane + 32 * h, kT - 1), p.M - 1)) * p.KB;
                    a[h] = b_lo < b_hi ? __ldg(sa[h] + b_lo) : 0.0f;
                    an[h] = b_lo + 1 < b_hi ? __ldg(sa[h] + b_lo + 1) : 0.0f;
                }
                const float *sb = p.sb + (static_cast<int64_t>(g) * p.sb_rows +
                                          (kMode == kRowScale ? min(n, p.N - 1) : j)) * p.KB;
                float w = b_lo < b_hi ? __ldg(sb + b_lo) : 0.0f;
                float wn = b_lo + 1 < b_hi ? __ldg(sb + b_lo + 1) : 0.0f;
                for (int32_t b = b_lo; b < b_hi; b++, it++) {
                    const uint32_t buf = it % F::bufs, bph = (it / F::bufs) & 1;
                    float sc[kHold];
#pragma unroll
                    for (int h = 0; h < kHold; h++) {
                        sc[h] = kMode == kRowScale ? a[h] : a[h] * w;
                        a[h] = an[h];
                        if (b + 2 < b_hi)
                            an[h] = __ldg(sa[h] + b + 2);
                    }
                    const float wk = w;
                    w = wn;
                    if (b + 2 < b_hi)
                        wn = __ldg(sb + b + 2);
                    warp_wait(smem_u32(&t.acc_full[buf]), bph, abort);
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kT / 16; c++) {
                        uint32_t r[16];
                        tmem_ld16(lanes + buf * kT + 16 * c, r);
                        tmem_wait_ld16(r);
                        if (c + 1 == kT / 16) {  // the buffer has been read
                            tc_fence_before();
                            mbar_arrive_cluster(smem_u32(&t.acc_empty[buf]), lane == 0);
                        }
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const int col = 16 * c + e;
                            float v = __uint_as_float(r[e]);
                            if (kMode == kRowScale)
                                v *= wk;
                            acc[col] = __fmaf_rn(v, __shfl_sync(0xffffffffu, sc[col / 32], col % 32),
                                                 acc[col]);
                        }
                    }
                }
            }
            if (S == 1) {
                if (n < p.N && *abort == 0) {
#pragma unroll
                    for (int e = 0; e < kT; e++)
                        if (e < rows) {
                            const int64_t at = static_cast<int64_t>(row0 + e) * p.N + n;
                            if (kF32)
                                static_cast<float *>(p.c)[at] = acc[e];
                            else
                                static_cast<uint16_t *>(p.c)[at] =
                                    static_cast<uint16_t>(cvt_bf16x2(acc[e], 0.0f));
                        }
                }
            } else {  // one tile: its stages are free, every copy has been waited for
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int e = 0; e < kT; e++)
                    part[e * 128 + 32 * wid + lane] = acc[e];
            }
        }
    }
    if (S > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        // CTA r adds up rows r, r + S, .. of the tile
        if (wid < 4 && idx0 < ntiles && *abort == 0) {
            const int32_t j = idx0 / mt, i = idx0 - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            const int32_t row0 = off[g] + (i - first[g]) * kT;
            const int32_t rows = min(kT, off[g + 1] - row0);
            const int32_t n = j * 128 + 32 * wid + lane;
            for (int32_t e = rank; e < rows; e += S) {
                float v = 0.0f;
                const float *own = reinterpret_cast<const float *>(smem) + e * 128 + 32 * wid + lane;
                for (int32_t r = 0; r < S; r++)
                    v += ld_cluster_f32(cluster_addr(own, r));
                if (n < p.N) {
                    const int64_t at = static_cast<int64_t>(row0 + e) * p.N + n;
                    if (kF32)
                        static_cast<float *>(p.c)[at] = v;
                    else
                        static_cast<uint16_t *>(p.c)[at] = static_cast<uint16_t>(cvt_bf16x2(v, 0.0f));
                }
            }
        }
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (wid == 5)
        tmem_free<1>(tmem, F::tmem_cols);
    if (threadIdx.x == 0 && t.abort && p.dev_status)
        atomicOr(p.dev_status, 2);
}

template <int kT, Mode kMode, bool kF32>
fq_status launch_few(const uint8_t *a, const uint8_t *b, int64_t K, const MmArgs &p, cudaStream_t st)
{
    using F = Few<kT>;
    CUtensorMap tx, tw;
    if (!encode_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, p.M, K, kBlockK, kT,
                              CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K,
                              static_cast<uint64_t>(p.G) * p.N, K, kBlockK, 128,
                              CU_TENSOR_MAP_SWIZZLE_128B, true)) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    const auto kern = fp8_matmul_few_kernel<kT, kMode, kF32>;
    const size_t dyn = 1024 + F::stages * (F::w_bytes + F::x_bytes) + sizeof(FewTail<kT>) +
                       2 * (p.G + 2) * sizeof(int32_t);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int64_t nt = (p.N + 127) / 128;
    // with one group the tiles are known, otherwise at most so many
    const int64_t tiles = (p.offs ? p.M / kT + (p.G < p.M ? p.G : p.M) + 1 : (p.M + kT - 1) / kT) * nt;
    // The blocks of K are split while an SM has no more than one CTA (with 64 rows,
    // which keep a CTA longer, two): 112 tiles of 14336 x 4096 took 15 to 16 us for 1
    // to 32 rows unsplit, 17 to 20 us halved, 20 us in quarters.
    const int64_t sms = sm_count();
    int S = 1;
    const int64_t slots = (kT == 64 ? 2 : 1) * sms;
    while (S < 8 && tiles * S * 2 <= slots && 4 * S <= p.KB)
        S *= 2;
    const int64_t most = S > 1 ? tiles : F::per_sm * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(S * (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(F::threads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tx, tw, p, static_cast<int32_t>(S)) != cudaSuccess)
        return launch_status();
    return launch_status();
}

// Whether tiles of one CTA (128 x 128) finish before tiles of a pair (256 x 256):
// rounds over the SMs, a round of pairs counting for two, times `percent` of a
// pair's time for the same work.  Measured both ways: forward 125 (N x K 4096 x
// 7168, 512 rows: 128 tiles, one round 21.4 us, pairs 27.0; 1024 rows: 256 tiles, two
// rounds 37.6, pairs 28.2), weight gradient 104 (1003 tokens, 8 x 1408 x 2048: 10
// rounds 28.1 us, 6 of pairs 30.9; 16384 tokens, 16 x 2048 x 2048: 27 rounds 150, 14 of
// pairs 144).
inline bool one_cta_tiles(int64_t rows, int64_t cols, int64_t groups, int percent)
{
    const int64_t sms = sm_count(), pairs = sms > 1 ? sms / 2 : 1;
    const int64_t one = (rows + 127) / 128 * ((cols + 127) / 128) * groups;
    const int64_t two = (rows + 255) / 256 * ((cols + 255) / 256) * groups;
    return (one + sms - 1) / sms * percent < (two + pairs - 1) / pairs * 200;
}

template <Mode kMode, bool kF32>
fq_status launch_forward(const uint8_t *a, const uint8_t *b, int64_t K, const MmArgs &p,
                         cudaStream_t st)
{
    // Which kernel, by the mean rows of a group and the tiles (N x K 4096 x 7168
    // unless said otherwise; us):
    //   rows 32: few rows 9.9, one CTA a tile 19.9, pairs 26.4
    //   rows 64: 12.3 (K split eight ways), 19.9, 26.5; but 14336 x 4096, where it
    //            is not split: 24.0, 14.4, 18.8; 32 groups of 64: 176, 167, 197
    //   32 groups of 128 rows: one CTA a tile 175, pairs 201; of 256: 288, 227
    // The counts themselves are on the device.  4096 rows over 256 groups: 1272 even, 1333
    // with half of them in one group, 1307 with one row in all the others; all in one
    // group 416, where the pairs of a dense product take 102.
    const int64_t mean = (static_cast<int64_t>(p.M) + p.G - 1) / p.G;
    const int64_t sms = sm_count(), nt = (p.N + 127) / 128;
    const int64_t b_rows = static_cast<int64_t>(p.G) * p.N;
    if (mean <= 16)
        return launch_few<16, kMode, kF32>(a, b, K, p, st);
    if (mean <= 32)
        return launch_few<32, kMode, kF32>(a, b, K, p, st);
    if (mean <= 64 && 2 * nt * p.G <= sms)
        return launch_few<64, kMode, kF32>(a, b, K, p, st);
    if (p.G > 1 ? mean <= 128 : one_cta_tiles(p.M, p.N, 1, 125))
        return launch_matmul<1, kMode, kF32>(a, p.M, b, b_rows, K, p.M, p, st);
    return launch_matmul<2, kMode, kF32>(a, p.M, b, b_rows, K, p.M, p, st);
}

// The transposed operands (rows of M tokens) re-laid for the weight gradient:
// row r of the workspace holds the row's 128-token blocks, each at a multiple
// of 128 bytes and filled up with zeros.  The rows of M tokens start at any
// byte where M % 16 != 0, and the groups at any token: neither is a tensor
// copy's alignment.  A lane makes 16 bytes of kAlignRun consecutive blocks, each
// from five aligned words.  Bound by HBM (every byte read and written once): 65536
// tokens x 9216 rows in 212 us, 5.7 TB/s; a block at a time, with a division and a
// search each, took 325 us.
constexpr int kAlignRun = 4;
__global__ void __launch_bounds__(kThreads) align_blocks_kernel(
    const uint8_t *__restrict__ a, int32_t a_rows, const uint8_t *__restrict__ b, int32_t b_rows,
    int32_t M, const int64_t *__restrict__ offs, int32_t G, int64_t pitch, uint8_t *__restrict__ out,
    int32_t *dev_status)
{
    extern __shared__ int32_t dyn[];
    int32_t *off = dyn, *first = dyn + G + 2;
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    if (threadIdx.x < 32) {
        const bool bad = load_row_groups(offs, G, M, 128, off, first);
        if (bad && dev_status && blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(dev_status, 1);
    }
    __syncthreads();
    griddep_launch_dependents();
    const int32_t blocks = first[G];
    const int64_t rows = static_cast<int64_t>(a_rows) + b_rows;
    const int32_t runs = (blocks + kAlignRun - 1) / kAlignRun;
    const int64_t quads = (rows + 3) / 4, items = quads * runs;
    const int lane = threadIdx.x & 31, sub = lane >> 3, chunk = lane & 7;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
         w < items; w += step) {
        const int64_t quad = w / runs, r = 4 * quad + sub;
        const int32_t blk0 = static_cast<int32_t>(w - quad * runs) * kAlignRun;
        if (r >= rows)
            continue;
        const bool in_a = r < a_rows;
        const uint8_t *base = in_a ? a : b;
        const int64_t size = static_cast<int64_t>(in_a ? a_rows : b_rows) * M;
        const int64_t row = (in_a ? r : r - a_rows) * M;
        uint8_t *to = out + r * pitch + 16 * chunk;
        int g = group_of_tile(first, G + 1, blk0);
        uint32_t v[kAlignRun][5];
        int32_t len[kAlignRun];
        int64_t at[kAlignRun];
#pragma unroll
        for (int u = 0; u < kAlignRun; u++) {
            const int32_t blk = blk0 + u;
            len[u] = 0;
            if (blk >= blocks)
                continue;
            while (blk >= first[g + 1])
                g++;
            const int32_t t0 = off[g] + (blk - first[g]) * 128 + 16 * chunk;
            len[u] = min(16, off[g + 1] - t0);
            at[u] = row + t0;
            const int64_t w0 = at[u] >> 2;
            const uint32_t *from = reinterpret_cast<const uint32_t *>(base) + w0;
            if (len[u] <= 0) {
#pragma unroll
                for (int i = 0; i < 5; i++)
                    v[u][i] = 0;
            } else if (4 * w0 + 20 <= size) {
#pragma unroll
                for (int i = 0; i < 5; i++)
                    v[u][i] = __ldg(from + i);
            } else {  // the tensor's last bytes
#pragma unroll
                for (int i = 0; i < 5; i++) {
                    v[u][i] = 0;
                    for (int k = 0; k < 4; k++)
                        if (4 * (w0 + i) + k < size)
                            v[u][i] |= static_cast<uint32_t>(base[4 * (w0 + i) + k]) << (8 * k);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAlignRun; u++) {
            if (blk0 + u >= blocks)
                break;
            const int sh = 8 * static_cast<int>(at[u] & 3);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                o[i] = __funnelshift_r(v[u][i], v[u][i + 1], sh);
                const int keep = len[u] - 4 * i;
                if (keep < 4)
                    o[i] = keep > 0 ? o[i] & ((1u << (8 * keep)) - 1) : 0;
            }
            *reinterpret_cast<uint4 *>(to + static_cast<int64_t>(blk0 + u) * 128) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

}  // namespace

}  // namespace fq

extern "C" fq_status fp8_matmul(const uint8_t *a, const float *sa, int64_t M, int64_t K,
                                const uint8_t *b, const float *sb, int64_t N, int b_block,
                                const int64_t *group_offsets, int32_t G, void *c, int c_f32,
                                int32_t *dev_status, void *stream)
{
    using namespace fq;
    if (M < 0 || M > INT32_MAX - 512 || N <= 0 || K <= 0 || K % 128 != 0 || K > INT32_MAX - 128)
        return FQ_ERR_SHAPE;
    if (G < 1 || G > FQ_COLS_MAX_GROUPS || (b_block != 1 && b_block != 128) ||
        (c_f32 != 0 && c_f32 != 1) || (!group_offsets && G != 1))
        return FQ_ERR_ARG;
    // 32-bit rows of b and 32-bit tile indices
    if (N > (INT32_MAX - 512) / G || (M / 128 + G + 2) * (N / 128 + 1) > INT32_MAX / 2)
        return FQ_ERR_SHAPE;
    if (M == 0)
        return FQ_OK;
    if (!a || !sa || !b || !sb || !c)
        return FQ_ERR_NULL;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c) ||
        !aligned16(group_offsets))
        return FQ_ERR_ALIGN;
    MmArgs p = {};
    p.sa = sa;
    p.sb = sb;
    p.offs = group_offsets;
    p.c = c;
    p.dev_status = dev_status;
    p.G = G;
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.KB = static_cast<int32_t>(K / 128);
    p.sb_rows = b_block == 1 ? p.N : (p.N + 127) / 128;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (b_block == 1)
        return c_f32 ? launch_forward<kRowScale, true>(a, b, K, p, st)
                     : launch_forward<kRowScale, false>(a, b, K, p, st);
    return c_f32 ? launch_forward<kTileScale, true>(a, b, K, p, st)
                 : launch_forward<kTileScale, false>(a, b, K, p, st);
}

extern "C" int64_t fp8_matmul_wgrad_workspace(int64_t M, int64_t N, int64_t K, int32_t G)
{
    if (M < 0 || M > INT32_MAX - 512 || N <= 0 || K <= 0 || G < 1 || G > FQ_COLS_MAX_GROUPS ||
        N > INT32_MAX - 512 || K > INT32_MAX - 512)
        return -1;
    const int64_t pitch = 128 * fp4_to_fp8_cols_scale_capacity(M, G);
    if (pitch > INT32_MAX - 512 || N + K > INT64_MAX / pitch)  // 32-bit coordinates of the copies
        return -1;
    return (N + K) * pitch;
}

extern "C" fq_status fp8_matmul_wgrad(const uint8_t *aT, const float *aT_scale, int64_t N,
                                      const uint8_t *bT, const float *bT_scale, int64_t K,
                                      int64_t M, const int64_t *group_offsets, int32_t G,
                                      int64_t cap, void *c, int c_f32, int accumulate,
                                      void *workspace, int64_t workspace_bytes,
                                      int32_t *dev_status, void *stream)
{
    using namespace fq;
    const int64_t need = fp8_matmul_wgrad_workspace(M, N, K, G);
    if (G < 1 || G > FQ_COLS_MAX_GROUPS || (c_f32 != 0 && c_f32 != 1) ||
        (accumulate != 0 && accumulate != 1) || (!group_offsets && G != 1))
        return FQ_ERR_ARG;
    const int64_t mt = (N + 127) / 128, nt = (K + 127) / 128;
    if (need < 0 || mt > INT32_MAX / nt / G || N > INT32_MAX / G)  // 32-bit tiles and rows of c
        return FQ_ERR_SHAPE;
    // one group from token 0 on, rows of M tokens 16-byte aligned: the blocks lie
    // where tensor copies can fetch them
    const bool in_place = !group_offsets && M % 16 == 0;
    if (cap < fp4_to_fp8_cols_scale_capacity(M, G) || (!in_place && workspace_bytes < need))
        return FQ_ERR_ARG;
    if ((M > 0 && (!aT || !aT_scale || !bT || !bT_scale)) || !c || (!in_place && !workspace))
        return FQ_ERR_NULL;
    if (!aligned16(aT) || !aligned16(aT_scale) || !aligned16(bT) || !aligned16(bT_scale) ||
        !aligned16(c) || !aligned16(workspace) || !aligned16(group_offsets))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint8_t *wa = aT, *wb = bT;
    int64_t pitch = M;
    if (in_place && M == 0) {
        // no blocks, so no copies: the maps need an address and a size, not operands
        wa = wb = static_cast<const uint8_t *>(c);
        pitch = 128;
    } else if (!in_place) {
        const int64_t blocks = fp4_to_fp8_cols_scale_capacity(M, G);
        pitch = 128 * blocks;
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        wa = ws;
        wb = ws + N * pitch;
        const size_t dyn = 2 * (G + 2) * sizeof(int32_t);
        const int64_t warps = ((N + K + 3) / 4) * ((blocks + kAlignRun - 1) / kAlignRun);
        const int grid = persistent_grid(align_blocks_kernel, kThreads, dyn, (warps + 7) / 8);
        if (launch_pdl(align_blocks_kernel, dim3(grid), dim3(kThreads), dyn, st, aT,
                       static_cast<int32_t>(N), bT, static_cast<int32_t>(K), static_cast<int32_t>(M),
                       group_offsets, G, pitch, ws, dev_status) != cudaSuccess)
            return launch_status();
    }
    MmArgs p = {};
    p.sa = aT_scale;
    p.sb = bT_scale;
    p.offs = group_offsets;
    p.c = c;
    p.dev_status = dev_status;
    p.G = G;
    p.M = static_cast<int32_t>(M);
    p.R = static_cast<int32_t>(N);
    p.N = static_cast<int32_t>(K);
    p.add = accumulate;
    if (one_cta_tiles(N, K, G, 104))
        return c_f32 ? launch_matmul<1, kWgrad, true>(wa, N, wb, K, pitch, G * N, p, st)
                     : launch_matmul<1, kWgrad, false>(wa, N, wb, K, pitch, G * N, p, st);
    return c_f32 ? launch_matmul<2, kWgrad, true>(wa, N, wb, K, pitch, G * N, p, st)
                 : launch_matmul<2, kWgrad, false>(wa, N, wb, K, pitch, G * N, p, st);
}
