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

constexpr int kTileM = 128;      // rows of a tile (TMEM lanes)
constexpr int kBlockK = 128;     // one scale block, one pipeline stage
constexpr int kPromoteWarps = 8;
constexpr int kMmThreads = (kPromoteWarps + 2) * 32;
constexpr int kRaster = 16;      // row tiles walked together over the columns

// What the second operand's scales and the tiles are:
//   kTileScale  forward, one scale per 128x128 weight tile
//   kRowScale   forward, one scale per weight row and block
//   kWgrad      weight gradient: per group, sum over its 128-token blocks of
//               products of transposed operands, both with a scale per row
//               and block
enum Mode { kTileScale, kRowScale, kWgrad };

template <int BN>
struct MmShape {
    static constexpr int stages = BN == 256 ? 4 : 6;
    static constexpr int a_bytes = kTileM * kBlockK;
    static constexpr int b_bytes = BN * kBlockK;
    static constexpr int cols = BN / 2;  // columns of a promoting thread
};

// Shared memory behind the operand stages.
template <int BN>
struct MmTail {
    uint64_t full[MmShape<BN>::stages], empty[MmShape<BN>::stages];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
    int32_t abort;
    float col_scale[2][BN];
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

template <Mode kMode, int BN>
__device__ __forceinline__ Tile tile_at(int32_t idx, const MmArgs &p, const int32_t *off,
                                        const int32_t *first, int32_t mt, int32_t nt)
{
    Tile t;
    int32_t i, j;
    if (kMode == kWgrad) {
        t.g = idx / (mt * nt);
        tile_coords(idx - t.g * mt * nt, mt, nt, i, j);
        t.row = t.arow = i * kTileM;
        t.n0 = t.brow = j * BN;
        t.end = p.R;
        t.blocks = first[t.g + 1] - first[t.g];
        t.xblk = first[t.g];
    } else {
        tile_coords(idx, mt, nt, i, j);
        t.g = group_of_tile(first, p.G + 1, i);
        t.row = t.arow = off[t.g] + (i - first[t.g]) * kTileM;
        t.n0 = j * BN;
        t.brow = t.g * p.N + t.n0;
        t.end = off[t.g + 1];
        t.blocks = t.g < p.G ? p.KB : 0;  // rows of no group are 0
        t.xblk = 0;
    }
    return t;
}

// Columns [col, col + 16) of one output row from 8 packed pairs; `fast` rows
// are 16-byte aligned.
template <bool kF32>
__device__ __forceinline__ void store16(void *c, int64_t row_off, int32_t col, int32_t N, bool fast,
                                        const uint64_t *acc)
{
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; i++)
        unpack2(acc[i], v[2 * i], v[2 * i + 1]);
    if (kF32) {
        float *p = static_cast<float *>(c) + row_off + col;
        if (fast && col + 16 <= N) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                reinterpret_cast<float4 *>(p)[i] =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++)
                if (col + i < N)
                    p[i] = v[i];
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(c) + row_off + col;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
        if (fast && col + 16 <= N) {
            reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++)
                if (col + i < N)
                    p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// acc += the 16 columns that c holds.
template <bool kF32>
__device__ __forceinline__ void add16(const void *c, int64_t row_off, int32_t col, int32_t N,
                                      uint64_t *acc)
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[2];
        unpack2(acc[i], v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t at = row_off + col + 2 * i + h;
            if (col + 2 * i + h < N)
                v[h] += kF32 ? static_cast<const float *>(c)[at]
                             : bf16_lo(static_cast<const uint16_t *>(c)[at]);
        }
        acc[i] = pack2(__float_as_uint(v[0]), __float_as_uint(v[1]));
    }
}

// Persistent, one CTA per SM.  Warps 0-7 add up the scaled blocks (warp w:
// TMEM lanes 32 (w mod 4).., columns BN/2 * (w / 4)..), warp 8 issues the
// tensor copies, warp 9 the MMAs.  Two TMEM buffers of BN columns: the MMAs of
// block b + 1 run while block b is scaled and added.
template <int BN, Mode kMode, bool kF32>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                      const MmArgs p)
{
    using S = MmShape<BN>;
    constexpr bool kColScale = kMode != kTileScale;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sA = smem, *sB = smem + S::stages * S::a_bytes;
    MmTail<BN> &t = *reinterpret_cast<MmTail<BN> *>(sB + S::stages * S::b_bytes);
    int32_t *off = reinterpret_cast<int32_t *>(&t + 1), *first = off + p.G + 2;

    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (wid == 9) {
        if (lane == 0) {
            for (int i = 0; i < S::stages; i++) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < 2; i++) {
                mbar_init(&t.acc_full[i], 1);
                mbar_init(&t.acc_empty[i], kPromoteWarps);
            }
            t.abort = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc(&t.tmem, 2 * BN);
    }
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    if (wid == 0) {
        const bool bad = load_row_groups(p.offs, p.G, p.M, kTileM, off, first);
        if (bad && p.dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(p.dev_status, 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = t.tmem;
    const int32_t mt = kMode == kWgrad ? (p.R + kTileM - 1) / kTileM : first[p.G + 1];
    const int32_t nt = (p.N + BN - 1) / BN;
    const int32_t ntiles = mt * nt * (kMode == kWgrad ? p.G : 1);

    if (wid == 8) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int32_t idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x) {
                const Tile tl = tile_at<kMode, BN>(idx, p, off, first, mt, nt);
                for (int32_t b = 0; b < tl.blocks; b++, it++) {
                    const uint32_t s = it % S::stages, ph = (it / S::stages) & 1;
                    if (!(ok = mbar_wait_or_abort(&t.empty[s], ph ^ 1, &t.abort)))
                        break;
                    mbar_arrive_expect_tx(&t.full[s], S::a_bytes + S::b_bytes);
                    tma_load_2d(sA + s * S::a_bytes, &ta, (tl.xblk + b) * kBlockK, tl.arow, &t.full[s]);
                    tma_load_2d(sB + s * S::b_bytes, &tb, (tl.xblk + b) * kBlockK, tl.brow, &t.full[s]);
                }
            }
            if (!ok)  // no copy may land after the CTA is gone
                for (uint32_t k = it > S::stages ? it - S::stages : 0; k < it; k++)
                    mbar_wait(&t.full[k % S::stages], (k / S::stages) & 1);
        }
        __syncwarp();
    } else if (wid == 9) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kTileM, BN);
            uint32_t it = 0;
            bool ok = true;
            for (int32_t idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x) {
                const int32_t blocks = tile_at<kMode, BN>(idx, p, off, first, mt, nt).blocks;
                for (int32_t b = 0; b < blocks; b++, it++) {
                    const uint32_t s = it % S::stages, ph = (it / S::stages) & 1;
                    const uint32_t buf = it & 1, bph = (it >> 1) & 1;
                    if (!(ok = mbar_wait_or_abort(&t.acc_empty[buf], bph ^ 1, &t.abort) &&
                               mbar_wait_or_abort(&t.full[s], ph, &t.abort)))
                        break;
                    tc_fence_after();
                    const uint64_t da = smem_desc_sw128(sA + s * S::a_bytes);
                    const uint64_t db = smem_desc_sw128(sB + s * S::b_bytes);
#pragma unroll
                    for (int k = 0; k < kBlockK / 32; k++)
                        mma_e4m3(tmem + buf * BN, da + 2 * k, db + 2 * k, idesc, k > 0);
                    mma_commit(&t.empty[s]);
                    mma_commit(&t.acc_full[buf]);
                }
            }
            if (!ok && it > 0)  // no MMA may be in flight when TMEM is freed
                mbar_wait(&t.acc_full[(it - 1) & 1], ((it - 1) >> 1) & 1);
        }
        __syncwarp();
    } else {
        const int half = wid >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (wid & 3)) << 16) + half * S::cols;
        const int esize = kF32 ? 4 : 2;
        const bool fast = (static_cast<int64_t>(p.N) * esize) % 16 == 0;
        uint32_t it = 0;
        bool ok = true;
        for (int32_t idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x) {
            const Tile tl = tile_at<kMode, BN>(idx, p, off, first, mt, nt);
            const int32_t row = tl.row + 32 * (wid & 3) + lane;
            const bool in = row < tl.end;
            uint64_t acc[S::cols / 2];
#pragma unroll
            for (int e = 0; e < S::cols / 2; e++)
                acc[e] = 0;
            if (tl.blocks > 0) {
                // scales of the row and of the column (or weight tile), and
                // their distance from block to block
                const int32_t col = tl.n0 + (kColScale ? static_cast<int32_t>(threadIdx.x) % BN
                                                       : half * S::cols);
                const int64_t sa_step = kMode == kWgrad ? p.R : 1;
                const int64_t sb_step = kMode == kWgrad ? p.N : 1;
                const float *sa, *sb;
                if (kMode == kWgrad) {
                    sa = p.sa + static_cast<int64_t>(tl.xblk) * p.R + min(row, p.R - 1);
                    sb = p.sb + static_cast<int64_t>(tl.xblk) * p.N + min(col, p.N - 1);
                } else {
                    sa = p.sa + static_cast<int64_t>(min(row, p.M - 1)) * p.KB;
                    sb = p.sb + (static_cast<int64_t>(tl.g) * p.sb_rows +
                                 min(kColScale ? col : col / 128, p.sb_rows - 1)) * p.KB;
                }
                float a0 = __ldg(sa), b0 = __ldg(sb);
                float a1 = tl.blocks > 1 ? __ldg(sa + sa_step) : 0.0f;
                float b1 = tl.blocks > 1 ? __ldg(sb + sb_step) : 0.0f;
                sa += 2 * sa_step;
                sb += 2 * sb_step;
                for (int32_t b = 0; b < tl.blocks; b++, it++) {
                    const float scale = kColScale ? a0 : a0 * b0;
                    const float col_scale = b0;
                    a0 = a1;
                    b0 = b1;
                    if (b + 2 < tl.blocks) {
                        a1 = __ldg(sa);
                        b1 = __ldg(sb);
                        sa += sa_step;
                        sb += sb_step;
                    }
                    const uint32_t buf = it & 1, bph = (it >> 1) & 1;
                    if (kColScale) {
                        if (threadIdx.x < BN)
                            t.col_scale[buf][threadIdx.x] = col_scale;
                        // a wait that gave up in one warp is known to all of them
                        // here: they leave the tile loop together
                        ok = !named_barrier_or(1, kPromoteWarps * 32, !ok);
                    }
                    ok = ok && mbar_wait_or_abort(&t.acc_full[buf], bph, &t.abort);
                    tc_fence_after();
                    const uint64_t sc = pack2(__float_as_uint(scale), __float_as_uint(scale));
                    const uint32_t addr = lane_base + buf * BN;
                    uint32_t r[2][16];
                    tmem_ld16(addr, r[0]);
#pragma unroll
                    for (int c = 0; c < S::cols / 16; c++) {
                        tmem_wait_ld(r[c & 1]);
                        if (c + 1 < S::cols / 16)
                            tmem_ld16(addr + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            uint64_t v = pack2(r[c & 1][2 * e], r[c & 1][2 * e + 1]);
                            if (kColScale) {
                                const float2 cs = *reinterpret_cast<const float2 *>(
                                    &t.col_scale[buf][half * S::cols + 16 * c + 2 * e]);
                                v = mul2(v, pack2(__float_as_uint(cs.x), __float_as_uint(cs.y)));
                            }
                            acc[8 * c + e] = fma2(v, sc, acc[8 * c + e]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&t.acc_empty[buf]);
                }
            }
            if (kColScale)
                ok = !named_barrier_or(1, kPromoteWarps * 32, !ok);
            if (in && ok) {
                const int64_t row_off =
                    ((kMode == kWgrad ? static_cast<int64_t>(tl.g) * p.R : 0) + row) * p.N;
#pragma unroll
                for (int c = 0; c < S::cols / 16; c++) {
                    const int32_t col = tl.n0 + half * S::cols + 16 * c;
                    if (col < p.N) {
                        if (kMode == kWgrad && p.add)
                            add16<kF32>(p.c, row_off, col, p.N, acc + 8 * c);
                        store16<kF32>(p.c, row_off, col, p.N, fast, acc + 8 * c);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (wid == 9)
        tmem_free(tmem, 2 * BN);
    if (threadIdx.x == 0 && t.abort && p.dev_status)
        atomicOr(p.dev_status, 2);
}

// Both operands: [rows, K bytes] matrices cut into 128-byte blocks along K.
template <int BN, Mode kMode, bool kF32>
fq_status launch_matmul(const uint8_t *a, int64_t a_rows, const uint8_t *b, int64_t b_rows,
                        int64_t K, int64_t tiles, const MmArgs &p, cudaStream_t st)
{
    CUtensorMap ta, tb;
    if (!encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, a_rows, K, kBlockK, kTileM,
                              CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K, b_rows, K, kBlockK, BN,
                              CU_TENSOR_MAP_SWIZZLE_128B, true)) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    using S = MmShape<BN>;
    const auto kern = fp8_matmul_kernel<BN, kMode, kF32>;
    const size_t dyn = 1024 + S::stages * (S::a_bytes + S::b_bytes) + sizeof(MmTail<BN>) +
                       2 * (p.G + 2) * sizeof(int32_t);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int grid = static_cast<int>(tiles < sm_count() ? tiles : sm_count());
    if (launch_pdl(kern, dim3(grid), dim3(kMmThreads), dyn, st, ta, tb, p) != cudaSuccess)
        return launch_status();
    return launch_status();
}

// The transposed operands (rows of M tokens) re-laid for the weight gradient:
// row r of the workspace holds the row's 128-token blocks, each at a multiple
// of 128 bytes and filled up with zeros.  The rows of M tokens start at any
// byte where M % 16 != 0, and the groups at any token: neither is a tensor
// copy's alignment.  A lane makes 16 bytes from five aligned words.
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
    const int64_t quads = (rows + 3) / 4, items = quads * blocks;
    const int lane = threadIdx.x & 31, sub = lane >> 3, chunk = lane & 7;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
         w < items; w += step) {
        const int64_t quad = w / blocks, r = 4 * quad + sub;
        const int32_t blk = static_cast<int32_t>(w - quad * blocks);
        if (r >= rows)
            continue;
        const int g = group_of_tile(first, G + 1, blk);
        const int32_t t0 = off[g] + (blk - first[g]) * 128 + 16 * chunk;
        const int32_t len = min(16, off[g + 1] - t0);
        uint32_t o[4] = {0, 0, 0, 0};
        if (len > 0) {
            const bool in_a = r < a_rows;
            const uint8_t *base = in_a ? a : b;
            const int64_t size = static_cast<int64_t>(in_a ? a_rows : b_rows) * M;
            const int64_t at = (in_a ? r : r - a_rows) * M + t0;
            const int64_t w0 = at >> 2;
            const int sh = 8 * static_cast<int>(at & 3);
            uint32_t v[5];
#pragma unroll
            for (int i = 0; i < 5; i++) {
                v[i] = 0;
                if (4 * (w0 + i) + 4 <= size) {
                    v[i] = __ldg(reinterpret_cast<const uint32_t *>(base) + w0 + i);
                } else {  // the tensor's last bytes
                    for (int k = 0; k < 4; k++)
                        if (4 * (w0 + i) + k < size)
                            v[i] |= static_cast<uint32_t>(base[4 * (w0 + i) + k]) << (8 * k);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                o[i] = __funnelshift_r(v[i], v[i + 1], sh);
                const int keep = len - 4 * i;
                if (keep < 4)
                    o[i] = keep > 0 ? o[i] & ((1u << (8 * keep)) - 1) : 0;
            }
        }
        *reinterpret_cast<uint4 *>(out + r * pitch + static_cast<int64_t>(blk) * 128 + 16 * chunk) =
            make_uint4(o[0], o[1], o[2], o[3]);
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
    const int64_t tiles = ((M + kTileM - 1) / kTileM + G + 1) * ((N + 255) / 256);
    if (b_block == 1)
        return c_f32 ? launch_matmul<256, kRowScale, true>(a, M, b, G * N, K, tiles, p, st)
                     : launch_matmul<256, kRowScale, false>(a, M, b, G * N, K, tiles, p, st);
    return c_f32 ? launch_matmul<256, kTileScale, true>(a, M, b, G * N, K, tiles, p, st)
                 : launch_matmul<256, kTileScale, false>(a, M, b, G * N, K, tiles, p, st);
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
    const int64_t mt = (N + kTileM - 1) / kTileM, nt = (K + 255) / 256;
    if (need < 0 || mt > INT32_MAX / nt / G)
        return FQ_ERR_SHAPE;
    if (cap < fp4_to_fp8_cols_scale_capacity(M, G) || workspace_bytes < need)
        return FQ_ERR_ARG;
    if ((M > 0 && (!aT || !aT_scale || !bT || !bT_scale)) || !c || !workspace)
        return FQ_ERR_NULL;
    if (!aligned16(aT) || !aligned16(aT_scale) || !aligned16(bT) || !aligned16(bT_scale) ||
        !aligned16(c) || !aligned16(workspace) || !aligned16(group_offsets))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t blocks = fp4_to_fp8_cols_scale_capacity(M, G), pitch = 128 * blocks;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t dyn = 2 * (G + 2) * sizeof(int32_t);
    const int64_t warps = ((N + K + 3) / 4) * blocks;
    const int grid = persistent_grid(align_blocks_kernel, kThreads, dyn, (warps + 7) / 8);
    if (launch_pdl(align_blocks_kernel, dim3(grid), dim3(kThreads), dyn, st, aT,
                   static_cast<int32_t>(N), bT, static_cast<int32_t>(K), static_cast<int32_t>(M),
                   group_offsets, G, pitch, ws, dev_status) != cudaSuccess)
        return launch_status();
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
    const int64_t tiles = mt * nt * G;
    const uint8_t *wb = ws + N * pitch;
    return c_f32 ? launch_matmul<256, kWgrad, true>(ws, N, wb, K, pitch, tiles, p, st)
                 : launch_matmul<256, kWgrad, false>(ws, N, wb, K, pitch, tiles, p, st);
}
