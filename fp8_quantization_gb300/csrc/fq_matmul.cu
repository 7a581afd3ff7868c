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
    int32_t G, M, N, KB;
    int32_t sb_rows;   // rows of sb per group
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

// Persistent, one CTA per SM.  Warps 0-7 add up the scaled blocks (warp w:
// TMEM lanes 32 (w mod 4).., columns BN/2 * (w / 4)..), warp 8 issues the
// tensor copies, warp 9 the MMAs.  Two TMEM buffers of BN columns: the MMAs of
// block b + 1 run while block b is scaled and added.
template <int BN, bool kColScale, bool kF32>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                      const MmArgs p)
{
    using S = MmShape<BN>;
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
    const int32_t mt = first[p.G + 1], nt = (p.N + BN - 1) / BN, ntiles = mt * nt;

    if (wid == 8) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int32_t idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x) {
                int32_t i, j;
                tile_coords(idx, mt, nt, i, j);
                const int g = group_of_tile(first, p.G + 1, i);
                if (g == p.G)
                    continue;
                const int32_t row = off[g] + (i - first[g]) * kTileM;
                const int32_t wrow = g * p.N + j * BN;
                for (int32_t b = 0; b < p.KB; b++, it++) {
                    const uint32_t s = it % S::stages, ph = (it / S::stages) & 1;
                    if (!(ok = mbar_wait_or_abort(&t.empty[s], ph ^ 1, &t.abort)))
                        break;
                    mbar_arrive_expect_tx(&t.full[s], S::a_bytes + S::b_bytes);
                    tma_load_2d(sA + s * S::a_bytes, &ta, b * kBlockK, row, &t.full[s]);
                    tma_load_2d(sB + s * S::b_bytes, &tb, b * kBlockK, wrow, &t.full[s]);
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
                int32_t i, j;
                tile_coords(idx, mt, nt, i, j);
                if (group_of_tile(first, p.G + 1, i) == p.G)
                    continue;
                for (int32_t b = 0; b < p.KB; b++, it++) {
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
            int32_t i, j;
            tile_coords(idx, mt, nt, i, j);
            const int g = group_of_tile(first, p.G + 1, i);
            const int32_t row = off[g] + (i - first[g]) * kTileM + 32 * (wid & 3) + lane;
            const bool in = row < off[g + 1];
            const int32_t n0 = j * BN;
            uint64_t acc[S::cols / 2];
#pragma unroll
            for (int e = 0; e < S::cols / 2; e++)
                acc[e] = 0;
            if (g < p.G) {
                const float *sa = p.sa + static_cast<int64_t>(min(row, p.M - 1)) * p.KB;
                const float *sb;
                if (kColScale)
                    sb = p.sb + (static_cast<int64_t>(g) * p.sb_rows +
                                 min(n0 + static_cast<int32_t>(threadIdx.x) % BN, p.N - 1)) * p.KB;
                else
                    sb = p.sb + (static_cast<int64_t>(g) * p.sb_rows +
                                 min((n0 + half * S::cols) / 128, p.sb_rows - 1)) * p.KB;
                float a0 = __ldg(sa), b0 = __ldg(sb);
                float a1 = p.KB > 1 ? __ldg(sa + 1) : 0.0f, b1 = p.KB > 1 ? __ldg(sb + 1) : 0.0f;
                for (int32_t b = 0; b < p.KB; b++, it++) {
                    const float scale = kColScale ? a0 : a0 * b0;
                    const float col = b0;
                    a0 = a1;
                    b0 = b1;
                    if (b + 2 < p.KB) {
                        a1 = __ldg(sa + b + 2);
                        b1 = __ldg(sb + b + 2);
                    }
                    const uint32_t buf = it & 1, bph = (it >> 1) & 1;
                    if (kColScale) {
                        if (threadIdx.x < BN)
                            t.col_scale[buf][threadIdx.x] = col;
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
                const int64_t row_off = static_cast<int64_t>(row) * p.N;
#pragma unroll
                for (int c = 0; c < S::cols / 16; c++) {
                    const int32_t col = n0 + half * S::cols + 16 * c;
                    if (col < p.N)
                        store16<kF32>(p.c, row_off, col, p.N, fast, acc + 8 * c);
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

template <int BN, bool kColScale, bool kF32>
fq_status launch_matmul(const uint8_t *a, const uint8_t *b, const MmArgs &p, cudaStream_t st)
{
    CUtensorMap ta, tb;
    const uint64_t K = static_cast<uint64_t>(p.KB) * 128;
    if (!encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, p.M, K, 128, kTileM,
                              CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K,
                              static_cast<uint64_t>(p.G) * p.N, K, 128, BN,
                              CU_TENSOR_MAP_SWIZZLE_128B, true)) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    using S = MmShape<BN>;
    const auto kern = fp8_matmul_kernel<BN, kColScale, kF32>;
    const size_t dyn = 1024 + S::stages * (S::a_bytes + S::b_bytes) + sizeof(MmTail<BN>) +
                       2 * (p.G + 2) * sizeof(int32_t);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int64_t tiles = ((p.M + kTileM - 1) / kTileM + p.G + 1) *
                          static_cast<int64_t>((p.N + BN - 1) / BN);
    const int grid = static_cast<int>(tiles < sm_count() ? tiles : sm_count());
    if (launch_pdl(kern, dim3(grid), dim3(kMmThreads), dyn, st, ta, tb, p) != cudaSuccess)
        return launch_status();
    return launch_status();
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
        return c_f32 ? launch_matmul<256, true, true>(a, b, p, st)
                     : launch_matmul<256, true, false>(a, b, p, st);
    return c_f32 ? launch_matmul<256, false, true>(a, b, p, st)
                 : launch_matmul<256, false, false>(a, b, p, st);
}
