// BF16 -> transposed FP8 E4M3 on ragged token groups: the weight gradient's
// operand, quantized along the tokens.
//
// Source: "Practical FP4 Training for Large-Scale MoE Models on Hopper GPUs",
// technical overview section 2: gradients stay in standard FP8 (item 2); the
// transposed operand's 128-token blocks follow the ragged per-expert groups
// without padding (item 3).  Quantizer, per block of at most 128 tokens of one
// group and one feature (binary32, one rounding per operation):
//   r = min(448 / amax, FLT_MAX), s = amax / 448, code = E4M3(x * r);
//   a block holding NaN or Inf gets s = NaN and codes 0x7F.
//
// 2 bytes read and 1 written per element, 4 bytes written per block and feature:
// 65536 x 2048 in 32 ragged groups in 73 us, 5.6 TB/s.  HBM and the instructions
// share the bound.  8 CTAs of 128 threads per SM, a tile of 64 features, the next
// tile's values fetched while the last is written out; 4 CTAs of 256 threads and 128
// features 5 % more, without the early fetch 10 %.  Blocks of fewer than 128 tokens in
// 16-byte pieces too: 256 groups of about 64 tokens, 16384 x 7168: 143 us, byte by
// byte 165.  Written as 4-byte words, a warp a row, 65536 x 2048 took 172 us; with the
// divisions in every thread 94.
#include <cfloat>

#include "fq_tc.cuh"

namespace fq {

namespace {

constexpr int kTok = 128;   // tokens of a block
constexpr int kFeat = 64;   // features of a tile
constexpr int kColThreads = 128;

// Byte of (feature, token) of a tile in shared memory: rows of 128 tokens and 8
// bytes, 80 bytes further after every 8 features.  A half-warp storing twice 8 tokens
// of 8 features 8 apart then touches 16 different 8-byte bank pairs, and a warp reading
// words 16 bytes apart of four rows meets every bank twice (rows of 128 bytes: four
// times, 78 us).
__device__ __forceinline__ int tile_byte(int f, int t) { return f * (kTok + 8) + (f >> 3) * 80 + t; }
constexpr int kTileBytes = kFeat * (kTok + 8) + (kFeat / 8) * 80 + 16;

__device__ __forceinline__ uint32_t cvt_e4m3_pair(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// One CTA tile = one 128-token block x 64 features.  Thread (q, c), q = 0..15
// and c = 0..7, holds tokens 8q..8q+7 of features 8c..8c+7: 16-byte loads of
// 128-byte row segments, the block maxima over the q by shuffle and shared
// memory, and 8 codes of one feature as one 8-byte shared store (the
// conversion takes two tokens of a feature at a time, so nothing is
// transposed in registers).  Rows of the transposed tile start at any byte of
// yT: they are written as aligned 16-byte pieces, the bytes at both ends alone.
__global__ void __launch_bounds__(kColThreads, 8) fp8_quantize_cols_kernel(
    const uint16_t *__restrict__ x, int32_t M, int32_t K, const int64_t *__restrict__ offs,
    int32_t G, uint8_t *__restrict__ yT, float *__restrict__ scale, int64_t cap, int32_t *dev_status)
{
    extern __shared__ int32_t dyn[];
    __shared__ __align__(16) uint16_t red[kColThreads / 32][kFeat];
    __shared__ __align__(16) float factor[kFeat];
    __shared__ __align__(16) uint8_t tile[kTileBytes];
    int32_t *off = dyn, *first = dyn + G + 2;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    const int q = tid >> 3, c = tid & 7;

    griddep_wait();  // the previous kernel's outputs (PDL launch)
    if (wid == 0) {
        const bool bad = load_row_groups(offs, G, M, kTok, off, first);
        if (bad && dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(dev_status, 1);
    }
    __syncthreads();
    const int32_t blocks = first[G + 1], used = first[G];
    const int32_t slabs = (K + kFeat - 1) / kFeat;
    // scale rows past the last block are 0
    for (int64_t i = static_cast<int64_t>(used) * K + blockIdx.x * kColThreads + tid; i < cap * K;
         i += static_cast<int64_t>(gridDim.x) * kColThreads)
        scale[i] = 0.0f;

    const int64_t tiles = static_cast<int64_t>(blocks) * slabs;
    if (blockIdx.x >= tiles)
        return;
    // the tile that is worked on; its values are fetched while the one before is
    // written out
    int32_t slab = blockIdx.x / blocks, blk = blockIdx.x - slab * blocks;
    const int32_t slab_step = gridDim.x / blocks, blk_step = gridDim.x - slab_step * blocks;
    int32_t g, t0, len, f0 = 0;
    uint4 v[8];
    const auto fetch = [&]() {
        g = group_of_tile(first, G + 1, blk);
        t0 = off[g] + (blk - first[g]) * kTok;
        len = min(kTok, off[g + 1] - t0);
        f0 = slab * kFeat;
        const int32_t f = f0 + 8 * c;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int t = 8 * q + j;
            v[j] = g < G && t < len && f < K
                       ? ld_nc_v4(x + static_cast<int64_t>(t0 + t) * K + f)
                       : make_uint4(0, 0, 0, 0);
        }
    };
    fetch();
    while (true) {
        uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; j++) {
            m[0] = absmax_bf16x2(m[0], v[j].x);
            m[1] = absmax_bf16x2(m[1], v[j].y);
            m[2] = absmax_bf16x2(m[2], v[j].z);
            m[3] = absmax_bf16x2(m[3], v[j].w);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            m[i] = max_u16x2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
            m[i] = max_u16x2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
        }
        if (lane < 8)
            *reinterpret_cast<uint4 *>(&red[wid][8 * c]) = make_uint4(m[0], m[1], m[2], m[3]);
        __syncthreads();  // also: the previous tile's rows are written out
        if (tid < kFeat) {  // one thread a feature: the divisions are made once
            uint32_t bits = 0;
#pragma unroll
            for (int w = 0; w < kColThreads / 32; w++)
                bits = max(bits, static_cast<uint32_t>(red[w][tid]));
            const float amax = __uint_as_float(bits << 16), nan = __uint_as_float(0x7FC00000u);
            const bool special = bits >= 0x7F80u;
            // a NaN factor gives every code 0x7F
            factor[tid] = special ? nan : fminf(__fdiv_rn(448.0f, amax), FLT_MAX);
            if (g < G && f0 + tid < K)
                scale[static_cast<int64_t>(blk) * K + f0 + tid] =
                    special ? nan : __fdiv_rn(amax, 448.0f);
        }
        __syncthreads();
        const uint32_t *vw = reinterpret_cast<const uint32_t *>(v);
        float r8[8];
        *reinterpret_cast<float4 *>(r8) = *reinterpret_cast<const float4 *>(factor + 8 * c);
        *reinterpret_cast<float4 *>(r8 + 4) = *reinterpret_cast<const float4 *>(factor + 8 * c + 4);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t u = vw[4 * (4 * h + j) + (e >> 1)];
                    p[j] = (e & 1) ? bf16_hi(u) : bf16_lo(u);
                }
                fmul2(p[0], p[1], r8[e], p[0], p[1]);
                fmul2(p[2], p[3], r8[e], p[2], p[3]);
                w[h] = cvt_e4m3_pair(p[0], p[1]) | (cvt_e4m3_pair(p[2], p[3]) << 16);
            }
            *reinterpret_cast<uint2 *>(tile + tile_byte(8 * c + e, 8 * q)) = make_uint2(w[0], w[1]);
        }
        const int32_t out_t0 = t0, out_len = len, out_f0 = f0;
        blk += blk_step;
        slab += slab_step;
        if (blk >= blocks) {
            blk -= blocks;
            slab++;
        }
        const bool more = slab < slabs;
        if (more)
            fetch();
        __syncthreads();
        // row f0 + r of yT: bytes t0 .. t0 + len - 1.  A full block: eight lanes a
        // row, lane c the 16-byte piece of yT that holds token 16 c, and two of the
        // 16 bytes at the ends that are no whole piece.
        if (out_len == kTok) {
            const int sub = lane >> 3, c8 = lane & 7;
            uint8_t *dst = yT + static_cast<int64_t>(out_f0 + 4 * wid + sub) * M + out_t0;
            const int64_t step = static_cast<int64_t>(M) * (kColThreads / 8);
#pragma unroll
            for (int i = 0; i < kFeat * 8 / kColThreads; i++, dst += step) {
                const int r = 4 * wid + sub + i * (kColThreads / 8);
                if (out_f0 + r >= K)
                    break;
                const uint8_t *src = tile + tile_byte(r, 0);
                const int lead = (16 - static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15u)) & 15;
                if (lead == 0) {
                    const uint2 *s8 = reinterpret_cast<const uint2 *>(src + 16 * c8);
                    *reinterpret_cast<uint4 *>(dst + 16 * c8) =
                        make_uint4(s8[0].x, s8[0].y, s8[1].x, s8[1].y);
                    continue;
                }
                if (c8 < 7) {
                    const int at = lead + 16 * c8, sh = 8 * (at & 3);
                    const uint32_t *s4 = reinterpret_cast<const uint32_t *>(src + (at & ~3));
                    const uint32_t v0 = s4[0], v1 = s4[1], v2 = s4[2], v3 = s4[3], v4 = s4[4];
                    *reinterpret_cast<uint4 *>(dst + at) =
                        make_uint4(__funnelshift_r(v0, v1, sh), __funnelshift_r(v1, v2, sh),
                                   __funnelshift_r(v2, v3, sh), __funnelshift_r(v3, v4, sh));
                }
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int e = c8 + 8 * h, at = e < lead ? e : kTok - 16 + e;
                    dst[at] = src[at];
                }
            }
        } else {  // the same for fewer tokens: up to 15 bytes at each end
            const int sub = lane >> 3, c8 = lane & 7;
            for (int r = 4 * wid + sub; r < kFeat && out_f0 + r < K; r += kColThreads / 8) {
                uint8_t *dst = yT + static_cast<int64_t>(out_f0 + r) * M + out_t0;
                const uint8_t *src = tile + tile_byte(r, 0);
                const int lead =
                    min(out_len, (16 - static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15u)) & 15);
                const int whole = (out_len - lead) >> 4;
                if (c8 < whole) {
                    const int at = lead + 16 * c8, sh = 8 * (at & 3);
                    const uint32_t *s4 = reinterpret_cast<const uint32_t *>(src + (at & ~3));
                    const uint32_t v0 = s4[0], v1 = s4[1], v2 = s4[2], v3 = s4[3], v4 = s4[4];
                    *reinterpret_cast<uint4 *>(dst + at) =
                        make_uint4(__funnelshift_r(v0, v1, sh), __funnelshift_r(v1, v2, sh),
                                   __funnelshift_r(v2, v3, sh), __funnelshift_r(v3, v4, sh));
                }
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int e = c8 + 8 * h, at = e < lead ? e : 16 * whole + e;
                    if (at < out_len)
                        dst[at] = src[at];
                }
            }
        }
        if (!more)
            break;
    }
}

}  // namespace

}  // namespace fq

extern "C" fq_status fp8_quantize_cols(const void *x, int64_t M, int64_t K,
                                       const int64_t *group_offsets, int32_t G, uint8_t *yT,
                                       float *yT_scale, int64_t cap, int32_t *dev_status,
                                       void *stream)
{
    using namespace fq;
    if (M < 0 || M > INT32_MAX - 512 || K <= 0 || K % 8 != 0 || K > INT32_MAX - 512)
        return FQ_ERR_SHAPE;
    if (G < 1 || G > FQ_COLS_MAX_GROUPS || (!group_offsets && G != 1))
        return FQ_ERR_ARG;
    if (cap < fp4_to_fp8_cols_scale_capacity(M, G))
        return FQ_ERR_ARG;
    if (cap > INT64_MAX / 4 / K)
        return FQ_ERR_SHAPE;
    if ((M > 0 && (!x || !yT)) || !yT_scale)
        return FQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(group_offsets) || !aligned16(yT) || !aligned16(yT_scale))
        return FQ_ERR_ALIGN;
    const size_t dyn = 2 * (G + 2) * sizeof(int32_t);
    const int64_t tiles = fp4_to_fp8_cols_scale_capacity(M, G) * ((K + kFeat - 1) / kFeat);
    const int grid = persistent_grid(fp8_quantize_cols_kernel, kColThreads, dyn, tiles);
    if (launch_pdl(fp8_quantize_cols_kernel, dim3(grid), dim3(kColThreads), dyn,
                   static_cast<cudaStream_t>(stream), static_cast<const uint16_t *>(x),
                   static_cast<int32_t>(M), static_cast<int32_t>(K), group_offsets, G, yT, yT_scale,
                   cap, dev_status) != cudaSuccess)
        return launch_status();
    return launch_status();
}
