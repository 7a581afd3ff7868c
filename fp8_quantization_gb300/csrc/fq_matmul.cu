// The products as they are (fp8_matmul) and the weight gradients.
#include "fq_matmul.cuh"

namespace fq {

namespace {

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
    MmArgs p;
    const fq_status bad =
        matmul_args(a, sa, M, K, b, sb, N, b_block, 1, group_offsets, G, c, dev_status, p);
    if (bad == FQ_ERR_SHAPE)
        return bad;
    if (c_f32 != 0 && c_f32 != 1)
        return FQ_ERR_ARG;
    if (bad != FQ_OK || M == 0)
        return bad;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (b_block == 1)
        return c_f32 ? launch_forward<kRowScale, kF32, kPlain>(a, b, K, p, st)
                     : launch_forward<kRowScale, kBf16, kPlain>(a, b, K, p, st);
    return c_f32 ? launch_forward<kTileScale, kF32, kPlain>(a, b, K, p, st)
                 : launch_forward<kTileScale, kBf16, kPlain>(a, b, K, p, st);
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
    if (one_cta_tiles(N, K, G, 256, 520))
        return c_f32 ? launch_matmul<1, kWgrad, kF32, kPlain>(wa, N, wb, K, pitch, G * N, p, st)
                     : launch_matmul<1, kWgrad, kBf16, kPlain>(wa, N, wb, K, pitch, G * N, p, st);
    return c_f32 ? launch_matmul<2, kWgrad, kF32, kPlain>(wa, N, wb, K, pitch, G * N, p, st)
                 : launch_matmul<2, kWgrad, kBf16, kPlain>(wa, N, wb, K, pitch, G * N, p, st);
}
