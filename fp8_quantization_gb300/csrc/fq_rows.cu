// Sums over rows: column sums of ragged groups of rows (the gradient of a bias
// per expert), and the weighted sum of a token's expert rows with its gradients.
//
//   group_sum_rows   out[g, n] = sum over m in group g of x[m, n]
//   moe_combine      out[t] = residual[t] + sum_j w[t, j] y[row[t, j]]
//   its gradients    dy[row] = w dout[t],   dw[t, j] = <dout[t], y[row]>
//
// All are bound by HBM: every row is read once, in 16-byte pieces.
#include <type_traits>

#include "fq_tc.cuh"

namespace fq {

namespace {

// Eight columns of a row: consecutive ones in 16-byte pieces (kVec) or, where rows
// are not 16-byte aligned, `step` apart, so that a warp's are neighbours.  Held as
// they were read until they are used, which keeps more rows in flight.
template <typename T, bool kVec>
struct Eight {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int kWords = kVec && !kWide ? 4 : 8;
    uint32_t u[kWords];

    // kConst: nothing in the kernel writes the row.
    template <bool kConst = true>
    __device__ __forceinline__ void load(const T *row, int64_t col, int64_t step, int64_t cols)
    {
        if (kVec) {
#pragma unroll
            for (int i = 0; i < kWords / 4; i++) {
                const uint4 *from = reinterpret_cast<const uint4 *>(row + col) + i;
                const uint4 a = kConst ? __ldg(from) : *from;
                u[4 * i] = a.x, u[4 * i + 1] = a.y, u[4 * i + 2] = a.z, u[4 * i + 3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i++) {
                const int64_t c = col + i * step;
                u[i] = c >= cols ? 0u : static_cast<uint32_t>(kConst ? __ldg(row + c) : row[c]);
            }
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        if (kWide)
            return __uint_as_float(u[i % kWords]);
        if (kVec)
            return i & 1 ? bf16_hi(u[i / 2 % kWords]) : bf16_lo(u[i / 2 % kWords]);
        return bf16_lo(u[i % kWords]);
    }
};

// T is uint32_t (FP32) or uint16_t (BF16).
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T *row, int64_t col, int64_t step, int64_t cols,
                                       const float *v)
{
    constexpr bool kWide = sizeof(T) == 4;
    if (kVec) {
        if (kWide) {
            float4 *to = reinterpret_cast<float4 *>(row + col);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(row + col) =
                make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                           cvt_bf16x2(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t c = col + i * step;
            if (c < cols) {
                if (kWide)
                    reinterpret_cast<float *>(row)[c] = v[i];
                else
                    reinterpret_cast<uint16_t *>(row)[c] =
                        static_cast<uint16_t>(cvt_bf16x2(v[i], 0.0f));
            }
        }
    }
}

// ---------------------------------------------------------------- column sums

constexpr int kSumCols = 256;  // columns of a CTA or a warp: 8 a lane
constexpr int kSumFew = 2048;  // up to so many rows: a CTA for a group's columns
constexpr int kSumWarp = 32;   // up to so many rows: a warp
// Rows of a group, on average, below which most pieces are short: 16384 x 7168 BF16 in 256
// groups, 64 rows each, 71 us as short ones, 78 as long; 65536 rows, 158 as long ones.
constexpr int kSumShort = 64;
// Rows of a partial sum.  65536 x 4096 BF16 in 32 groups, L2 flushed: 256 rows 110 us,
// 512 108, 1024 106; 16384 x 2048 in 8: 25.2, 28.3, 35.5; 4096 x 1024: 15.0, 21.2, 30.4.
// So long pieces, but shorter ones where each of the 152 SMs would not have four (a number, not
// the current device's: the workspace's size does not depend on where it is asked for);
// 55482 x 144 FP32 in one group: 128 rows 18.6 (the join), 512 14.0.
constexpr int64_t kSumMany = 4 * 152;
constexpr int32_t sum_rows(int64_t M, int64_t N)
{
    if (M <= 16384)
        return 128;
    return M / 512 * ((N + kSumCols - 1) / kSumCols) >= kSumMany ? 512 : 256;
}

// What the threads before this one hold, added up, and (all) what all hold.
template <int kCta>
__device__ int32_t sum_before(int32_t v, int32_t &all)
{
    __shared__ int32_t total[32];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t incl = v;
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, incl, d);
        incl += lane >= d ? u : 0;
    }
    if (lane == 31)
        total[wid] = incl;
    __syncthreads();
    const int32_t t = lane < kCta / 32 ? total[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, t);
    const int32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? t : 0);
    __syncthreads();
    return before + incl - v;
}

// off[0..G + 1] and, with rows > 0, first[0..G] as load_row_groups gives them, for all of
// the CTA's threads (and whether the offsets were malformed, for the first).  By all
// threads, a few groups each, where there are many: one warp takes 10 us for 1024 groups.
template <int kCta>
__device__ bool sum_groups(const int64_t *__restrict__ offs, int32_t G, int32_t M, int32_t rows,
                           int32_t *off, int32_t *first)
{
    __shared__ int32_t most[32];
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    if (G <= 64) {
        bool bad = false;
        if (wid == 0)
            bad = load_row_groups(offs, G, M, rows > 0 ? rows : 1, off, first);
        __syncthreads();
        return bad;
    }
    const int per = (G + kCta) / kCta;  // G + 1 entries
    const int lo = min(tid * per, G + 1), hi = min(lo + per, G + 1);
    bool bad = false;
    int32_t run = 0;
    for (int i = lo; i < hi; i++) {
        const int64_t v = offs ? offs[i] : (i == 0 ? 0 : M);
        run = max(run, i == 0 || v < 0 ? 0 : static_cast<int32_t>(v < M ? v : M));
        bad |= run != v;
        off[i] = run;
    }
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, run, d);
        run = max(run, lane >= d ? u : 0);
    }
    if (lane == 31)
        most[wid] = run;
    run = __shfl_up_sync(0xffffffffu, run, 1);
    if (tid == 0)
        off[G + 1] = M;
    __syncthreads();
    const int32_t before = max(lane > 0 ? run : 0,
                               __reduce_max_sync(0xffffffffu, lane < wid ? most[lane] : 0));
    for (int i = lo; i < hi; i++) {
        bad |= off[i] < before;
        off[i] = max(off[i], before);
    }
    bad = __syncthreads_or(bad);
    if (rows == 0)
        return bad;
    int32_t sum = 0, all;
    for (int i = lo; i < hi; i++)
        sum += (off[i + 1] - off[i] + rows - 1) / rows;
    sum = sum_before<kCta>(sum, all);
    for (int i = lo; i < hi; i++) {
        first[i] = sum;
        sum += (off[i + 1] - off[i] + rows - 1) / rows;
    }
    __syncthreads();
    return bad;
}

// The sums of a lane's columns over rows lo, lo + step, .. below hi.
template <typename T, bool kVec>
__device__ __forceinline__ void sum_columns(const T *__restrict__ x, int32_t lo, int32_t hi,
                                            int32_t step, int64_t col, int64_t N, float *acc)
{
    constexpr int kAhead = kVec && sizeof(T) == 2 ? 8 : 4;  // rows in flight
#pragma unroll
    for (int i = 0; i < 8; i++)
        acc[i] = 0.0f;
    if (col >= N)
        return;
    int32_t r = lo;
    for (; r + (kAhead - 1) * step < hi; r += kAhead * step) {
        Eight<T, kVec> v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            v[u].load(x + static_cast<int64_t>(r + step * u) * N, col, 32, N);
#pragma unroll
        for (int u = 0; u < kAhead; u++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                acc[i] += v[u].at(i);
    }
    if (r < hi) {  // the rest, as many rows at once
        Eight<T, kVec> v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            if (r + step * u < hi)
                v[u].load(x + static_cast<int64_t>(r + step * u) * N, col, 32, N);
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            if (r + step * u < hi)
#pragma unroll
                for (int i = 0; i < 8; i++)
                    acc[i] += v[u].at(i);
    }
}

// Column sums of a piece of up to `rows` rows of a group (from its first row on), or of
// whole groups (rows = 0).  A group of one piece goes to out, added to what is there (add)
// or not, the others' pieces to partial [pieces, N].  Warp w adds up rows w, w + kWarps,
// ..; the warps' sums of a column are added in warp order.  Bound by HBM: 65536 x 7168
// BF16 in 162 us, 5.8 TB/s.  A CTA for every piece, since the next CTA's loads fill the gap at
// the end of this one's: a persistent grid took 121 us where this takes 108.  But where
// most pieces are short (kShort), what a CTA costs before its first row is what counts: a
// grid that fits at once, where a warp takes a piece of up to kSumWarp rows and a CTA only
// the longer ones.  4096 x 7168 BF16 in 256 groups 17 us, a CTA a piece 92; 1024 rows in
// 1024 groups 11, 1028.  Four CTAs an SM leave 64 registers, and spills of 16 bytes for BF16,
// 24 with kShort, 56 to 152 where rows are not aligned.
template <typename T, bool kVec, int kWarps, bool kShort>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 4 : 1) group_sum_part_kernel(
    const T *__restrict__ x, int32_t M, int64_t N, const int64_t *__restrict__ offs, int32_t G,
    int32_t rows, float *__restrict__ partial, float *__restrict__ out, int32_t add,
    int32_t *dev_status)
{
    extern __shared__ int32_t dyn[];
    __shared__ float sums[kWarps][kSumCols];
    int32_t *off = dyn, *first = dyn + G + 2;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    if (sum_groups<kWarps * 32>(offs, G, M, rows, off, first) && dev_status && blockIdx.x == 0 &&
        threadIdx.x == 0)
        atomicOr(dev_status, 1);
    const int64_t strips = (N + kSumCols - 1) / kSumCols;
    const int64_t items = strips * (rows > 0 ? first[G] : G);
    struct Piece {
        int32_t unit, g, lo, hi;
    };
    const auto several = [&](int g) { return rows > 0 && first[g + 1] - first[g] > 1; };
    // the columns run fastest: CTAs next to one another read the same rows
    const auto piece = [&](int64_t item) {
        Piece v;
        v.unit = static_cast<int32_t>(item / strips);
        v.g = rows > 0 ? group_of_tile(first, G, v.unit) : v.unit;
        v.lo = off[v.g];
        v.hi = off[v.g + 1];
        if (several(v.g)) {
            v.lo += (v.unit - first[v.g]) * rows;
            v.hi = min(v.lo + rows, v.hi);
        }
        return v;
    };
    const auto target = [&](const Piece &v) {
        return several(v.g) ? partial + v.unit * N : out + v.g * N;
    };
    const auto column = [&](int64_t item, const Piece &v) { return (item - v.unit * strips) * kSumCols; };
    // The pieces that a CTA takes are listed where they are few.
    int32_t n_long = 0;
    int32_t *list = first + G + 2;
    if (kShort) {
        const auto longs = [&](int g) {
            const int32_t pieces = rows > 0 ? first[g + 1] - first[g] : 1;
            return pieces > 1 ? pieces : (off[g + 1] - off[g] > kSumWarp ? 1 : 0);
        };
        const int per = (G + kWarps * 32 - 1) / (kWarps * 32);
        const int lo = min(static_cast<int>(threadIdx.x) * per, G), hi = min(lo + per, G);
        int32_t at = 0;
        for (int g = lo; g < hi; g++)
            at += longs(g);
        at = sum_before<kWarps * 32>(at, n_long);
        for (int g = lo; g < hi; g++)
            for (int32_t i = 0, n = longs(g); i < n; i++)
                list[at++] = (rows > 0 ? first[g] : g) + i;
        __syncthreads();
    }
    const int64_t cta_items = kShort ? strips * n_long : items;
    for (int64_t k = blockIdx.x; k < cta_items; k += gridDim.x) {
        const int32_t nth = static_cast<int32_t>(k / strips);
        const int64_t item = kShort ? k + (list[nth] - nth) * strips : k;
        const Piece v = piece(item);
        float acc[8];
        sum_columns<T, kVec>(x, v.lo + wid, v.hi, kWarps, column(item, v) + (kVec ? 8 * lane : lane),
                             N, acc);
#pragma unroll
        for (int i = 0; i < 8; i++)
            sums[wid][kVec ? 8 * lane + i : lane + 32 * i] = acc[i];
        __syncthreads();
        const int64_t col = column(item, v) + threadIdx.x;
        if (threadIdx.x < kSumCols && col < N) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; w++)
                sum += sums[w][threadIdx.x];
            float *to = target(v) + col;
            *to = add && !several(v.g) ? *to + sum : sum;
        }
        __syncthreads();
    }
    if (rows > 0 && !add)  // groups without a piece
        for (int32_t g = blockIdx.x; g < G; g += gridDim.x)
            if (first[g] == first[g + 1])
                for (int64_t n = threadIdx.x; n < N; n += kWarps * 32)
                    out[g * N + n] = 0.0f;
    if (!kShort)
        return;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + wid; item < items;
         item += static_cast<int64_t>(gridDim.x) * kWarps) {
        const Piece v = piece(item);
        if (v.hi - v.lo > kSumWarp || several(v.g))
            continue;
        const int64_t col = column(item, v) + (kVec ? 8 * lane : lane);
        float acc[8];
        sum_columns<T, kVec>(x, v.lo, v.hi, 1, col, N, acc);
        if (col >= N)
            continue;
        uint32_t *to = reinterpret_cast<uint32_t *>(out + v.g * N);
        if (add) {
            Eight<uint32_t, kVec> old;
            old.template load<false>(to, col, 32, N);
#pragma unroll
            for (int i = 0; i < 8; i++)
                acc[i] += old.at(i);
        }
        store8<uint32_t, kVec>(to, col, 32, N, acc);
    }
}

// The sums of groups of more pieces than one: 32 columns a CTA, eight warps that take
// every eighth, their sums in warp order.  The offsets are not written by the kernel
// before, whose start has waited for what wrote them.
__global__ void __launch_bounds__(kThreads) group_sum_join_kernel(
    const float *__restrict__ partial, int32_t M, int64_t N, const int64_t *__restrict__ offs,
    int32_t G, int32_t rows, float *__restrict__ out, int32_t add)
{
    extern __shared__ int32_t dyn[];
    __shared__ float sums[kThreads / 32][32];
    int32_t *off = dyn, *first = dyn + G + 2, *list = off;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    sum_groups<kThreads>(offs, G, M, rows, off, first);
    const int per = (G + kThreads - 1) / kThreads;
    const int lo = min(static_cast<int>(threadIdx.x) * per, G), hi = min(lo + per, G);
    int32_t at = 0, n_groups;
    for (int g = lo; g < hi; g++)
        at += first[g + 1] - first[g] > 1;
    at = sum_before<kThreads>(at, n_groups);
    for (int g = lo; g < hi; g++)  // off is not read any more
        if (first[g + 1] - first[g] > 1)
            list[at++] = g;
    __syncthreads();
    griddep_wait();  // the partial sums (PDL launch)
    griddep_launch_dependents();
    const int64_t strips = (N + 31) / 32, items = strips * n_groups;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int32_t k = static_cast<int32_t>(item / strips), g = list[k];
        const int64_t n = (item - k * strips) * 32 + lane;
        float v = 0.0f;
        if (n < N)
#pragma unroll 8
            for (int32_t u = first[g] + wid; u < first[g + 1]; u += kThreads / 32)
                v += __ldg(partial + u * N + n);
        sums[wid][lane] = v;
        __syncthreads();
        if (wid == 0 && n < N) {
#pragma unroll
            for (int w = 1; w < kThreads / 32; w++)
                v += sums[w][lane];
            out[g * N + n] = add ? out[g * N + n] + v : v;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- a token's rows

constexpr int kCombineThreads = 128;
constexpr int kRowsAhead = 8;  // rows in flight

// Tokens (or tokens' columns) that are worked on at once where one has up to kAhead rows.
template <typename Ty, bool kVec>
constexpr int at_once(int ahead)
{
    return ahead == 8 ? 1 : (ahead == 4 || sizeof(Ty) == 4 || !kVec ? 2 : 4);
}

// A thread takes eight columns of a token: consecutive ones, or `per` apart where rows
// are not 16-byte aligned; the threads of a token follow one another (per = H / 8,
// rounded up).  Bound by HBM: 8192 tokens x 8 rows x 7168 BF16 in 158 us, 6.7 TB/s.  With few
// rows a token (kAhead of 2 or 4, k no more) a thread takes several such pieces, or
// too little would be in flight: 16384 x 2 x 4096 BF16 with a residual 150 -> 111 us.
template <typename Ty, typename To, bool kVec, int kAhead>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(
    const Ty *__restrict__ y, int32_t R, int64_t H, const int32_t *__restrict__ row_of_pair,
    const float *__restrict__ weights, int32_t T, int32_t k, const To *residual, To *out,
    int32_t per)
{
    constexpr int kItems = at_once<Ty, kVec>(kAhead);
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    const int64_t items = static_cast<int64_t>(T) * per;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kCombineThreads;
    for (int64_t item0 = static_cast<int64_t>(blockIdx.x) * kCombineThreads + threadIdx.x;
         item0 < items; item0 += stride * kItems) {
        int64_t t[kItems], col[kItems];
        Eight<To, kVec> old[kItems];
#pragma unroll
        for (int i = 0; i < kItems; i++) {
            const int64_t item = item0 + i * stride;
            // (in 32 bits also for what lies behind the last item)
            t[i] = items <= INT32_MAX ? static_cast<uint32_t>(item) / static_cast<uint32_t>(per)
                                      : item / per;
            col[i] = (item - t[i] * per) * (kVec ? 8 : 1);
            if (residual && (kItems == 1 || t[i] < T))  // may be out itself
                old[i].template load<false>(residual + t[i] * H, col[i], per, H);
        }
        float acc[kItems][8] = {};
        if (kItems == 1 && residual)
#pragma unroll
            for (int c = 0; c < 8; c++)
                acc[0][c] = old[0].at(c);
        for (int32_t j0 = 0; j0 < (kAhead < 8 ? 1 : k); j0 += kAhead) {
            Eight<Ty, kVec> v[kItems][kAhead];
            float w[kItems][kAhead];
            bool there[kItems][kAhead];
#pragma unroll
            for (int i = 0; i < kItems; i++)
#pragma unroll
                for (int u = 0; u < kAhead; u++) {
                    const int64_t token = kItems == 1 ? t[i] : min(t[i], static_cast<int64_t>(T - 1));
                    const int64_t pair = token * k + min(j0 + u, k - 1);
                    const int32_t r = __ldg(row_of_pair + pair);
                    there[i][u] = (kItems == 1 || t[i] < T) && j0 + u < k && r >= 0 && r < R;
                    w[i][u] = weights ? __ldg(weights + pair) : 1.0f;
                    if (there[i][u])
                        v[i][u].load(y + static_cast<int64_t>(r) * H, col[i], per, H);
                }
#pragma unroll
            for (int i = 0; i < kItems; i++) {
                if (kItems > 1 && residual)
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        acc[i][c] = old[i].at(c);
#pragma unroll
                for (int u = 0; u < kAhead; u++)
                    if (there[i][u])
#pragma unroll
                        for (int c = 0; c < 8; c++)
                            acc[i][c] = __fmaf_rn(w[i][u], v[i][u].at(c), acc[i][c]);
                if (kItems > 1 && t[i] < T)
                    store8<To, kVec>(out + t[i] * H, col[i], per, H, acc[i]);
            }
        }
        if (kItems == 1)
            store8<To, kVec>(out + t[0] * H, col[0], per, H, acc[0]);
    }
}

constexpr int kBackThreads = 128;

// kWarps warps take a token: its dout is read once for its rows, eight at a time; a
// thread's parts of the products <dout, y> are added over the lanes and the warps in a
// fixed order.  Then rows without a pair are cleared.  One warp a token up to 1024
// columns (1810 tokens x 3 rows x 768 FP32 with the sum before it: 23.7 us by four), four
// above.  Bound by HBM: 8192 tokens x 8 rows x 7168 BF16 in 300 us, 6.7 TB/s.  With few rows
// a token (kAhead of 2 or 4, k no more) several tokens at once: 16384 x 2 x 4096 BF16 179
// -> 115 us.
template <typename Ty, typename Td, bool kVec, int kWarps, int kAhead>
__global__ void __launch_bounds__(kBackThreads, 4) moe_combine_backward_kernel(
    const Td *__restrict__ dout, const Ty *__restrict__ y, int32_t R, int64_t H,
    const int32_t *__restrict__ row_of_pair, const int32_t *__restrict__ pair_of_row,
    const float *__restrict__ weights, int32_t T, int32_t k, Ty *__restrict__ dy,
    float *__restrict__ dweights)
{
    constexpr int kTeam = 32 * kWarps, kTeams = kBackThreads / kTeam;
    constexpr int kTokens = at_once<Ty, kVec>(kAhead), kRows = kTokens * kAhead;
    static_assert(kRows <= kRowsAhead, "a sum of a team's lanes for every row");
    __shared__ float sums[kBackThreads / 32][kRowsAhead];
    __shared__ int32_t bare[kBackThreads];
    __shared__ int32_t nbare;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, own = tid % kTeam;
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTeams + tid / kTeam; t0 < T;
         t0 += stride * kTokens) {
        for (int32_t j0 = 0; j0 < (kAhead < 8 ? 1 : k); j0 += kAhead) {
            int32_t row[kRows];
            bool mine[kRows];  // whether the row's gradient is this pair's
            float w[kRows], dot[kRows];
#pragma unroll
            for (int u = 0; u < kRows; u++) {
                const int64_t t = t0 + u / kAhead * stride;
                const int32_t j = j0 + u % kAhead;
                const int32_t pair =
                    static_cast<int32_t>(min(t, static_cast<int64_t>(T - 1))) * k + min(j, k - 1);
                const int32_t r = __ldg(row_of_pair + pair);
                row[u] = t < T && j < k && r >= 0 && r < R ? r : -1;
                mine[u] = dy && row[u] >= 0 && __ldg(pair_of_row + r) == pair;
                w[u] = weights ? __ldg(weights + pair) : 1.0f;
                dot[u] = 0.0f;
            }
            for (int64_t col = kVec ? 8 * own : own; col < H; col += 8 * kTeam) {
                Eight<Td, kVec> d[kTokens];
#pragma unroll
                for (int i = 0; i < kTokens; i++)
                    if (i == 0 || t0 + i * stride < T)
                        d[i].load(dout + (t0 + i * stride) * H, col, kTeam, H);
                if (dweights) {
                    Eight<Ty, kVec> v[kRows];
#pragma unroll
                    for (int u = 0; u < kRows; u++)
                        if (row[u] >= 0)
                            v[u].load(y + static_cast<int64_t>(row[u]) * H, col, kTeam, H);
#pragma unroll
                    for (int u = 0; u < kRows; u++)
                        if (row[u] >= 0)
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                dot[u] = __fmaf_rn(d[u / kAhead].at(i), v[u].at(i), dot[u]);
                }
#pragma unroll
                for (int u = 0; u < kRows; u++)
                    if (mine[u]) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            o[i] = w[u] * d[u / kAhead].at(i);
                        store8<Ty, kVec>(dy + static_cast<int64_t>(row[u]) * H, col, kTeam, H, o);
                    }
            }
            if (dweights) {
#pragma unroll
                for (int u = 0; u < kRows; u++) {
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1)
                        dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], s);
                    if (lane == 0)
                        sums[wid][u] = dot[u];
                }
                if (kWarps > 1)
                    __syncthreads();
                else
                    __syncwarp();
                const int64_t t = t0 + own / kAhead * stride;
                const int32_t j = j0 + own % kAhead;
                if (own < kRows && j < k && t < T) {
                    const int first = wid / kWarps * kWarps;
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < kWarps; i++)
                        v += sums[first + i][own];
                    dweights[t * k + j] = v;
                }
                if (kWarps > 1)
                    __syncthreads();
                else
                    __syncwarp();
            }
        }
    }
    __syncthreads();
    if (!dy)
        return;
    const int64_t n = static_cast<int64_t>(T) * k;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kBackThreads; r0 < R;
         r0 += static_cast<int64_t>(gridDim.x) * kBackThreads) {
        if (tid == 0)
            nbare = 0;
        __syncthreads();
        if (r0 + tid < R) {
            const int32_t pair = __ldg(pair_of_row + r0 + tid);
            if (pair < 0 || pair >= n || __ldg(row_of_pair + pair) != r0 + tid)
                bare[atomicAdd(&nbare, 1)] = tid;
        }
        __syncthreads();
        const float zero[8] = {};
        for (int32_t i = 0; i < nbare; i++)
            for (int64_t col = kVec ? 8 * tid : tid; col < H; col += 8 * kBackThreads)
                store8<Ty, kVec>(dy + (r0 + bare[i]) * H, col, kBackThreads, H, zero);
        __syncthreads();
    }
}

// f with the rows of a token that a kernel takes at once; several tokens at once only
// where there are many (4096 tokens x 2 x 4096 BF16, gradients: 46 us one at once, 29 four)
// and not for three or four FP32 rows (16384 x 4 x 2048, dy alone: 117 us one, 142 two).
template <typename Ty, typename F>
fq_status with_ahead(int32_t k, bool many, const F &f)
{
    using std::integral_constant;
    if (many && k <= 2)
        return f(integral_constant<int, 2>{});
    if constexpr (sizeof(Ty) == 2)
        if (many && k <= 4)
            return f(integral_constant<int, 4>{});
    return f(integral_constant<int, 8>{});
}

template <typename Ty, typename To>
fq_status launch_combine(const void *y, int64_t R, int64_t H, const int32_t *row_of_pair,
                         const float *weights, int64_t T, int32_t k, const void *residual,
                         void *out, cudaStream_t st)
{
    const int64_t per = (H + 7) / 8, ctas = (T * per + kCombineThreads - 1) / kCombineThreads;
    return with_ahead<Ty>(k, ctas >= 16 * sm_count(), [&](auto ahead) {
        constexpr int kAhead = decltype(ahead)::value;
        const int items = H % 8 == 0 ? at_once<Ty, true>(kAhead) : at_once<Ty, false>(kAhead);
        const auto kern = H % 8 == 0 ? moe_combine_kernel<Ty, To, true, kAhead>
                                     : moe_combine_kernel<Ty, To, false, kAhead>;
        const int grid = persistent_grid(kern, kCombineThreads, 0, (ctas + items - 1) / items, 4);
        if (launch_pdl(kern, dim3(grid), dim3(kCombineThreads), 0, st, static_cast<const Ty *>(y),
                       static_cast<int32_t>(R), H, row_of_pair, weights, static_cast<int32_t>(T), k,
                       static_cast<const To *>(residual), static_cast<To *>(out),
                       static_cast<int32_t>(per)) != cudaSuccess)
            return launch_status();
        return launch_status();
    });
}

template <typename Ty, typename Td>
fq_status launch_combine_backward(const void *dout, const void *y, int64_t R, int64_t H,
                                  const int32_t *row_of_pair, const int32_t *pair_of_row,
                                  const float *weights, int64_t T, int32_t k, void *dy,
                                  float *dweights, cudaStream_t st)
{
    static_assert(kBackThreads == 128, "four warps");
    const bool one = H <= 1024;
    const int64_t rows = (R + kBackThreads - 1) / kBackThreads, teams = one ? (T + 3) / 4 : T;
    return with_ahead<Ty>(k, teams >= 16 * sm_count(), [&](auto ahead) {
        constexpr int kAhead = decltype(ahead)::value;
        const int tokens = H % 8 == 0 ? at_once<Ty, true>(kAhead) : at_once<Ty, false>(kAhead);
        const auto kern = H % 8 == 0 ? (one ? moe_combine_backward_kernel<Ty, Td, true, 1, kAhead>
                                            : moe_combine_backward_kernel<Ty, Td, true, 4, kAhead>)
                                     : (one ? moe_combine_backward_kernel<Ty, Td, false, 1, kAhead>
                                            : moe_combine_backward_kernel<Ty, Td, false, 4, kAhead>);
        const int64_t ctas = (teams + tokens - 1) / tokens;
        const int grid = persistent_grid(kern, kBackThreads, 0, ctas > rows ? ctas : rows, 4);
        if (launch_pdl(kern, dim3(grid), dim3(kBackThreads), 0, st, static_cast<const Td *>(dout),
                       static_cast<const Ty *>(y), static_cast<int32_t>(R), H, row_of_pair,
                       pair_of_row, weights, static_cast<int32_t>(T), k, static_cast<Ty *>(dy),
                       dweights) != cudaSuccess)
            return launch_status();
        return launch_status();
    });
}

bool combine_shape(int64_t R, int64_t H, int64_t T, int32_t k)
{
    return R >= 0 && R <= INT32_MAX - 512 && H > 0 && H <= INT32_MAX - 4096 && T >= 0 &&
           T <= (INT32_MAX - 512) / (k > 0 ? k : 1);
}

}  // namespace

}  // namespace fq

extern "C" int64_t group_sum_rows_workspace(int64_t M, int64_t N, int32_t G)
{
    using namespace fq;
    if (M < 0 || M > INT32_MAX - 512 || N <= 0 || G < 1 || G > FQ_COLS_MAX_GROUPS)
        return -1;
    const int64_t units = M / sum_rows(M, N) + G, strips = (N + kSumCols - 1) / kSumCols;
    if (N > INT64_MAX / 8 / units || strips > INT64_MAX / 2 / units)
        return -1;
    return M <= kSumFew ? 0 : 4 * units * N;
}

extern "C" fq_status group_sum_rows(const void *x, int x_f32, int64_t M, int64_t N,
                                    const int64_t *group_offsets, int32_t G, float *out,
                                    int accumulate, void *workspace, int64_t workspace_bytes,
                                    int32_t *dev_status, void *stream)
{
    using namespace fq;
    if (G < 1 || G > FQ_COLS_MAX_GROUPS || (x_f32 != 0 && x_f32 != 1) ||
        (accumulate != 0 && accumulate != 1) || (!group_offsets && G != 1))
        return FQ_ERR_ARG;
    const int64_t need = group_sum_rows_workspace(M, N, G);
    if (need < 0)
        return FQ_ERR_SHAPE;
    if (workspace_bytes < need)
        return FQ_ERR_ARG;
    if ((M > 0 && !x) || !out || (need > 0 && !workspace))
        return FQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(group_offsets) || !aligned16(out) || !aligned16(workspace))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t dyn = 2 * (G + 2) * sizeof(int32_t);
    float *partial = static_cast<float *>(workspace);
    const int32_t m = static_cast<int32_t>(M);
    const int64_t strips = (N + kSumCols - 1) / kSumCols;
    const bool few = M <= kSumFew;
    const int32_t rows = few ? 0 : sum_rows(M, N);
    const int64_t items = strips * (few ? G : M / rows + G);
    // whether most pieces are short
    const bool shorts = G > 32 && M < kSumShort * static_cast<int64_t>(G);
    const auto sums = [&](auto type, auto warps, auto is_short) {
        using T = decltype(type);
        constexpr int kWarps = decltype(warps)::value;
        constexpr bool kShort = decltype(is_short)::value;
        const auto kern = N % 8 == 0 ? group_sum_part_kernel<T, true, kWarps, kShort>
                                     : group_sum_part_kernel<T, false, kWarps, kShort>;
        // the list of long pieces: fewer than M / kSumWarp
        const size_t dyn_part = dyn + (kShort ? kSumShort / kSumWarp * G * sizeof(int32_t) : 0);
        const int64_t grid = kShort ? persistent_grid(kern, kWarps * 32, dyn_part, items)
                                    : (items < INT32_MAX ? items : INT32_MAX);
        return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), dyn_part, st,
                          static_cast<const T *>(x), m, N, group_offsets, G, rows, partial, out,
                          accumulate, dev_status);
    };
    const auto launch = [&](auto type) {
        using std::integral_constant;
        if (shorts)
            return sums(type, integral_constant<int, 8>{}, std::true_type{});
        return few ? sums(type, integral_constant<int, 32>{}, std::false_type{})
                   : sums(type, integral_constant<int, 8>{}, std::false_type{});
    };
    if ((x_f32 ? launch(uint32_t{}) : launch(uint16_t{})) != cudaSuccess)
        return launch_status();
    if (few)
        return launch_status();
    const int join = persistent_grid(group_sum_join_kernel, kThreads, dyn,
                                     (N + 31) / 32 * G);
    if (launch_pdl(group_sum_join_kernel, dim3(join), dim3(kThreads), dyn, st, partial, m, N,
                   group_offsets, G, rows, out, accumulate) != cudaSuccess)
        return launch_status();
    return launch_status();
}

extern "C" fq_status moe_combine(const void *y, int y_f32, int64_t R, int64_t H,
                                 const int32_t *row_of_pair, const float *weights, int64_t T,
                                 int32_t k, const void *residual, void *out, int out_f32,
                                 void *stream)
{
    using namespace fq;
    if (!combine_shape(R, H, T, k))
        return FQ_ERR_SHAPE;
    if (k < 1 || k > FQ_ROUTE_MAX_K || (y_f32 != 0 && y_f32 != 1) || (out_f32 != 0 && out_f32 != 1))
        return FQ_ERR_ARG;
    if (T == 0)
        return FQ_OK;
    if ((R > 0 && !y) || !row_of_pair || !out)
        return FQ_ERR_NULL;
    if (!aligned16(y) || !aligned16(row_of_pair) || !aligned16(weights) || !aligned16(residual) ||
        !aligned16(out))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (y_f32)
        return out_f32 ? launch_combine<uint32_t, uint32_t>(y, R, H, row_of_pair, weights, T, k, residual, out, st)
                       : launch_combine<uint32_t, uint16_t>(y, R, H, row_of_pair, weights, T, k, residual, out, st);
    return out_f32 ? launch_combine<uint16_t, uint32_t>(y, R, H, row_of_pair, weights, T, k, residual, out, st)
                   : launch_combine<uint16_t, uint16_t>(y, R, H, row_of_pair, weights, T, k, residual, out, st);
}

extern "C" fq_status moe_combine_backward(const void *dout, int dout_f32, const void *y, int y_f32,
                                          int64_t R, int64_t H, const int32_t *row_of_pair,
                                          const int32_t *pair_of_row, const float *weights,
                                          int64_t T, int32_t k, void *dy, float *dweights,
                                          void *stream)
{
    using namespace fq;
    if (!combine_shape(R, H, T, k))
        return FQ_ERR_SHAPE;
    if (k < 1 || k > FQ_ROUTE_MAX_K || (y_f32 != 0 && y_f32 != 1) ||
        (dout_f32 != 0 && dout_f32 != 1) || (dweights && !weights))
        return FQ_ERR_ARG;
    const bool rows = dy && R > 0, scores = dweights && T > 0;
    if (!rows && !scores)
        return FQ_OK;
    if ((T > 0 && (!dout || !row_of_pair)) || (rows && !pair_of_row) || (scores && R > 0 && !y))
        return FQ_ERR_NULL;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(row_of_pair) || !aligned16(pair_of_row) ||
        !aligned16(weights) || !aligned16(dy) || !aligned16(dweights))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!rows)
        dy = nullptr;
    if (y_f32)
        return dout_f32 ? launch_combine_backward<uint32_t, uint32_t>(dout, y, R, H, row_of_pair, pair_of_row, weights, T, k, dy, dweights, st)
                        : launch_combine_backward<uint32_t, uint16_t>(dout, y, R, H, row_of_pair, pair_of_row, weights, T, k, dy, dweights, st);
    return dout_f32 ? launch_combine_backward<uint16_t, uint32_t>(dout, y, R, H, row_of_pair, pair_of_row, weights, T, k, dy, dweights, st)
                    : launch_combine_backward<uint16_t, uint16_t>(dout, y, R, H, row_of_pair, pair_of_row, weights, T, k, dy, dweights, st);
}
