// Routing of tokens to experts: scores, choice, weights, their gradient, and
// the order of the rows that the ragged per-expert calls take.
//
// Source: "Practical FP4 Training for Large-Scale MoE Models on Hopper GPUs",
// technical overview section 2 item 3: tokens form ragged per-expert groups
// without padding.  The pages fix no router; the forms are the usual ones:
//   score  s_e = exp(l_e) / sum_f exp(l_f)   or   1 / (1 + exp(-l_e))
//   choice c_e = s_e + bias_e (the bias balances the experts and takes no part
//          in the weights); with expert groups only the experts of the
//          `keep` groups with the largest sum of their best `top` choices
//   ids    the k largest choices, ties to the lowest index
//   weight w_j = scale * s_j, or scale * s_j / (sum of the chosen s)
// in binary32; the quotients relative to the largest chosen score, so that they
// hold where the scores themselves underflow.  A logit that is NaN or at or below
// BF16's lowest finite value masks its expert: never chosen, score 0.  A slot
// without an expert (fewer than k available) gets id -1 and weight 0.
#include <cfloat>
#include <cmath>

#include "fq_common.cuh"

namespace fq {

namespace {

constexpr float kMasked = -0x1.FEp127f;  // BF16's lowest finite value
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int32_t E, k;
    int32_t n_groups, keep, top;
    float scale;
    float *w;
    int32_t *ids;
};

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void *logits, int64_t at)
{
    return kBf16 ? bf16_lo(__ldg(static_cast<const uint16_t *>(logits) + at))
                 : __ldg(static_cast<const float *>(logits) + at);
}

__device__ __forceinline__ float sigmoid_score(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// Unsigned key in the order of the floats (never 0 for a number above -inf).
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Largest of the warp's values, none of them NaN.
__device__ __forceinline__ float warp_max(float v)
{
    return key_value(__reduce_max_sync(kFull, order_key(v)));
}

// The score of logit l (at most `top`) up to a factor of the row, so that the largest
// is 1/2 or more: exp(l - top), or the sigmoid exp(l) / (1 + exp(l)) times exp(-top)
// where top < 0.
template <bool kSigmoid>
__device__ __forceinline__ float relative_score(float l, float top)
{
    if (!kSigmoid)
        return expf(l - top);
    const float e = expf(-fabsf(l));
    return __fdiv_rn(l < 0.0f ? expf(l - fminf(top, 0.0f)) : 1.0f, 1.0f + e);
}

// Largest key of the warp and the lowest lane that has it; 0 if none.
__device__ __forceinline__ uint32_t warp_best(uint32_t key, int &lane)
{
    const uint32_t m = __reduce_max_sync(kFull, key);
    lane = __ffs(__ballot_sync(kFull, key == m)) - 1;
    return m;
}

// Lane l's logits kVals l .. of a row, -inf past its E.  Rows of whole chunks of 16
// bytes (of a lane's share where that is less) start at a multiple of them.
template <bool kBf16, int kVals>
__device__ __forceinline__ void load_logits(const void *logits, int64_t row, int32_t E, float (&l)[kVals])
{
    constexpr int size = kBf16 ? 2 : 4, chunk = kVals * size < 16 ? kVals : 16 / size;
    const int e0 = (threadIdx.x & 31) * kVals;
    if constexpr (chunk * size >= 4) {
        if (E % chunk == 0) {
            const char *at = static_cast<const char *>(logits) + (row + e0) * size;
#pragma unroll
            for (int i0 = 0; i0 < kVals; i0 += chunk) {
                const bool in = e0 + i0 < E;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (in) {
                    if constexpr (chunk * size == 16)
                        v = __ldg(reinterpret_cast<const uint4 *>(at + i0 * size));
                    else if constexpr (chunk * size == 8) {
                        const uint2 h = __ldg(reinterpret_cast<const uint2 *>(at));
                        v.x = h.x, v.y = h.y;
                    } else
                        v.x = __ldg(reinterpret_cast<const uint32_t *>(at));
                }
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < chunk; i++) {
                    const uint32_t word = w[kBf16 ? i / 2 : i];
                    const float x = !kBf16 ? __uint_as_float(word) : i & 1 ? bf16_hi(word) : bf16_lo(word);
                    l[i0 + i] = in ? x : -INFINITY;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < kVals; i++)
        l[i] = e0 + i < E ? load_logit<kBf16>(logits, row + e0 + i) : -INFINITY;
}

// One warp per token; lane l holds the kVals experts from kVals l on, so that ties
// of the warp's largest key go to the lowest lane: one maximum and one ballot a
// choice.  A lane's keys are sorted once in runs of four (stable), and the choices
// look at the runs' heads only.  Bound by the integer pipe (75 % busy; about 680
// instructions a token), not by memory: 16384 x 256 BF16 logits (8.4 MB), k = 8, in
// 14.25 us; FP32, sigmoid, bias, the best 4 of 8 groups 26.7 us, 8 tokens of it 4.9.
// With every lane's keys looked through in each round, and the experts strided over
// the lanes (a second reduction for ties): 18.1, 46 and 6.5 us.  Left to itself the
// compiler keeps the registers at 48 to 128 and spills: 1000 experts 53 us for 43.
template <int kVals, bool kBf16, bool kSigmoid, bool kNorm>
__global__ void __launch_bounds__(kThreads, kVals <= 8 ? 4 : 2) moe_route_kernel(const RouteArgs p)
{
    constexpr int kRun = kVals < 4 ? kVals : 4, kRuns = kVals / kRun;
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, e0 = lane * kVals;
    const int per_group = p.E / p.n_groups;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < p.T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t row = t * p.E;
        float l[kVals];
        load_logits<kBf16, kVals>(p.logits, row, p.E, l);
        float mx = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < kVals; i++) {
            l[i] = l[i] > kMasked ? fminf(l[i], FLT_MAX) : -INFINITY;
            mx = fmaxf(mx, l[i]);
        }
        if (!kSigmoid) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
        }
        float sum = 0.0f;
        uint32_t key[kVals];  // of the scores, which are 0 or above: 0 where masked
#pragma unroll
        for (int i = 0; i < kVals; i++) {
            const float s = kSigmoid ? sigmoid_score(l[i]) : expf(l[i] - mx);
            if (!kSigmoid)
                sum += s;
            key[i] = l[i] > -INFINITY ? __float_as_uint(s) | 0x80000000u : 0u;
        }
        if (!kSigmoid && (!kNorm || p.bias))
            sum = warp_sum(sum);
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < kVals; i++)
                if (key[i]) {
                    const float s = key_value(key[i]);
                    const float c = (kSigmoid ? s : __fdiv_rn(s, sum)) + __ldg(p.bias + e0 + i);
                    key[i] = c > -INFINITY ? order_key(c) : 0u;
                }
        }

        if (p.n_groups > 1) {
            // the lane's two best keys among its experts from `lo` to `hi`
            uint32_t m1 = 0, m2 = 0;
            const auto best_two = [&](int lo, int hi) {
                m1 = m2 = 0;
#pragma unroll
                for (int i = 0; i < kVals; i++) {
                    const uint32_t v = e0 + i >= lo && e0 + i < hi ? key[i] : 0u;
                    m2 = max(m2, min(m1, v));
                    m1 = max(m1, v);
                }
            };
            const bool whole = per_group % kVals == 0;  // a lane's experts are of one group
            if (whole)
                best_two(0, p.E);
            uint32_t score = 0;  // of group g in lane g
            for (int g = 0; g < p.n_groups; g++) {
                const int lo = g * per_group, hi = lo + per_group;
                if (!whole)
                    best_two(lo, hi);
                const bool in = !whole || (e0 >= lo && e0 < hi);
                int l1;
                const uint32_t k1 = warp_best(in ? m1 : 0u, l1);
                uint32_t sk = k1;
                if (p.top == 2) {
                    const uint32_t k2 = __reduce_max_sync(kFull, !in ? 0u : lane == l1 ? m2 : m1);
                    if (k2) {
                        const float v = key_value(k1) + key_value(k2);
                        sk = order_key(v == 0.0f ? 0.0f : v);
                    }
                }
                if (lane == g)
                    score = sk;
            }
            uint32_t kept = 0;
            for (int j = 0; j < p.keep; j++) {
                int g;
                if (!warp_best(score, g))
                    break;
                kept |= 1u << g;
                if (lane == g)
                    score = 0;
            }
            int g = e0 / per_group, end = (g + 1) * per_group;
#pragma unroll
            for (int i = 0; i < kVals; i++) {
                if (e0 + i == end) {
                    g++;
                    end += per_group;
                }
                if (e0 + i < p.E && !((kept >> g) & 1u))
                    key[i] = 0;
            }
        }

        // runs of four keys in descending order, equal ones as they stand, with the
        // places they had, a byte each
        uint32_t place[kRuns];
#pragma unroll
        for (int q = 0; q < kRuns; q++) {
            uint32_t at[kRun];
#pragma unroll
            for (int i = 0; i < kRun; i++)
                at[i] = q * kRun + i;
#pragma unroll
            for (int n = kRun - 1; n > 0; n--)
#pragma unroll
                for (int i = 0; i < n; i++) {
                    uint32_t &a = key[q * kRun + i], &b = key[q * kRun + i + 1];
                    const bool swap = b > a;
                    const uint32_t hi = max(a, b), lo = min(a, b), x = at[i];
                    a = hi;
                    b = lo;
                    at[i] = swap ? at[i + 1] : x;
                    at[i + 1] = swap ? x : at[i + 1];
                }
            place[q] = 0;
#pragma unroll
            for (int i = 0; i < kRun; i++)
                place[q] |= at[i] << (8 * i);
        }

        int id = -1;  // of slot `lane`
        for (int j = 0; j < p.k; j++) {
            uint32_t m = key[0], at = place[0];
            int run = 0;
#pragma unroll
            for (int q = 1; q < kRuns; q++) {
                const bool more = key[q * kRun] > m;
                m = more ? key[q * kRun] : m;
                at = more ? place[q] : at;
                run = more ? q : run;
            }
            int src;
            if (!warp_best(m, src))
                break;
            const int e = __shfl_sync(kFull, e0 + static_cast<int>(at & 255u), src);
            if (lane == j)
                id = e;
            if (lane != src)
                run = -1;
#pragma unroll
            for (int q = 0; q < kRuns; q++)
                if (run == q) {
#pragma unroll
                    for (int i = 0; i < kRun - 1; i++)
                        key[q * kRun + i] = key[q * kRun + i + 1];
                    key[q * kRun + kRun - 1] = 0;
                    place[q] >>= 8;
                }
        }
        float w = 0.0f, v = -INFINITY;
        if (id >= 0)
            v = fminf(load_logit<kBf16>(p.logits, row + id), FLT_MAX);
        // normalised: relative to the largest of the chosen, as in the backward pass;
        // a bias may choose far below the row's largest, where the scores underflow
        const float top = kNorm ? warp_max(v) : mx;
        if (id >= 0)
            w = kNorm ? relative_score<kSigmoid>(v, top) : kSigmoid ? sigmoid_score(v) : expf(v - top);
        if (kNorm)
            sum = warp_sum(w);
        if (kNorm || !kSigmoid)
            w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
        if (lane < p.k) {
            p.w[t * p.k + lane] = w * p.scale;
            p.ids[t * p.k + lane] = id;
        }
    }
}

struct RouteGradArgs {
    const void *logits;
    const int32_t *ids;
    const float *dw;
    int64_t T;
    int32_t E, k;
    float scale;
    void *dl;
};

__device__ __forceinline__ void store_grad(void *dl, int64_t at, float v, bool bf16)
{
    if (bf16)
        static_cast<uint16_t *>(dl)[at] = static_cast<uint16_t>([&] {
            uint32_t r;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
            return r;
        }());
    else
        static_cast<float *>(dl)[at] = v;
}

// One warp per token.  Bound by latency (ids, their logits, reductions over the warp;
// memory 22 % busy): 16384 x 256 BF16 in 4.5 us out of the L2 and 7.4 us alone, 65536 x
// 256 19.9 us; FP32 sigmoid 5.45 us; not normalised, which reads the row three times,
// 10.5 us.
// With q_j = s_j / sum of the chosen s (normalised) the
// gradient of a chosen score is ds_j = scale (dw_j - sum_i dw_i q_i) / sum;
// through the softmax that is dl_j = scale q_j (dw_j - sum_i dw_i q_i) and 0
// elsewhere, through the sigmoid that times 1 - s_j: the chosen logits are enough,
// and nothing is divided by a sum that may underflow.  Not normalised, softmax:
// dl_e = p_e (ds_e - sum_j ds_j p_j) for every expert.  An id that stands in several
// slots has the sum of their gradients.
template <bool kBf16, bool kSigmoid, bool kNorm>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(const RouteGradArgs p)
{
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < p.T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t row = t * p.E;
        int id = lane < p.k ? __ldg(p.ids + t * p.k + lane) : -1;
        float l = -INFINITY, dw = 0.0f;
        if (id >= 0 && id < p.E)
            l = load_logit<kBf16>(p.logits, row + id);
        const unsigned same = __match_any_sync(kFull, id);  // while the logit is on its way
        const bool repeated = __any_sync(kFull, id >= 0 && (same & (same - 1)) != 0);
        if (l > kMasked) {
            l = fminf(l, FLT_MAX);
            dw = __ldg(p.dw + t * p.k + lane) * p.scale;
        } else {
            id = -1;
        }
        float d = 0.0f, rest = 0.0f;  // gradient of the slot's logit; of another logit: -rest * p_e
        float mx = -FLT_MAX, inv = 0.0f;
        if (kSigmoid) {
            // 1 - s as the sigmoid of -l: the difference would cancel next to s = 1
            const float e = expf(-fabsf(l)), large = __fdiv_rn(1.0f, 1.0f + e), small = e * large;
            const float slope = l < 0.0f ? large : small;
            float q = l < 0.0f ? small : large, mean = 0.0f;  // q: the weight without `scale`
            if (kNorm) {
                const float top = fminf(warp_max(l), 0.0f);
                if (l < 0.0f)
                    q = id >= 0 ? expf(l - top) * large : 0.0f;
                const float sum = warp_sum(q);
                q = sum > 0.0f ? __fdiv_rn(q, sum) : 0.0f;
                mean = warp_sum(dw * q);
            }
            d = q * (dw - mean) * slope;
        } else {
            if (id >= 0)
                mx = l;
            if (!kNorm)
                for (int e = lane; e < p.E; e += 32) {
                    const float v = load_logit<kBf16>(p.logits, row + e);
                    if (v > kMasked)
                        mx = fmaxf(mx, fminf(v, FLT_MAX));
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
            const float ex = id >= 0 ? expf(l - mx) : 0.0f;
            float sum = ex;
            if (!kNorm) {
                sum = 0.0f;
                for (int e = lane; e < p.E; e += 32) {
                    const float v = load_logit<kBf16>(p.logits, row + e);
                    if (v > kMasked)
                        sum += expf(fminf(v, FLT_MAX) - mx);
                }
            }
            sum = warp_sum(sum);
            inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
            const float q = ex * inv;
            rest = warp_sum(dw * q);
            d = q * (dw - rest);
        }
        for (int e = lane; e < p.E; e += 32) {
            float v = 0.0f;
            if (!kSigmoid && !kNorm) {
                const float x = load_logit<kBf16>(p.logits, row + e);
                if (x > kMasked)
                    v = -rest * (expf(fminf(x, FLT_MAX) - mx) * inv);
            }
            store_grad(p.dl, row + e, v, kBf16);
        }
        if (repeated) {  // the first slot's lane takes the sum, in slot order
            constexpr bool kRow = !kSigmoid && !kNorm;  // `rest` counts once for a logit
            const float part = kRow ? dw : d;
            float total = 0.0f;
            for (int j = 0; j < p.k; j++) {
                const float v = __shfl_sync(kFull, part, j);
                if ((same >> j) & 1u)
                    total += v;
            }
            d = kRow ? expf(l - mx) * inv * (total - rest) : total;
            if (lane != __ffs(same) - 1)
                id = -1;
        }
        __syncwarp();  // the chosen logits' gradients go over the row
        if (id >= 0)
            store_grad(p.dl, row + id, d, kBf16);
    }
}

// ---------------------------------------------------------------- rows by expert

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBatch = 8;       // loads in flight of a lane
constexpr int64_t kSortAlone = 8192;  // pairs that one CTA sorts by itself
constexpr int64_t kSortMin = 4096;    // pairs of a CTA otherwise, at least

// CTAs of the sort: the counters that each of them reads (one per expert and CTA)
// stay within 64 Ki words.
inline int32_t sort_ctas(int64_t n, int32_t E)
{
    if (n <= kSortAlone)
        return 1;
    const int64_t by_pairs = (n + kSortMin - 1) / kSortMin, by_words = 65536 / E;
    const int64_t most = by_words < 256 ? by_words : 256;
    return static_cast<int32_t>(by_pairs < most ? by_pairs : most);
}

// Pairs lo .. hi - 1 of warp `w` of all warps: runs of consecutive pairs.
__device__ __forceinline__ void sort_run(int64_t n, int64_t w, int64_t warps, int64_t &lo, int64_t &hi)
{
    const int64_t per = ((n + warps - 1) / warps + 31) / 32 * 32;
    lo = min(n, per * w);
    hi = min(n, lo + per);
}

// Adds the pairs of a run to the counters of their experts.
__device__ __forceinline__ void sort_count(const int32_t *__restrict__ ids, int64_t lo, int64_t hi,
                                           int32_t E, uint32_t *count)
{
    for (int64_t i0 = lo + (threadIdx.x & 31); i0 < hi; i0 += 32 * kSortBatch) {
        int32_t e[kSortBatch];
#pragma unroll
        for (int u = 0; u < kSortBatch; u++)
            e[u] = i0 + 32 * u < hi ? __ldg(ids + i0 + 32 * u) : -1;
#pragma unroll
        for (int u = 0; u < kSortBatch; u++)
            if (e[u] >= 0 && e[u] < E)
                atomicAdd(count + e[u], 1u);
    }
}

// Pairs per expert of each CTA of the sort, counts[CTA][E].
__global__ void __launch_bounds__(kSortThreads) moe_sort_count_kernel(
    const int32_t *__restrict__ ids, int64_t n, int32_t E, uint32_t *__restrict__ counts)
{
    extern __shared__ uint32_t count[];  // [E]
    for (int i = threadIdx.x; i < E; i += kSortThreads)
        count[i] = 0;
    __syncthreads();
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();
    int64_t lo, hi;
    sort_run(n, static_cast<int64_t>(blockIdx.x) * kSortWarps + (threadIdx.x >> 5),
             static_cast<int64_t>(gridDim.x) * kSortWarps, lo, hi);
    sort_count(ids, lo, hi, E, count);
    __syncthreads();
    for (int i = threadIdx.x; i < E; i += kSortThreads)
        counts[static_cast<int64_t>(blockIdx.x) * E + i] = count[i];
}

// Stable counting sort.  Every warp owns a run of consecutive pairs: it counts its
// pairs per expert in its own counters, the counters become start rows (over the
// experts, then the CTAs, then the warps), and the warp goes over its run again in
// order, a pair's row being its expert's counter plus its rank among the lanes
// with the same expert.  counts: of every CTA (nullptr with one CTA).  Deterministic
// (the only atomics are counts).  Bound by latency: 524288 pairs, 256 experts in
// 13.6 us with the counting kernel (128 CTAs), 512 pairs in 4.4 us.  One cluster of
// 16 CTAs took 37 us: too few SMs for the instructions.
__global__ void __launch_bounds__(kSortThreads) moe_sort_rows_kernel(
    const int32_t *__restrict__ ids, int64_t n, int32_t E, const uint32_t *__restrict__ counts,
    int64_t *__restrict__ offs, int32_t *__restrict__ pair_of_row, int32_t *__restrict__ row_of_pair)
{
    extern __shared__ uint32_t count[];  // [kSortWarps][E]
    __shared__ uint32_t warp_tot[kSortWarps];
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kSortWarps * E; i += kSortThreads)
        count[i] = 0;
    __syncthreads();
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();

    uint32_t *mine = count + wid * E;
    int64_t lo, hi;
    sort_run(n, static_cast<int64_t>(blockIdx.x) * kSortWarps + wid,
             static_cast<int64_t>(gridDim.x) * kSortWarps, lo, hi);
    sort_count(ids, lo, hi, E, mine);
    __syncthreads();

    uint32_t rows = 0;  // of the experts before this round's, in the end of all
    for (int e0 = 0; e0 < E; e0 += kSortThreads) {
        const int e = e0 + tid;
        uint32_t before = 0, all = 0;  // the expert's pairs: of the CTAs before, of all
        uint32_t from[kSortWarps];     // of this CTA's warps before
        if (e < E) {
            if (counts) {
                const int ctas = gridDim.x, self = blockIdx.x;
#pragma unroll 32
                for (int c = 0; c < ctas; c++) {
                    const uint32_t v = __ldg(counts + static_cast<int64_t>(c) * E + e);
                    before += c < self ? v : 0;
                    all += v;
                }
            }
            uint32_t c[kSortWarps], run = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; w++)
                c[w] = count[w * E + e];
#pragma unroll
            for (int w = 0; w < kSortWarps; w++) {
                from[w] = run;
                run += c[w];
            }
            if (!counts)
                all = run;
        }
        uint32_t incl = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, incl, d);
            if (lane >= d)
                incl += u;
        }
        if (lane == 31)
            warp_tot[wid] = incl;
        __syncthreads();
        uint32_t start = rows + incl - all;
#pragma unroll
        for (int w = 0; w < kSortWarps; w++) {
            const uint32_t v = warp_tot[w];
            start += w < wid ? v : 0;
            rows += v;
        }
        if (e < E) {
            if (blockIdx.x == 0)
                offs[e] = start;
#pragma unroll
            for (int w = 0; w < kSortWarps; w++)
                count[w * E + e] = start + before + from[w];
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        offs[E] = rows;

    const int bits = 32 - __clz(E);  // of an expert, or of E for none
    for (int64_t i0 = lo + lane; i0 - lane < hi; i0 += 32 * kSortBatch) {
        int32_t id[kSortBatch];
#pragma unroll
        for (int u = 0; u < kSortBatch; u++)
            id[u] = i0 + 32 * u < hi ? __ldg(ids + i0 + 32 * u) : -1;
#pragma unroll
        for (int u = 0; u < kSortBatch; u++) {
            const int64_t i = i0 + 32 * u;
            const int32_t e = id[u] >= 0 && id[u] < E ? id[u] : E;
            unsigned same = kFull;  // the lanes with this lane's expert
            for (int b = 0; b < bits; b++) {
                const unsigned v = __ballot_sync(kFull, (e >> b) & 1);
                same &= (e >> b) & 1 ? v : ~v;
            }
            int32_t row = -1;
            if (e < E)
                row = static_cast<int32_t>(mine[e] + __popc(same & ((1u << lane) - 1)));
            __syncwarp();
            if (e < E && lane == __ffs(same) - 1)
                mine[e] += __popc(same);
            __syncwarp();
            if (i < hi) {
                row_of_pair[i] = row;
                if (row >= 0)
                    pair_of_row[row] = static_cast<int32_t>(i);
            }
        }
    }
    // rows of no expert
    for (int64_t r = rows + static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; r < n;
         r += static_cast<int64_t>(gridDim.x) * kSortThreads)
        pair_of_row[r] = -1;
}

template <int kVals>
void *route_kernel(bool bf16, bool sigmoid, bool norm)
{
#define FQ_PICK(B, S, N) reinterpret_cast<void *>(moe_route_kernel<kVals, B, S, N>)
    if (bf16)
        return sigmoid ? (norm ? FQ_PICK(true, true, true) : FQ_PICK(true, true, false))
                       : (norm ? FQ_PICK(true, false, true) : FQ_PICK(true, false, false));
    return sigmoid ? (norm ? FQ_PICK(false, true, true) : FQ_PICK(false, true, false))
                   : (norm ? FQ_PICK(false, false, true) : FQ_PICK(false, false, false));
#undef FQ_PICK
}

using RouteKernel = void (*)(const RouteArgs);
using RouteGradKernel = void (*)(const RouteGradArgs);

RouteGradKernel grad_kernel(bool bf16, bool sigmoid, bool norm)
{
#define FQ_PICK(B, S, N) moe_route_backward_kernel<B, S, N>
    if (bf16)
        return sigmoid ? (norm ? FQ_PICK(true, true, true) : FQ_PICK(true, true, false))
                       : (norm ? FQ_PICK(true, false, true) : FQ_PICK(true, false, false));
    return sigmoid ? (norm ? FQ_PICK(false, true, true) : FQ_PICK(false, true, false))
                   : (norm ? FQ_PICK(false, false, true) : FQ_PICK(false, false, false));
#undef FQ_PICK
}

bool flag(int v) { return v == 0 || v == 1; }

}  // namespace

}  // namespace fq

extern "C" fq_status moe_route(const void *logits, int logits_f32, int64_t T, int32_t E, int32_t k,
                               const float *bias, int sigmoid, int32_t n_groups,
                               int32_t keep_groups, int32_t group_top, int renormalize, float scale,
                               float *weights, int32_t *ids, void *stream)
{
    using namespace fq;
    if (T < 0 || T > INT64_MAX / 4096)
        return FQ_ERR_SHAPE;
    if (E < 1 || E > FQ_COLS_MAX_GROUPS || k < 1 || k > FQ_ROUTE_MAX_K || k > E ||
        !flag(logits_f32) || !flag(sigmoid) || !flag(renormalize) || n_groups < 1 ||
        n_groups > FQ_ROUTE_MAX_GROUPS || E % n_groups != 0 || keep_groups < 1 ||
        keep_groups > n_groups || group_top < 1 || group_top > 2)
        return FQ_ERR_ARG;
    if (T == 0)
        return FQ_OK;
    if (!logits || !weights || !ids)
        return FQ_ERR_NULL;
    if (!aligned16(logits) || !aligned16(bias) || !aligned16(weights) || !aligned16(ids))
        return FQ_ERR_ALIGN;
    const RouteArgs p = {logits, bias, T, E, k, n_groups, keep_groups, group_top, scale, weights,
                         ids};
    const bool bf16 = !logits_f32;
    const int vals = (E + 31) / 32;
    void *kern = vals <= 1   ? route_kernel<1>(bf16, sigmoid, renormalize)
                 : vals <= 2 ? route_kernel<2>(bf16, sigmoid, renormalize)
                 : vals <= 4 ? route_kernel<4>(bf16, sigmoid, renormalize)
                 : vals <= 8 ? route_kernel<8>(bf16, sigmoid, renormalize)
                 : vals <= 16 ? route_kernel<16>(bf16, sigmoid, renormalize)
                              : route_kernel<32>(bf16, sigmoid, renormalize);
    const RouteKernel f = reinterpret_cast<RouteKernel>(kern);
    const int grid = persistent_grid(f, kThreads, 0, (T + kWarps - 1) / kWarps, 4);
    if (launch_pdl(f, dim3(grid), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), p) !=
        cudaSuccess)
        return launch_status();
    return launch_status();
}

extern "C" fq_status moe_route_backward(const void *logits, int logits_f32, int64_t T, int32_t E,
                                        const int32_t *ids, const float *dweights, int32_t k,
                                        int sigmoid, int renormalize, float scale, void *dlogits,
                                        void *stream)
{
    using namespace fq;
    if (T < 0 || T > INT64_MAX / 4096)
        return FQ_ERR_SHAPE;
    if (E < 1 || E > FQ_COLS_MAX_GROUPS || k < 1 || k > FQ_ROUTE_MAX_K || k > E ||
        !flag(logits_f32) || !flag(sigmoid) || !flag(renormalize))
        return FQ_ERR_ARG;
    if (T == 0)
        return FQ_OK;
    if (!logits || !ids || !dweights || !dlogits)
        return FQ_ERR_NULL;
    if (!aligned16(logits) || !aligned16(ids) || !aligned16(dweights) || !aligned16(dlogits))
        return FQ_ERR_ALIGN;
    const RouteGradArgs p = {logits, ids, dweights, T, E, k, scale, dlogits};
    const RouteGradKernel f = grad_kernel(!logits_f32, sigmoid, renormalize);
    const int grid = persistent_grid(f, kThreads, 0, (T + kWarps - 1) / kWarps, 4);
    if (launch_pdl(f, dim3(grid), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), p) !=
        cudaSuccess)
        return launch_status();
    return launch_status();
}

extern "C" int64_t moe_sort_rows_workspace(int64_t n, int32_t E)
{
    using namespace fq;
    if (n < 0 || n > INT32_MAX - 512 || E < 1 || E > FQ_COLS_MAX_GROUPS)
        return -1;
    const int64_t ctas = sort_ctas(n, E);
    return ctas > 1 ? ctas * E * static_cast<int64_t>(sizeof(uint32_t)) : 0;
}

extern "C" fq_status moe_sort_rows(const int32_t *ids, int64_t n, int32_t E, int64_t *group_offsets,
                                   int32_t *pair_of_row, int32_t *row_of_pair, void *workspace,
                                   int64_t workspace_bytes, void *stream)
{
    using namespace fq;
    if (n < 0 || n > INT32_MAX - 512)
        return FQ_ERR_SHAPE;
    if (E < 1 || E > FQ_COLS_MAX_GROUPS)
        return FQ_ERR_ARG;
    const int64_t need = moe_sort_rows_workspace(n, E);
    if (workspace_bytes < need)
        return FQ_ERR_ARG;
    if (!group_offsets || (n > 0 && (!ids || !pair_of_row || !row_of_pair)) || (need > 0 && !workspace))
        return FQ_ERR_NULL;
    if (!aligned16(ids) || !aligned16(group_offsets) || !aligned16(pair_of_row) ||
        !aligned16(row_of_pair) || !aligned16(workspace))
        return FQ_ERR_ALIGN;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int32_t ctas = sort_ctas(n, E);
    uint32_t *counts = ctas > 1 ? static_cast<uint32_t *>(workspace) : nullptr;
    if (counts && launch_pdl(moe_sort_count_kernel, dim3(ctas), dim3(kSortThreads), E * sizeof(uint32_t),
                             st, ids, n, E, counts) != cudaSuccess)
        return launch_status();
    const size_t dyn = kSortWarps * static_cast<size_t>(E) * sizeof(uint32_t);
    if (dyn > 48 * 1024 &&
        cudaFuncSetAttribute(moe_sort_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    if (launch_pdl(moe_sort_rows_kernel, dim3(ctas), dim3(kSortThreads), dyn, st, ids, n, E, counts,
                   group_offsets, pair_of_row, row_of_pair) != cudaSuccess)
        return launch_status();
    return launch_status();
}
