// Activations between two products, their gradients, and what the products'
// epilogues are given.
//
//   act(x) = x s(x),   s = 1 (none), [x > 0] (relu), sigma(x) (silu),
//            sigma(2 sqrt(2/pi) (x + 0.044715 x^3)) (gelu_tanh: the tanh form
//            x / 2 (1 + tanh u) is x sigma(2 u))
//   act'(x) = s + x s (1 - s) t'(x),   t the sigmoid's argument
#pragma once

#include "fq_tc.cuh"

namespace fq {

struct EpiArgs {
    const float *bias;  // [G, N] or NULL
    const void *in;     // residual in c's type (may be c) or NULL; gradients: z, BF16
    void *side;         // BF16 z beside c; gradients: h; or NULL
    float *scales;      // of a quantized c
    int32_t act;        // FQ_ACT_*
};

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One form for both sigmoids, t = x (c0 + c1 x^2), and one for none and relu: the
// epilogues exist once for each form (kSigmoid), without branches inside (65536 x
// 2048 x 7168, gradient of silu: 1559 us with a branch a value, 846 without an
// activation).  The base-2 exponential (2 ulp) and the reciprocal (1 ulp) of the
// hardware.  The argument's rounding enters e^-|t| with the factor |t|: s is off by
// ((1 - s) (4.5 + 2.5 |t|) + 3) 2^-23 of its value at most, which is below the rounding of a
// BF16 or E4M3 result, not below that of an FP32 one (some 50 2^-23 at t = -20).
// Both instructions give 0 for what is below 2^-126.  So the exponential is taken of half
// of its argument, h = 2^(-|t| log2(e) / 2), whose square is e^-|t|, and x s is multiplied
// together from x: x s is right down to the smallest numbers (1 / (1 + e^-t) by itself
// is 0 from t = -87.3 on, where silu is -5e-37).
// Pairs of values are computed together where an instruction takes two.
struct Act {
    static constexpr float kLog2e = 1.4426950408889634f, kMost = 3.402823466e38f;
    float c0, c1;
    bool relu;

    static __device__ __forceinline__ bool sigmoid(int32_t act) { return act >= FQ_ACT_SILU; }
    __device__ __forceinline__ explicit Act(int32_t act)
        : c0(act == FQ_ACT_GELU_TANH ? 1.5957691216057308f : 1.0f),  // 2 sqrt(2 / pi)
          c1(act == FQ_ACT_GELU_TANH ? 0.044715f * 1.5957691216057308f : 0.0f),
          relu(act == FQ_ACT_RELU)
    {
    }
    // act of two values.  Beyond |x| = 200 s is 0 or 1, and the bound keeps c1 x^2 from
    // being 0 times infinity; -inf counts as the lowest finite value, whose product with
    // s = 0 is a zero.
    template <bool kSigmoid>
    __device__ __forceinline__ uint64_t value(uint64_t x) const
    {
        float v[2];
        unpack2(x, v[0], v[1]);
        if (!kSigmoid)
            return pack2f(relu && v[0] <= 0.0f ? 0.0f : v[0], relu && v[1] <= 0.0f ? 0.0f : v[1]);
        const uint64_t b = pack2f(fminf(fabsf(v[0]), 200.0f), fminf(fabsf(v[1]), 200.0f));
        const uint64_t poly = fma_x2(mul_x2(both(-0.5f * kLog2e * c1), b), b, both(-0.5f * kLog2e * c0));
        float t[2], h[2], d[2];
        unpack2(mul_x2(x, poly), t[0], t[1]);
        h[0] = ex2_approx(-fabsf(t[0]));
        h[1] = ex2_approx(-fabsf(t[1]));
        const uint64_t hh = pack2f(h[0], h[1]);
        unpack2(fma_x2(hh, hh, both(1.0f)), d[0], d[1]);
        // s = r where t >= 0, h h r below
        const uint64_t m = pack2f(t[0] <= 0.0f ? 1.0f : h[0], t[1] <= 0.0f ? 1.0f : h[1]);
        const uint64_t most = pack2f(fmaxf(v[0], -kMost), fmaxf(v[1], -kMost));
        return mul_x2(mul_x2(mul_x2(most, pack2f(rcp_approx(d[0]), rcp_approx(d[1]))), m), m);
    }
    // act (returned) and act' (slope) of two values.  With e = exp(-|t|), s is 1 / (1 + e)
    // or e / (1 + e) and s (1 - s) = e / (1 + e)^2, so that nothing cancels.
    template <bool kSigmoid>
    __device__ __forceinline__ uint64_t gradient(uint64_t x, uint64_t &slope) const
    {
        float v[2];
        unpack2(x, v[0], v[1]);
        if (!kSigmoid) {
            float d[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const bool off = relu && v[i] <= 0.0f;
                d[i] = off ? 0.0f : (v[i] != v[i] ? v[i] : 1.0f);
                v[i] = off ? 0.0f : v[i];
            }
            slope = pack2f(d[0], d[1]);
            return pack2f(v[0], v[1]);
        }
        const uint64_t b = pack2f(within(v[0], 200.0f), within(v[1], 200.0f));
        // (poly: half of -log2(e) t / x)
        const uint64_t q = mul_x2(both(-0.5f * kLog2e * c1), b), poly = fma_x2(q, b, both(-0.5f * kLog2e * c0));
        float t[2], e[2], r[2], s[2];
        unpack2(mul_x2(x, poly), t[0], t[1]);
        e[0] = ex2_approx(-fabsf(t[0]));
        e[1] = ex2_approx(-fabsf(t[1]));
        const uint64_t hh = pack2f(e[0], e[1]), ee = mul_x2(hh, hh);
        unpack2(add_x2(ee, both(1.0f)), r[0], r[1]);
        const uint64_t rr = pack2f(rcp_approx(r[0]), rcp_approx(r[1])), er = mul_x2(ee, rr);
        unpack2(rr, r[0], r[1]);
        unpack2(er, s[0], s[1]);
        s[0] = t[0] <= 0.0f ? r[0] : s[0];
        s[1] = t[1] <= 0.0f ? r[1] : s[1];
        // -log2(e) / 2 t'(x) = poly + 2 q b
        const uint64_t dt = fma_x2(add_x2(q, q), b, poly);
        const uint64_t bk = mul_x2(b, both(-2.0f / kLog2e));
        slope = fma_x2(mul_x2(er, rr), mul_x2(bk, dt), pack2f(s[0], s[1]));
        return mul_x2(pack2f(fmaxf(v[0], -kMost), fmaxf(v[1], -kMost)), pack2f(s[0], s[1]));
    }
    static __device__ __forceinline__ uint64_t both(float x) { return pack2f(x, x); }
    // x between -most and most
    static __device__ __forceinline__ float within(float x, float most)
    {
        float y;
        asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
        return y;
    }
};

// The quantization of a block with largest magnitude `most` (its bits; those of
// a NaN are above infinity's): code = E4M3(x * r), scale s.
__device__ __forceinline__ bool e4m3_factors(uint32_t most, float &r, float &s)
{
    const bool special = most >= 0x7F800000u;
    const float amax = __uint_as_float(most), nan = __uint_as_float(0x7FC00000u);
    r = special ? nan : fminf(__fdiv_rn(448.0f, amax), 3.402823466e38f);
    s = special ? nan : __fdiv_rn(amax, 448.0f);
    return special;
}

// Two FP32 -> packed E4M3 (lo in the low byte), saturating at 448.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fq
