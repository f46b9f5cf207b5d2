// gate.h -- the gate of a feed-forward block, h = act(g) u, and its derivatives:
// shared by the gated product, its finishing pass and the backward pass.
#ifndef FP8Q_GATE_H
#define FP8Q_GATE_H

#include "gemm_kernels.h"

namespace fp8q {

constexpr int kActSilu = 3; // beside Act; only the gated calls take it

// 1 / (1 + e^-x) with one exp2 and one reciprocal (1 ulp each).  The exponent's one
// rounding and the constant's are worth 1.22 |x| 2^-24 of e^-x, so of the result where
// x is negative (12 x 2^-24 at -10); bringing that to a few 2^-24 takes four
// operations more, an eighth of the backward pass's arithmetic, for results that 8-bit
// codes hold to 2^-4.  0 below -88, where e^-x leaves binary32, 1 at +inf.
__device__ __forceinline__ float sigmoid_f32(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// act(x) and act'(x).
//   ReLU: x < 0 -> 0, NaN kept; the derivative at 0 is 0, at NaN NaN
//   GELU: x Phi(x); Phi(x) + x phi(x) (Phi within 2^-21, phi's exponent rounded as above)
//   SiLU: x p with p = sigmoid(x); p (1 + x (1 - p))
// GELU and SiLU are NaN at -inf (-inf times 0).
template <int ACT> __device__ __forceinline__ float act_f32(float x)
{
    if constexpr (ACT == kActRelu) return x < 0.0f ? 0.0f : x;
    else if constexpr (ACT == kActGelu) return gelu_f32(x);
    else return x * sigmoid_f32(x);
}

template <int ACT> __device__ __forceinline__ void act_and_grad(float x, float &a, float &d)
{
    if constexpr (ACT == kActRelu) {
        a = x < 0.0f ? 0.0f : x;
        d = x > 0.0f ? 1.0f : x == x ? 0.0f : x;
    } else if constexpr (ACT == kActGelu) {
        const float phi = 0.398942280f * __builtin_amdgcn_exp2f(-0.721347520f * x * x);
        const float cdf = gelu_cdf_f32(x);
        a = x * cdf;
        d = fmaf(x, phi, cdf);
    } else {
        const float p = sigmoid_f32(x);
        a = x * p;
        d = fmaf(a, 1.0f - p, p);
    }
}

// f(constant of the activation) for a wave-uniform one
template <typename Fn> __device__ __forceinline__ void with_act(int act, Fn f)
{
    if (act == kActSilu) f(PhaseC<kActSilu>{});
    else if (act == kActGelu) f(PhaseC<kActGelu>{});
    else f(PhaseC<kActRelu>{});
}

// and of the FP8 format
template <typename Fn> __device__ __forceinline__ void with_fmt(int fmt, Fn f)
{
    if (fmt == kE4M3) f(PhaseC<kE4M3>{});
    else f(PhaseC<kE5M2>{});
}

// Magnitude bits of the largest of n values, NaN if one is: v_maximum3_f32 takes two
// values and their magnitudes in one instruction, where the integer maximum of
// magnitude bits takes four.
template <int n> __device__ __forceinline__ uint32_t absmax_bits(const float *v)
{
    float m = __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
    for (int e = 2; e < n; e += 2)
        m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[e])),
                                          __builtin_fabsf(v[e + 1]));
    return f32_absbits(m);
}

#define FP8Q_DPP(V, CTRL) (uint32_t) __builtin_amdgcn_update_dpp(0, (int)(V), CTRL, 0xF, 0xF, false)

// Reductions of several values over lanes, halving: lanes that differ in one bit
// split the values between them, so n values over m lanes take about 3 n operations
// instead of 3 n log m.  Of n values in m, n / 2 are left: lanes with the bit
// clear have the first half.
template <int n> __device__ __forceinline__ void halve_32(uint32_t *m) // lane ^ 32
{
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const auto p = __builtin_amdgcn_permlane32_swap(m[i], m[i + n / 2], false, false);
        m[i] = max((uint32_t)p[0], (uint32_t)p[1]);
    }
}
template <int n> __device__ __forceinline__ void halve_16(uint32_t *m) // lane ^ 16
{
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const auto p = __builtin_amdgcn_permlane16_swap(m[i], m[i + n / 2], false, false);
        m[i] = max((uint32_t)p[0], (uint32_t)p[1]);
    }
}
// `up`: the lane's bit; CTRL: a row permutation that changes it
template <int n, int CTRL> __device__ __forceinline__ void halve_dpp(uint32_t *m, bool up)
{
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const uint32_t keep = up ? m[i + n / 2] : m[i], give = up ? m[i] : m[i + n / 2];
        m[i] = max(keep, FP8Q_DPP(give, CTRL));
    }
}

// current_scales of a block's maximum (fp32 magnitude bits) with margin 0, the
// divisions in three operations each.  Both formats' maxima are 7 times a
// power of two: q + r / 7 with r = a - 7 q exact is a / 7 correctly rounded
// (1 / 7 rounded to nearest is enough for that), and one Newton step of
// v_rcp_f32 is 1 / s correctly rounded.  Both equal the IEEE quotient on the MI355X
// for every mantissa, at exponents from the floor's to the largest.  An
// infinite or NaN maximum takes the division.
__device__ __forceinline__ Scales block_scales(uint32_t most, int fmt)
{
    const float top = fmt == kE4M3 ? 0x1p-6f : 0x1p-13f; // 7 / FP8_MAX
    if (__builtin_expect(most >= kInfBits, 0))
        return current_scales(__uint_as_float(canonical_amax_bits(most)), 7.0f / top, 0);
    const float a = fmaxf(__uint_as_float(most), kAmaxFloor);
    const float q = a * (1.0f / 7.0f), s = fmaf(fmaf(-7.0f, q, a), 1.0f / 7.0f, q) * top;
    const float y = __builtin_amdgcn_rcpf(s);
    return Scales{s, fmaf(fmaf(-s, y, 1.0f), y, y)};
}

// Four codes of a block whose maximum is finite and gave the scale: no product
// is NaN or above FP8_MAX (1 + 3 2^-24), which rounds to FP8_MAX, so neither the NaN
// test nor the clamp of encode4 is needed.
template <int F> __device__ __forceinline__ uint32_t encode_fit(float x0, float x1, float x2, float x3, float scale)
{
    int r;
    if constexpr (F == kE4M3) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(x0 * scale, x1 * scale, 0, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(x2 * scale, x3 * scale, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(x0 * scale, x1 * scale, 0, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(x2 * scale, x3 * scale, r, true);
    }
    return (uint32_t)r;
}

// The code of x in a block whose maximum is infinite or NaN, so that its scale is 0
// or NaN: a NaN product's with x's sign, else a zero's.
__device__ __forceinline__ uint32_t encode_bad(float x, float scale)
{
    const float y = x * scale;
    return (y != y ? 0x7Fu : 0u) | (__float_as_uint(x) >> 24 & 0x80u);
}

// Four codes with the scale of their block, or of a block each (column codes),
// where `finite` says that all of these are finite.
template <int F>
__device__ __forceinline__ uint32_t encode_block(float x0, float x1, float x2, float x3, float scale, bool finite)
{
    if (__builtin_expect(finite || finite_nonzero(scale), 1)) return encode_fit<F>(x0, x1, x2, x3, scale);
    return encode_bad(x0, scale) | encode_bad(x1, scale) << 8 | encode_bad(x2, scale) << 16 |
           encode_bad(x3, scale) << 24;
}

// What a gated product writes of its rows.
struct GatedOut {
    void *H; // [rows][F], null: none
    int h_dtype;
    uint8_t *q_h; // codes [rows][F] and scales, null: none
    float *s_h;
    int h_fmt;
    uint8_t *q_gu; // codes [rows][2F] of g and u and scales, null: none
    float *s_gu;
    int gu_fmt;
    int act;
    float *ws; // few rows with codes: g and u as floats [rows][2F], for the finishing pass
};

struct GatedArgs {
    const uint8_t *A, *B;
    const float *sA, *sB;
    const int32_t *offsets;
    int groups, rows;
    int64_t F, K;
    GatedOut out;
    hipStream_t stream;
    int cus;
};

} // namespace fp8q

#endif // FP8Q_GATE_H
