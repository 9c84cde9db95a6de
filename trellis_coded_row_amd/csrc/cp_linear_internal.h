// Internal interface of the readout's product, its gradients and dropout
// (include/cp_linear.h): launch parameters, the mask, the activations and the
// product's epilogue.
#pragma once

#include "cp_ops_internal.h"

namespace cpk {

// Activations as in cp_act (include/cp_linear.h).
enum Act { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };

// Dropout of a matrix: threshold 0 keeps everything (rng is not read).
struct Drop {
    uint32_t threshold;
    float scale;
    const uint64_t *rng;
};

// What a product's sums become. The residual and both outputs are of the
// output's type, the bias of the operands'.
struct Epilogue {
    const void *bias, *residual;
    uint64_t residual_stride;
    void *y, *z;  // z: contiguous
    uint64_t y_stride;
    int act;
    Drop drop;
};

// out[m][n] = the sum over K of A times B: where an operand is "across", its
// rows run along K (K x m, K x n), else they are m or n rows of K.
struct LinearArgs {
    const void *a, *b;
    uint64_t a_stride, b_stride;
    int dtype;
    uint64_t m, n, k;
    Epilogue e;
    uint8_t *workspace;
    hipStream_t stream;
};
// (cp_linear's; and of the other two, with their outputs' m and n and their sums' k)
uint64_t linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype);
uint64_t linear_tile_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype);
hipError_t linear_rows_by_rows(const LinearArgs &a);      // A, B: rows of K (cp_linear)
hipError_t linear_rows_by_columns(const LinearArgs &a);   // B across (cp_linear_dx)
hipError_t linear_columns_by_columns(const LinearArgs &a);  // both across, 32-bit output (cp_linear_dw)

struct ActGradArgs {
    const void *dy, *z;
    uint64_t dy_stride, z_stride;
    int dtype;
    uint64_t m, n;
    int act;
    Drop drop;
    void *dz;
    float *db;
    uint8_t *workspace;
    hipStream_t stream;
};
uint64_t act_grad_workspace_bytes(uint64_t m, uint64_t n);
hipError_t act_grad(const ActGradArgs &a);

struct DropoutArgs {
    const void *x, *residual;
    uint64_t x_stride, residual_stride;
    int dtype;
    uint64_t n, d;
    Drop drop;
    void *y;
    hipStream_t stream;
};
hipError_t dropout(const DropoutArgs &a);

// ---------------------------------------------------------------- device

// The generator's key and the part of its counter that a launch shares.
struct Mask {
    uint32_t key0, key1, offset0, offset1, threshold;
    float scale;
};

__device__ __forceinline__ Mask mask_of(const Drop &d)
{
    Mask m{};
    m.threshold = d.threshold;
    m.scale = d.scale;
    if (d.threshold) {
        const uint64_t seed = d.rng[0], offset = d.rng[1];
        m.key0 = (uint32_t)seed;
        m.key1 = (uint32_t)(seed >> 32);
        m.offset0 = (uint32_t)offset;
        m.offset1 = (uint32_t)(offset >> 32);
    }
    return m;
}

__device__ __forceinline__ uint32_t exclusive_or(uint64_t a, uint32_t b, uint32_t c)
{
    return __builtin_amdgcn_bitop3_b32((uint32_t)a, b, c, 0x96);
}

// Philox4x32-10: ten rounds of two 32 x 32-bit products, whose halves change
// places, with a key that moves by a constant. 20 products of 64 bits for 8
// values: with 16 bits for each value their time stays below that of the
// values' own bytes.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, const Mask &m)
{
    uint32_t c2 = m.offset0, c3 = m.offset1, k0 = m.key0, k1 = m.key1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = exclusive_or(b >> 32, c1, k0);
        c1 = (uint32_t)b;
        c2 = exclusive_or(a >> 32, c3, k1);
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// Drops from columns [c, c + 8) of a row (c a multiple of 8).
__device__ __forceinline__ void drop8(const Mask &m, uint32_t row, uint32_t c, float *f)
{
    const u32x4 w = philox(c >> 3, row, m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t half = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
        f[e] = half >= m.threshold ? f[e] * m.scale : 0.0f;
    }
}

__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }

// Phi(-x) exp(x^2 / 2) of the normal distribution. It is smooth in t = 1 / (1 +
// 0.35 x) for x >= 0 and goes to 0 with it: t times a polynomial of degree 8,
// fitted here over x < 14 (beyond, the exponential is 0) to the least relative
// error, 3.2e-8.
__device__ __forceinline__ float normal_tail(float x)
{
    const float t = reciprocal(__builtin_fmaf(0.35f, x, 1.0f));
    float p = -0.029145967215299606f;
    p = __builtin_fmaf(p, t, 0.14397187530994415f);
    p = __builtin_fmaf(p, t, -0.2557145953178406f);
    p = __builtin_fmaf(p, t, 0.15917456150054932f);
    p = __builtin_fmaf(p, t, -0.023110102862119675f);
    p = __builtin_fmaf(p, t, 0.10550811141729355f);
    p = __builtin_fmaf(p, t, 0.119832843542099f);
    p = __builtin_fmaf(p, t, 0.13986186683177948f);
    p = __builtin_fmaf(p, t, 0.13962140679359436f);
    return p * t;
}

// 2^(y + rest) for a y of up to 150 and its rounding's rest: an exponent in
// one 32-bit number would carry that rounding, 10^-6 of the power's size.
__device__ __forceinline__ float power_of_two(float y, float rest)
{
    const float e = __builtin_amdgcn_exp2f(y);
    return __builtin_fmaf(0.6931471805599453f * e, rest, e);
}

// exp(-x), exp(-x^2 / 2) and exp(-2 u) of gelu_tanh's u = sqrt(2 / pi) (x +
// 0.044715 x^3) (0 where they are below 2^-126). WIDE, for what stays in 32 bits
// and x of 0 to 10^4: within 4 x 2^-24 of their size, the exponents' constants in
// two parts, and each product with its rest. Else the exponent is one 32-bit
// number, off by up to 343 x 2^-24 of the power's size (2^-15.6), which a result
// of 16 bits does not show, and x may be below 0.
template <bool WIDE>
__device__ __forceinline__ float exp_minus(float x)
{
#pragma clang fp contract(off)
    const float y = -1.4426950408889634f * x;
    if constexpr (!WIDE) return __builtin_amdgcn_exp2f(y);
    return power_of_two(y, __builtin_fmaf(-1.925963033e-8f, x, __builtin_fmaf(-1.4426950408889634f, x, -y)));
}

template <bool WIDE>
__device__ __forceinline__ float bell(float x)
{
#pragma clang fp contract(off)
    const float h = x * x, y = -0.72134752044448170f * h;
    if constexpr (!WIDE) return __builtin_amdgcn_exp2f(y);
    const float l = __builtin_fmaf(x, x, -h);
    const float rest = __builtin_fmaf(-0.72134752044448170f, l, __builtin_fmaf(-0.72134752044448170f, h, -y));
    return power_of_two(y, __builtin_fmaf(-9.629815167e-9f, h, rest));
}

template <bool WIDE>
__device__ __forceinline__ float exp_minus_cubic(float x)
{
#pragma clang fp contract(off)
    // x (2.302 + 0.1029 x^2), the factors of x with 2 sqrt(2 / pi) / log(2)
    const float a = 2.302208185195923f, b = 0.10294324159622192f, h = x * x;
    if constexpr (!WIDE) return __builtin_amdgcn_exp2f(-x * __builtin_fmaf(b, h, a));
    const float l = __builtin_fmaf(x, x, -h), w = b * h;
    const float w_rest = __builtin_fmaf(-2.0161985415e-9f, h, __builtin_fmaf(b, l, __builtin_fmaf(b, h, -w)));
    const float s = a + w, of_w = s - a;  // (a sum and its rounding, whichever is larger)
    const float s_rest = ((a - (s - of_w)) + (w - of_w)) + w_rest + 1.2948402350e-8f;
    const float y = -s * x;
    return power_of_two(y, __builtin_fmaf(-s_rest, x, __builtin_fmaf(-s, x, -y)));
}

// An activation by its share, z share(z) with share(-z) = 1 - share(z). Below 0
// the share goes to 0, and is computed to its own size: a value is within 18 x
// 2^-24 of its size where WIDE, else within 2^-15 (1,000 x 2,050 x 1,030 in f16 with
// gelu_tanh takes 19.0 us, and 20.9 where WIDE). Past 10^4 the share is at its
// limit anyway, and an infinity would meet the 0 it goes to.
template <int ACT, bool WIDE>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == kRelu) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == kGelu || ACT == kGeluTanh || ACT == kSilu) {
        const float from = __builtin_elementwise_maximum(z, -1e4f);  // (NaN stays)
        if constexpr (ACT != kGelu && !WIDE) {
            const float e = ACT == kSilu ? exp_minus<false>(from) : exp_minus_cubic<false>(from);
            return from * reciprocal(1.0f + e);
        }
        const float x = __builtin_elementwise_minimum(__builtin_fabsf(z), 1e4f);
        float below, above;
        if constexpr (ACT == kGelu) {
            below = bell<WIDE>(x) * normal_tail(x);
            above = 1.0f - below;
        } else {
            const float e = ACT == kSilu ? exp_minus<WIDE>(x) : exp_minus_cubic<WIDE>(x);
            above = reciprocal(1.0f + e);
            below = e * above;
        }
        return from * (z < 0.0f ? below : above);
    }
    return z;
}

// The slope at -x of a smooth activation, for x of 0 to 10^4; at x it is 1 less
// that. Near 0 for a large x, and then to its own size: a product of the
// exponential and what is left of the slope's two terms, within 16 x 2^-24 of
// their magnitudes.
template <int ACT>
__device__ __forceinline__ float act_slope_below(float x)
{
    static_assert(ACT == kGelu || ACT == kGeluTanh || ACT == kSilu, "");
    if constexpr (ACT == kGelu)
        return bell<true>(x) * __builtin_fmaf(-0.3989422804014327f, x, normal_tail(x));
    const float e = ACT == kSilu ? exp_minus<true>(x) : exp_minus_cubic<true>(x), r = reciprocal(1.0f + e);
    const float bend = ACT == kSilu ? 1.0f : 1.5957691216057308f * __builtin_fmaf(0.134145f, x * x, 1.0f);
    return e * r * __builtin_fmaf(-x * r, bend, 1.0f);
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == kRelu) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == kGelu || ACT == kGeluTanh || ACT == kSilu) {
        const float below = act_slope_below<ACT>(__builtin_elementwise_minimum(__builtin_fabsf(z), 1e4f));
        return z < 0.0f ? below : 1.0f - below;
    }
    return 1.0f;
}

template <int ACT, bool WIDE>
__device__ __forceinline__ void act_values(float *f)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = act_value<ACT, WIDE>(f[e]);
}

// The bias of columns [c, c + 8), zeros without one.
template <int DT>
__device__ __forceinline__ void bias8(const Epilogue &e, uint32_t c, uint32_t n, float *b)
{
    typename Elem<DT>::vec8 v = {};
    if (e.bias && c < n) v = load8<DT>((const typename Elem<DT>::raw *)e.bias, c, n);
#pragma unroll
    for (int q = 0; q < 8; ++q) b[q] = Elem<DT>::get(v[q]);
}

// The residual of columns [c, c + 8) of a row (zeros' bits without one).
template <int OUT>
__device__ __forceinline__ typename Elem<OUT>::vec8 residual8(const Epilogue &e, uint64_t row, uint32_t c, uint32_t n)
{
    typename Elem<OUT>::vec8 v = {};
    if (e.residual) v = load8<OUT>((const typename Elem<OUT>::raw *)e.residual + row * e.residual_stride, c, n);
    return v;
}

// Sums [c, c + 8) of a row of n (c a multiple of 8, below n) through the
// epilogue, with their bias and residual in hand.
template <int OUT>
__device__ __forceinline__ void finish8(const Epilogue &e, const Mask &mask, uint64_t row, uint32_t c, uint32_t n,
                                        float *f, const float *bias, typename Elem<OUT>::vec8 residual)
{
    if (e.bias) {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] += bias[q];
    }
    if (e.z) store8<OUT>((typename Elem<OUT>::raw *)e.z + row * n, c, n, f);
    constexpr bool WIDE = OUT == kF32;
    if (e.act == kRelu) act_values<kRelu, WIDE>(f);
    else if (e.act == kGelu) act_values<kGelu, WIDE>(f);
    else if (e.act == kGeluTanh) act_values<kGeluTanh, WIDE>(f);
    else if (e.act == kSilu) act_values<kSilu, WIDE>(f);
    if (mask.threshold) drop8(mask, (uint32_t)row, c, f);
    if (e.residual) {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] += Elem<OUT>::get(residual[q]);
    }
    store8<OUT>((typename Elem<OUT>::raw *)e.y + row * e.y_stride, c, n, f);
}

}  // namespace cpk
