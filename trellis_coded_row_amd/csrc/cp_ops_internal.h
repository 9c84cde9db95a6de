// Internal interface of the dense operators (include/cp_ops.h): launch
// parameters, and the device helpers their kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cpk {

// Element types as in cp_dtype (include/cp_ops.h).
enum DType { kF32 = 0, kBF16 = 1, kF16 = 2 };

constexpr uint32_t dtype_bytes(int t) { return t == kF32 ? 4u : 2u; }

constexpr uint64_t align256(uint64_t x) { return (x + 255) & ~(uint64_t)255; }

constexpr uint64_t div_up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

struct EmbedLookupArgs {
    const void *table;
    int table_dtype;
    uint64_t rows, d, row_stride;
    const int64_t *ids;
    uint64_t n;
    float scale;
    void *out;
    int out_dtype;
    int32_t *bad_id;
    hipStream_t stream;
};
hipError_t embed_lookup(const EmbedLookupArgs &a);

struct EmbedPlanArgs {
    const int64_t *ids;
    uint64_t n, rows;
    int32_t *order, *slot;
    int64_t *unique;
    int32_t *starts;
    int64_t *count;
    uint8_t *workspace;
    hipStream_t stream;
};
uint64_t embed_plan_workspace_bytes(uint64_t n, uint64_t rows);
hipError_t embed_plan(const EmbedPlanArgs &a);

struct EmbedGradArgs {
    const int32_t *order, *slot;
    const int64_t *unique;
    const int32_t *starts;
    const int64_t *count;
    uint64_t n, rows;  // rows 0: distinct rows only
    const void *dout;
    int dtype;
    uint64_t d, stride;
    float scale;
    float *grad;
    uint8_t *workspace;
    hipStream_t stream;
};
uint64_t embed_grad_workspace_bytes(uint64_t n, uint64_t d);
hipError_t embed_grad(const EmbedGradArgs &a);

struct NormArgs {
    const void *x, *residual, *weight;
    uint64_t x_stride, residual_stride;
    int dtype;
    uint64_t n, d;
    float eps;
    void *h, *y;
    uint8_t *q, *q_scale;
    uint64_t q_stride, scale_stride;
    float *rstd;
    hipStream_t stream;
};
hipError_t rms_norm(const NormArgs &a);

struct NormGradArgs {
    const void *dy, *x, *weight, *dres;
    uint64_t dy_stride, x_stride, dres_stride;
    const float *rstd;
    int dtype;
    uint64_t n, d;
    void *dx;
    float *dw;
    uint8_t *workspace;
    hipStream_t stream;
};
uint64_t rms_norm_grad_workspace_bytes(uint64_t n, uint64_t d);
hipError_t rms_norm_grad(const NormGradArgs &a);

struct QuantArgs {
    const void *x;
    int dtype;
    uint64_t n, d, x_stride;
    bool blocks;
    uint8_t *q, *scale, *qt, *scale_t;
    uint64_t q_stride, scale_stride, qt_stride, scale_t_stride;
    hipStream_t stream;
};
hipError_t quantize_fp8(const QuantArgs &a);

struct GemmArgs {
    const uint8_t *a, *a_scale, *b, *b_scale;
    uint64_t a_stride, a_scale_stride, b_stride, b_scale_stride;
    bool b_blocks;
    uint64_t m, n, k;
    void *out;
    uint64_t out_stride;
    int out_dtype;
    uint8_t *workspace;
    hipStream_t stream;
};
uint64_t gemm_fp8_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int out_dtype);
hipError_t gemm_fp8(const GemmArgs &a);

// ---------------------------------------------------------------- device

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 elements at any element-aligned address: gfx950 reads and writes
// 16 bytes at any alignment in one access, so rows of odd length need no
// path of their own.
template <int DT>
struct Elem;

template <>
struct Elem<kF32> {
    typedef float raw;
    typedef float vec8 __attribute__((ext_vector_type(8), aligned(4)));
    static __device__ __forceinline__ float get(raw r) { return r; }
    static __device__ __forceinline__ raw put(float f) { return f; }
};

template <>
struct Elem<kBF16> {
    typedef uint16_t raw;
    typedef uint16_t vec8 __attribute__((ext_vector_type(8), aligned(2)));
    static __device__ __forceinline__ float get(raw r) { return __uint_as_float((uint32_t)r << 16); }
    static __device__ __forceinline__ raw put(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};

template <>
struct Elem<kF16> {
    typedef uint16_t raw;
    typedef uint16_t vec8 __attribute__((ext_vector_type(8), aligned(2)));
    static __device__ __forceinline__ float get(raw r) { return (float)__builtin_bit_cast(_Float16, r); }
    static __device__ __forceinline__ raw put(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};

// Elements [c, c + 8) of a row of d, zeros past its end.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::vec8 load8(const typename Elem<DT>::raw *row, uint32_t c, uint32_t d)
{
    typedef typename Elem<DT>::vec8 V;
    V v;
    if (c + 8 <= d) {
        v = *reinterpret_cast<const V *>(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < d ? row[c + e] : (typename Elem<DT>::raw)0;
    }
    return v;
}

template <int DT, bool NT = false>
__device__ __forceinline__ void store8(typename Elem<DT>::raw *row, uint32_t c, uint32_t d, const float *f)
{
    typedef typename Elem<DT>::vec8 V;
    V v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Elem<DT>::put(f[e]);
    if (c + 8 <= d) {
        if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<V *>(row + c));
        else *reinterpret_cast<V *>(row + c) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < d) row[c + e] = v[e];
    }
}

// |x| as its bits, 0 for what is not finite: the larger magnitude has the
// larger bits, so a maximum of these is a maximum of finite magnitudes.
__device__ __forceinline__ uint32_t finite_bits(float x)
{
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// The e8m0 byte of a group's scale from the bits of its largest magnitude A:
// A = 1.m * 2^(E - 127) and 448 = 1.75 * 2^8, so the least e with
// A <= 448 * 2^e is E - 135, one more when 1.m > 1.75; the byte is e + 127,
// not below 0 (A below 2^-119 or so: its values round to zero or nearly).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    if (amax_bits == 0) return 127u;
    const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b > 0 ? (uint32_t)b : 0u;
}

// 2^-e for the scale byte e + 127 (at most 247, so this is a normal number).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// x in the units of its scale; what is not finite becomes NaN.
__device__ __forceinline__ float scaled_or_nan(float x, float inv)
{
    return __builtin_isfinite(x) ? x * inv : __builtin_nanf("");
}

// Four values in e4m3 (round to nearest even), each times inv.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, float inv)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_or_nan(a, inv), scaled_or_nan(b, inv), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(scaled_or_nan(c, inv), scaled_or_nan(d, inv), r, true);
    return (uint32_t)r;
}

// The same for finite values.
__device__ __forceinline__ uint32_t finite_to_e4m3x4(float a, float b, float c, float d, float inv)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
    return (uint32_t)r;
}

// The value of the lane r places further round this lane's row of 16.
template <int R>
__device__ __forceinline__ int row_rotate(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, 0x120 | R, 0xF, 0xF, false);
}

// Maximum over the 16 lanes of a row, in every lane of it.
__device__ __forceinline__ uint32_t max_of_16(uint32_t v)
{
    uint32_t o = (uint32_t)row_rotate<8>((int)v);
    v = v > o ? v : o;
    o = (uint32_t)row_rotate<4>((int)v);
    v = v > o ? v : o;
    o = (uint32_t)row_rotate<2>((int)v);
    v = v > o ? v : o;
    o = (uint32_t)row_rotate<1>((int)v);
    return v > o ? v : o;
}

// Sum over the wave, the same bits in every lane of a row of 16 and across
// rows (each step adds the same two numbers in both lanes).
__device__ __forceinline__ float sum_of_64(float v)
{
    v += __int_as_float(row_rotate<8>(__float_as_int(v)));
    v += __int_as_float(row_rotate<4>(__float_as_int(v)));
    v += __int_as_float(row_rotate<2>(__float_as_int(v)));
    v += __int_as_float(row_rotate<1>(__float_as_int(v)));
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    return v;
}

}  // namespace cpk
