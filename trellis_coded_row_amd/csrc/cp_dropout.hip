// cp_dropout.hip - dropout with a mask that follows from (seed, offset, row,
// column), and the gradient back through a product's epilogue:
//
//   y  = drop(x) + residual
//   dz = drop(dy) act'(z), db = the sum of dz's rows
//
// Both read each value once and are bound by memory.
#include <type_traits>

#include "cp_linear_internal.h"

namespace cpk {

namespace {

// Threads of a workgroup: 2^tx along a row, 8 columns each, the others along
// the rows. A wave takes 512 columns where there are as many.
struct Layout {
    uint32_t tx, columns, groups;  // workgroups along the columns, and along the rows
    bool many;                     // several rows in flight
    bool runs;                     // their order, see place_of
};

// Rows a thread has in flight where there are enough for eight workgroups on
// each compute unit, else one: four for dropout (393,216 x 512 in bf16: 144 us,
// with two 159; 1,000 x 2,050: 6.1, with two 4.1, with one 3.9), two for the
// gradient, which needs the registers.
constexpr uint32_t kDropRows = 4, kGradRows = 2;

// (n is not 0)
Layout layout_of(uint64_t m, uint64_t n, int dtype, uint32_t rows)
{
    constexpr uint64_t most = 2048;  // workgroups: eight for each compute unit
    Layout l{};
    l.runs = n * dtype_bytes(dtype) % 128 != 0;
    l.tx = 0;
    while (l.tx < 6 && (8u << l.tx) < n) ++l.tx;
    // (fewer lanes along a row where more than an eighth of them would lie past its end)
    while (l.tx > 3 && div_up(n, 8u << l.tx) * (8u << l.tx) > n + n / 8 + 8) --l.tx;
    l.columns = (uint32_t)div_up(n, 8u << l.tx);
    l.many = l.columns * div_up(m, (256u >> l.tx) * rows) >= most;
    const uint64_t at_once = (256u >> l.tx) * (l.many ? rows : 1), whole = div_up(m, at_once);
    const uint64_t want = div_up(most, l.columns);
    l.groups = (uint32_t)(whole < want ? whole : want);
    if (l.groups == 0) l.groups = 1;
    return l;
}

// 8 values of a row: all of them, or those before the row's end.
template <int DT, bool WHOLE>
__device__ __forceinline__ typename Elem<DT>::vec8 get8(const typename Elem<DT>::raw *row, uint32_t c, uint32_t n)
{
    if constexpr (WHOLE) return *reinterpret_cast<const typename Elem<DT>::vec8 *>(row + c);
    return load8<DT>(row, c, n);
}

template <int DT, bool WHOLE>
__device__ __forceinline__ void put8(typename Elem<DT>::raw *row, uint32_t c, uint32_t n, const float *f)
{
    store8<DT>(row, c, WHOLE ? c + 8 : n, f);
}

// A workgroup's place: its first column and row, and how far its rows lie apart.
struct Place {
    uint32_t group, column, groups, c, ty, row;
};

__device__ __forceinline__ Place place_of(uint32_t tx, uint32_t columns, bool runs)
{
    Place p;
    // Places in turn, or for each of the 8 XCDs (workgroup ids taken in turn) a
    // contiguous run of them, where rows start inside a line: the pieces of a
    // row that share one then meet in one L2 (60,000 x 1,100 in f16: 66 -> 62
    // us; rows that start on lines are read faster in turn, 8,192 x 16,384 in
    // bf16 104 us against 108).
    const uint32_t xcd = blockIdx.x & 7u, per = gridDim.x >> 3, extra = gridDim.x & 7u;
    const uint32_t id = runs ? xcd * per + (xcd < extra ? xcd : extra) + (blockIdx.x >> 3) : blockIdx.x;
    p.group = id / columns;
    p.column = id - p.group * columns;
    p.groups = gridDim.x / columns;
    p.c = (p.column << (3 + tx)) + (threadIdx.x & ((1u << tx) - 1)) * 8;
    p.ty = 256u >> tx;
    p.row = threadIdx.x >> tx;
    return p;
}

// Calls work(row) for this thread's rows, R at a time: first load(q,
// row) for each, then work(q, row). Rows are counted in 64 bits: they end near
// 2^31.
template <uint32_t R, typename Load, typename Work>
__device__ __forceinline__ void over_rows(const Place &p, uint32_t rows, Load load, Work work)
{
    for (uint64_t at = (uint64_t)p.group * p.ty * R + p.row; at < rows;
         at += (uint64_t)p.groups * p.ty * R) {
#pragma unroll
        for (uint32_t q = 0; q < R; ++q) load(q, at + q * p.ty < rows ? at + q * p.ty : at);
#pragma unroll
        for (uint32_t q = 0; q < R; ++q)
            if (at + q * p.ty < rows) work(q, at + q * p.ty);
    }
}

template <int DT, bool RESIDUAL, uint32_t R>
__global__ __launch_bounds__(256) void dropout_rows(const typename Elem<DT>::raw *x, uint64_t x_stride,
                                                    const typename Elem<DT>::raw *residual, uint64_t residual_stride,
                                                    uint32_t n, uint32_t d, uint32_t tx, uint32_t columns, bool runs, Drop drop,
                                                    typename Elem<DT>::raw *y)
{
    const Mask mask = mask_of(drop);
    const Place p = place_of(tx, columns, runs);
    const auto rows = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        typename Elem<DT>::vec8 v[R], r[R];
        over_rows<R>(
            p, n,
            [&](uint32_t q, uint64_t row) {
                v[q] = get8<DT, WHOLE>(x + row * x_stride, p.c, d);
                if constexpr (RESIDUAL) r[q] = get8<DT, WHOLE>(residual + row * residual_stride, p.c, d);
            },
            [&](uint32_t q, uint64_t row) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = Elem<DT>::get(v[q][e]);
                if (mask.threshold) drop8(mask, (uint32_t)row, p.c, f);
                if constexpr (RESIDUAL) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += Elem<DT>::get(r[q][e]);
                }
                put8<DT, WHOLE>(y + row * d, p.c, d, f);
            });
    };
    if (__all(p.c + 8 <= d)) rows(std::true_type{});
    else if (p.c < d) rows(std::false_type{});
}

// The slope of a smooth activation from 512 cubics in LDS, for |z| in pieces of
// 1 / PIECES: of the slope at -|z|, from which that at |z| is 1 less it, so that
// a slope far below 0 keeps its own size's precision (held as 1/2 and an odd
// part it would be the difference of two halves, off by 3e-8 whatever its size).
// A piece's cubic goes through the slope at its ends and a quarter from each, and
// is off by at most h^4 / 1536 times the fourth derivative: 5 x 2^-24 of the
// slope's terms where it falls fastest. With the roundings of the four values
// and of the cubic's own a slope is within 44 x 2^-24 of them (7 at most in 2^21
// values of each). From -DEEP down the formula takes over, for values of a wave
// that has some; past DEEP the slope is 1.
// The formula alone would bound the time: 8,192 x 16,384 in bf16 with dropout and
// z of deviation 1.5 takes 152 to 154 us with gelu (5.3 TB/s; by the formula
// 169), 152 with gelu_tanh (181), 151 with silu (154). With z of deviation 6, where
// every wave has deep values, 181, 192 and 154.
template <int ACT>
struct Slopes {
    static constexpr bool TABLE = ACT == kGelu || ACT == kGeluTanh || ACT == kSilu;
    static constexpr uint32_t COUNT = TABLE ? 512 : 1;
    static constexpr float PIECES = ACT == kSilu ? 16.0f : 64.0f;  // for each 1 of |z|
    static constexpr float DEEP = ACT == kSilu ? 32.0f : ACT == kGelu ? 8.0f : 6.0f;  // (a gelu_tanh falls faster)

    static __device__ __forceinline__ void fill(f32x4 *cubic)
    {
        if constexpr (TABLE) {
            for (uint32_t i = threadIdx.x; i < COUNT; i += 256) {
                const auto slope = [&](float at) { return act_slope_below<ACT>(((float)i + at) * (1.0f / PIECES)); };
                const float a0 = slope(0.0f), b0 = slope(0.25f), b1 = slope(0.75f), a1 = slope(1.0f);
                const float even_a = 0.5f * (a1 + a0), odd_a = a1 - a0, even_b = 0.5f * (b1 + b0), odd_b = 2.0f * (b1 - b0);
                // about the middle, then from the piece's start
                const float c2 = (even_a - even_b) * (16.0f / 3.0f), c3 = (odd_a - odd_b) * (16.0f / 3.0f);
                const float c1 = odd_b - 0.0625f * c3;
                cubic[i] = f32x4{a0, c1 - c2 + 0.75f * c3, c2 - 1.5f * c3, c3};
            }
            __syncthreads();
        }
    }

    // of z above -DEEP
    static __device__ __forceinline__ float at(const f32x4 *cubic, float z)
    {
        if constexpr (!TABLE) return act_slope<ACT>(z);
        // NaN takes the last piece (a whole number cannot be made of it) and stays NaN on the way through it
        const float far = PIECES * __builtin_fabsf(z), last = 511.99997f;
        const f32x4 c = cubic[(uint32_t)__builtin_fminf(far, last)];
        const float f = __builtin_amdgcn_fractf(__builtin_elementwise_minimum(far, last));
        const float below = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(c[3], f, c[2]), f, c[1]), f, c[0]);
        return z < 0.0f ? below : 1.0f - below;
    }

    // The slopes at 8 values.
    static __device__ __forceinline__ void at8(const f32x4 *cubic, const float *z, float *slope)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) slope[e] = at(cubic, z[e]);
        if constexpr (TABLE) {
            // the largest bits are those of the value furthest below 0 (or of a NaN)
            uint32_t low = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) low = __float_as_uint(z[e]) > low ? __float_as_uint(z[e]) : low;
            if (low >= __float_as_uint(-DEEP)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (z[e] <= -DEEP) slope[e] = act_slope<ACT>(z[e]);
            }
        }
    }
};

template <int DT, int ACT, uint32_t R>
__global__ __launch_bounds__(256) void act_grad_rows(const typename Elem<DT>::raw *dy, uint64_t dy_stride,
                                                     const typename Elem<DT>::raw *z, uint64_t z_stride, uint32_t m,
                                                     uint32_t n, uint32_t tx, uint32_t columns, bool runs, Drop drop,
                                                     typename Elem<DT>::raw *dz, float *__restrict__ partial)
{
    typedef Slopes<ACT> S;
    __shared__ __attribute__((aligned(16))) union {
        f32x4 cubic[S::COUNT];
        float sums[256][9];
    } lds;
    const Mask mask = mask_of(drop);
    const Place p = place_of(tx, columns, runs);
    S::fill(lds.cubic);
    float db[8] = {};
    const auto rows = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        typename Elem<DT>::vec8 v[R], s[R];
        over_rows<R>(
            p, m,
            [&](uint32_t q, uint64_t row) {
                v[q] = get8<DT, WHOLE>(dy + row * dy_stride, p.c, n);
                if constexpr (ACT != kNone) s[q] = get8<DT, WHOLE>(z + row * z_stride, p.c, n);
            },
            [&](uint32_t q, uint64_t row) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = Elem<DT>::get(v[q][e]);
                if constexpr (ACT != kNone) {
                    float z8[8], slope[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) z8[e] = Elem<DT>::get(s[q][e]);
                    S::at8(lds.cubic, z8, slope);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= slope[e];
                }
                if (mask.threshold) drop8(mask, (uint32_t)row, p.c, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) db[e] += f[e];
                put8<DT, WHOLE>(dz + row * n, p.c, n, f);
            });
    };
    if (__all(p.c + 8 <= n)) rows(std::true_type{});
    else if (p.c < n) rows(std::false_type{});
    if (!partial) return;
    // the workgroup's rows, in order
    __syncthreads();  // (the cubics' place is taken)
#pragma unroll
    for (int e = 0; e < 8; ++e) lds.sums[threadIdx.x][e] = db[e];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < (8u << tx); i += 256) {
        float t = 0.0f;
        for (uint32_t q = 0; q < p.ty; ++q) t += lds.sums[(q << tx) + (i >> 3)][i & 7u];
        const uint32_t at = (p.column << (3 + tx)) + i;
        if (at < n) partial[(uint64_t)p.group * n + at] = t;
    }
}

// db = the sum of the partial rows, in a fixed order: 32 columns a workgroup, 32
// threads for each.
__global__ __launch_bounds__(1024) void sum_rows(const float *__restrict__ partial, uint32_t count, uint32_t n,
                                                 float *__restrict__ db)
{
    __shared__ float sums[32][33];
    const uint32_t g = threadIdx.x >> 5;
    for (uint32_t first = blockIdx.x * 32; first < n; first += gridDim.x * 32) {
        const uint32_t c = first + (threadIdx.x & 31u);
        float t = 0.0f;
        if (c < n) {
#pragma unroll 8
            for (uint32_t p = g; p < count; p += 32) t += partial[(uint64_t)p * n + c];
        }
        sums[g][threadIdx.x & 31u] = t;
        __syncthreads();
        if (g == 0 && c < n) {
#pragma unroll
            for (int q = 1; q < 32; ++q) t += sums[q][threadIdx.x & 31u];
            db[c] = t;
        }
        __syncthreads();
    }
}

constexpr uint64_t kMostSums = 1u << 20;    // a launch has fewer than 2^32 threads, and columns stay below 2^32

template <int DT, bool RESIDUAL, uint32_t R>
hipError_t launch_dropout(const DropoutArgs &a, const Layout &l)
{
    typedef const typename Elem<DT>::raw *in;
    dropout_rows<DT, RESIDUAL, R><<<l.columns * l.groups, 256, 0, a.stream>>>(
        (in)a.x, a.x_stride, (in)a.residual, a.residual_stride, (uint32_t)a.n, (uint32_t)a.d, l.tx, l.columns, l.runs,
        a.drop, (typename Elem<DT>::raw *)a.y);
    return hipGetLastError();
}

template <int DT>
hipError_t dropout_of(const DropoutArgs &a)
{
    const Layout l = layout_of(a.n, a.d, DT, kDropRows);
    if (a.residual) return l.many ? launch_dropout<DT, true, kDropRows>(a, l) : launch_dropout<DT, true, 1>(a, l);
    return l.many ? launch_dropout<DT, false, kDropRows>(a, l) : launch_dropout<DT, false, 1>(a, l);
}

template <int DT, int ACT, uint32_t R>
hipError_t launch_act_grad(const ActGradArgs &a, const Layout &l)
{
    typedef const typename Elem<DT>::raw *in;
    act_grad_rows<DT, ACT, R><<<l.columns * l.groups, 256, 0, a.stream>>>(
        (in)a.dy, a.dy_stride, (in)a.z, a.z_stride, (uint32_t)a.m, (uint32_t)a.n, l.tx, l.columns, l.runs, a.drop,
        (typename Elem<DT>::raw *)a.dz, a.db ? (float *)a.workspace : nullptr);
    if (a.db) {
        const uint64_t wgs = div_up(a.n, 32);
        sum_rows<<<(uint32_t)(wgs < kMostSums ? wgs : kMostSums), 1024, 0, a.stream>>>(
            (const float *)a.workspace, l.groups, (uint32_t)a.n, a.db);
    }
    return hipGetLastError();
}

template <int DT, int ACT>
hipError_t act_grad_with(const ActGradArgs &a)
{
    const Layout l = layout_of(a.m, a.n, DT, kGradRows);
    return l.many ? launch_act_grad<DT, ACT, kGradRows>(a, l) : launch_act_grad<DT, ACT, 1>(a, l);
}

template <int DT>
hipError_t act_grad_of(const ActGradArgs &a)
{
    switch (a.act) {
    case kRelu: return act_grad_with<DT, kRelu>(a);
    case kGelu: return act_grad_with<DT, kGelu>(a);
    case kGeluTanh: return act_grad_with<DT, kGeluTanh>(a);
    case kSilu: return act_grad_with<DT, kSilu>(a);
    default: return act_grad_with<DT, kNone>(a);
    }
}

}  // namespace

uint64_t act_grad_workspace_bytes(uint64_t m, uint64_t n)
{
    return 4ull * layout_of(m, n, kF32, kGradRows).groups * n;
}

hipError_t act_grad(const ActGradArgs &a)
{
    if (a.dtype == kBF16) return act_grad_of<kBF16>(a);
    if (a.dtype == kF16) return act_grad_of<kF16>(a);
    return act_grad_of<kF32>(a);
}

hipError_t dropout(const DropoutArgs &a)
{
    if (a.dtype == kBF16) return dropout_of<kBF16>(a);
    if (a.dtype == kF16) return dropout_of<kF16>(a);
    return dropout_of<kF32>(a);
}

}  // namespace cpk
