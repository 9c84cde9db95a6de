// cp_dropout.hip - dropout with a mask that follows from (seed, offset, row,
// column), and the gradient back through a product's epilogue:
//
//   y  = drop(x) + residual
//   dz = drop(dy) act'(z), db = the sum of dz's rows
//
// Both read each value once and are bound by memory.
#include "cp_linear_internal.h"

namespace cpk {

namespace {

// Threads of a workgroup: 2^tx along a row, 8 columns each, the others along
// the rows. A wave takes 512 columns where there are as many.
struct Layout {
    uint32_t tx, columns, groups;  // workgroups along the columns, and along the rows
};

constexpr uint32_t kRowsAtOnce = 4;  // rows a thread has in flight

Layout layout_of(uint64_t m, uint64_t n, uint64_t most)
{
    Layout l{};
    l.tx = 0;
    while (l.tx < 6 && (8u << l.tx) < n) ++l.tx;
    l.columns = (uint32_t)div_up(n, 8u << l.tx);
    const uint64_t at_once = (256u >> l.tx) * kRowsAtOnce, whole = div_up(m, at_once);
    const uint64_t want = div_up(most, l.columns);
    l.groups = (uint32_t)(whole < want ? whole : want);
    if (l.groups == 0) l.groups = 1;
    return l;
}

template <int DT, bool RESIDUAL>
__global__ __launch_bounds__(256) void dropout_rows(const typename Elem<DT>::raw *x, uint64_t x_stride,
                                                    const typename Elem<DT>::raw *residual, uint64_t residual_stride,
                                                    uint32_t n, uint32_t d, uint32_t tx, uint32_t columns, Drop drop,
                                                    typename Elem<DT>::raw *y)
{
    const Mask mask = mask_of(drop);
    const uint32_t group = blockIdx.x / columns, column = blockIdx.x - group * columns, groups = gridDim.x / columns;
    const uint32_t c = (column << (3 + tx)) + (threadIdx.x & ((1u << tx) - 1)) * 8, ty = 256u >> tx;
    if (c >= d) return;
    // (counted in 64 bits: the rows end near 2^31)
    for (uint64_t at = (uint64_t)group * ty * kRowsAtOnce + (threadIdx.x >> tx); at < n;
         at += (uint64_t)groups * ty * kRowsAtOnce) {
        typename Elem<DT>::vec8 v[kRowsAtOnce], r[kRowsAtOnce];
#pragma unroll
        for (uint32_t q = 0; q < kRowsAtOnce; ++q) {
            const uint64_t row = at + q * ty < n ? at + q * ty : at;
            v[q] = load8<DT>(x + row * x_stride, c, d);
            if constexpr (RESIDUAL) r[q] = load8<DT>(residual + row * residual_stride, c, d);
        }
#pragma unroll
        for (uint32_t q = 0; q < kRowsAtOnce; ++q) {
            const uint64_t row = at + q * ty;
            if (row >= n) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = Elem<DT>::get(v[q][e]);
            if (mask.threshold) drop8(mask, (uint32_t)row, c, f);
            if constexpr (RESIDUAL) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += Elem<DT>::get(r[q][e]);
            }
            store8<DT>(y + row * d, c, d, f);
        }
    }
}

template <int DT, int ACT>
__global__ __launch_bounds__(256) void act_grad_rows(const typename Elem<DT>::raw *dy, uint64_t dy_stride,
                                                     const typename Elem<DT>::raw *z, uint64_t z_stride, uint32_t m,
                                                     uint32_t n, uint32_t tx, uint32_t columns, Drop drop,
                                                     typename Elem<DT>::raw *dz, float *__restrict__ partial)
{
    __shared__ float sums[256][9];
    const Mask mask = mask_of(drop);
    const uint32_t group = blockIdx.x / columns, column = blockIdx.x - group * columns, groups = gridDim.x / columns;
    const uint32_t c = (column << (3 + tx)) + (threadIdx.x & ((1u << tx) - 1)) * 8, ty = 256u >> tx;
    float db[8] = {};
    for (uint64_t at = (uint64_t)group * ty * kRowsAtOnce + (threadIdx.x >> tx); at < m && c < n;
         at += (uint64_t)groups * ty * kRowsAtOnce) {
        typename Elem<DT>::vec8 v[kRowsAtOnce], s[kRowsAtOnce];
#pragma unroll
        for (uint32_t q = 0; q < kRowsAtOnce; ++q) {
            const uint64_t row = at + q * ty < m ? at + q * ty : at;
            v[q] = load8<DT>(dy + row * dy_stride, c, n);
            if constexpr (ACT != kNone) s[q] = load8<DT>(z + row * z_stride, c, n);
        }
#pragma unroll
        for (uint32_t q = 0; q < kRowsAtOnce; ++q) {
            const uint64_t row = at + q * ty;
            if (row >= m) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = Elem<DT>::get(v[q][e]);
                if constexpr (ACT != kNone) f[e] *= act_slope<ACT>(Elem<DT>::get(s[q][e]));
            }
            if (mask.threshold) drop8(mask, (uint32_t)row, c, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) db[e] += f[e];
            store8<DT>(dz + row * n, c, n, f);
        }
    }
    if (!partial) return;
    // the workgroup's rows, in order
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = db[e];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < (8u << tx); i += 256) {
        float t = 0.0f;
        for (uint32_t q = 0; q < ty; ++q) t += sums[(q << tx) + (i >> 3)][i & 7u];
        const uint32_t at = (column << (3 + tx)) + i;
        if (at < n) partial[(uint64_t)group * n + at] = t;
    }
}

// db = the sum of the partial rows, in order: 32 columns a workgroup, 8 threads
// for each.
__global__ __launch_bounds__(256) void sum_rows(const float *__restrict__ partial, uint32_t count, uint32_t n,
                                                float *__restrict__ db)
{
    __shared__ float sums[8][32];
    const uint32_t g = threadIdx.x >> 5;
    for (uint32_t first = blockIdx.x * 32; first < n; first += gridDim.x * 32) {
        const uint32_t c = first + (threadIdx.x & 31u);
        float t = 0.0f;
        if (c < n)
            for (uint32_t p = g; p < count; p += 8) t += partial[(uint64_t)p * n + c];
        sums[g][threadIdx.x & 31u] = t;
        __syncthreads();
        if (g == 0 && c < n) {
#pragma unroll
            for (int q = 1; q < 8; ++q) t += sums[q][threadIdx.x & 31u];
            db[c] = t;
        }
        __syncthreads();
    }
}

constexpr uint64_t kMostWorkgroups = 2048;  // eight for each compute unit
constexpr uint64_t kMostSums = 1u << 20;    // a launch has fewer than 2^32 threads, and columns stay below 2^32

template <int DT>
hipError_t launch_dropout(const DropoutArgs &a)
{
    typedef const typename Elem<DT>::raw *in;
    const Layout l = layout_of(a.n, a.d, kMostWorkgroups);
    const uint32_t blocks = l.columns * l.groups;
    if (a.residual)
        dropout_rows<DT, true><<<blocks, 256, 0, a.stream>>>((in)a.x, a.x_stride, (in)a.residual, a.residual_stride,
                                                             (uint32_t)a.n, (uint32_t)a.d, l.tx, l.columns, a.drop,
                                                             (typename Elem<DT>::raw *)a.y);
    else
        dropout_rows<DT, false><<<blocks, 256, 0, a.stream>>>((in)a.x, a.x_stride, nullptr, 0, (uint32_t)a.n,
                                                              (uint32_t)a.d, l.tx, l.columns, a.drop,
                                                              (typename Elem<DT>::raw *)a.y);
    return hipGetLastError();
}

template <int DT, int ACT>
hipError_t launch_act_grad(const ActGradArgs &a)
{
    typedef const typename Elem<DT>::raw *in;
    const Layout l = layout_of(a.m, a.n, kMostWorkgroups);
    act_grad_rows<DT, ACT><<<l.columns * l.groups, 256, 0, a.stream>>>(
        (in)a.dy, a.dy_stride, (in)a.z, a.z_stride, (uint32_t)a.m, (uint32_t)a.n, l.tx, l.columns, a.drop,
        (typename Elem<DT>::raw *)a.dz, a.db ? (float *)a.workspace : nullptr);
    if (a.db) {
        const uint64_t wgs = div_up(a.n, 32);
        sum_rows<<<(uint32_t)(wgs < kMostSums ? wgs : kMostSums), 256, 0, a.stream>>>(
            (const float *)a.workspace, l.groups, (uint32_t)a.n, a.db);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t act_grad_of(const ActGradArgs &a)
{
    switch (a.act) {
    case kRelu: return launch_act_grad<DT, kRelu>(a);
    case kGelu: return launch_act_grad<DT, kGelu>(a);
    case kGeluTanh: return launch_act_grad<DT, kGeluTanh>(a);
    case kSilu: return launch_act_grad<DT, kSilu>(a);
    default: return launch_act_grad<DT, kNone>(a);
    }
}

}  // namespace

uint64_t act_grad_workspace_bytes(uint64_t m, uint64_t n)
{
    return 4ull * layout_of(m, n, kMostWorkgroups).groups * n;
}

hipError_t act_grad(const ActGradArgs &a)
{
    if (a.dtype == kBF16) return act_grad_of<kBF16>(a);
    if (a.dtype == kF16) return act_grad_of<kF16>(a);
    return act_grad_of<kF32>(a);
}

hipError_t dropout(const DropoutArgs &a)
{
    if (a.dtype == kBF16) return launch_dropout<kBF16>(a);
    if (a.dtype == kF16) return launch_dropout<kF16>(a);
    return launch_dropout<kF32>(a);
}

}  // namespace cpk
