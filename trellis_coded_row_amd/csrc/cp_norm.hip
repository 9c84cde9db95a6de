// cp_norm.hip - root-mean-square norm with the residual's addition and an
// 8-bit output, and its gradient.
//
//   h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//   dx = rstd (g - xhat mean(g xhat)) + dres, g = dy w, xhat = x rstd
//   dw = sum over rows of dy xhat
//
// Both are bound by memory: a row of up to 32,768 columns is read once and
// stays in registers between its reduction and its outputs (in the gradient of
// more than 16,384 columns some of it in scratch memory, see there); longer
// ones are read twice. Sums run in 32 bits.
//
// h stays in 32 bits on its way to y and rstd. The gradient is taken at the h
// that was stored, which is rounded: in 16 bits, at slightly another point.
#include "cp_ops_internal.h"

namespace cpk {

namespace {

// Rows or workgroups of one launch, at most: its threads (1,024 a workgroup)
// are counted in 32 bits, and a launch of more than 2^32 runs the remainder
// alone, without an error.
constexpr uint64_t kMaxRows = 1u << 21;

// Sum over the W waves that share a row (W == 1: the wave alone).
template <int W>
__device__ __forceinline__ float row_sum(float v, float *part)
{
    v = sum_of_64(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int q = 0; q < W; ++q) v += part[q];
    }
    return v;
}

// The 8-bit outputs of columns [c, c + 8) (y zero past the row's end); the
// 16 lanes of a row of lanes hold one group of 128.
__device__ __forceinline__ void put_group(const float *y, uint32_t c, uint32_t d, uint8_t *q, uint8_t *scale)
{
    float most = 0.0f;  // NaN where one of the values is
#pragma unroll
    for (int e = 0; e < 8; ++e) most = __builtin_elementwise_maximum(most, __builtin_fabsf(y[e]));
    uint32_t top = max_of_16(__float_as_uint(most) & 0x7FFFFFFFu);
    const bool odd = top >= 0x7F800000u;  // the group has values that are not finite
    if (odd) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = finite_bits(y[e]);
            m = m > b ? m : b;
        }
        top = max_of_16(m);
    }
    const uint32_t sb = scale_byte(top);
    const float inv = inverse_scale(sb);
    if (c >= d) return;
    u32x2 v;
    if (odd) {
        v[0] = to_e4m3x4(y[0], y[1], y[2], y[3], inv);
        v[1] = to_e4m3x4(y[4], y[5], y[6], y[7], inv);
    } else {
        v[0] = finite_to_e4m3x4(y[0], y[1], y[2], y[3], inv);
        v[1] = finite_to_e4m3x4(y[4], y[5], y[6], y[7], inv);
    }
    if (c + 8 <= d) {
        *reinterpret_cast<u32x2 *>(q + c) = v;
    } else {
        for (uint32_t e = 0; c + e < d; ++e) q[c + e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3u)));
    }
    if ((threadIdx.x & 15u) == 0) scale[c >> 7] = (uint8_t)sb;
}

// Registers that a row's values (x, the residual, the weight) and those of the
// next row take, per lane; where they are few enough, workgroups stay, keep
// the weight, and read the next row while they work on this one.
template <int DT, int IT, bool RES>
constexpr bool kAhead = (RES ? 5 : 3) * IT * (DT == kF32 ? 8 : 4) <= 40;

constexpr uint32_t kAheadWaves = 4096;  // waves that stay: four for each SIMD unit

// W waves per row, IT chunks of 8 columns per lane: chunk i of a lane is
// columns 8 (64 W i + lane of the row).
//
// Bound by memory: 4,096 bf16 rows of 24,576 to 8 bits take 63 us, 4.8 TB/s (a
// copy reaches 5.0). With one row per workgroup, none read ahead, 73 us: then
// a workgroup's loads, its barrier and its stores follow one another. That is
// how rows too long to be read ahead go (kAhead): the same rows with a residual
// take 132 us, in 32 bits 243, both 5.4 TB/s with part of them in the last level
// cache.
template <int DT, int W, int IT, bool RES>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64, 4) void norm_rows(
    const typename Elem<DT>::raw *__restrict__ x, uint64_t x_stride, const typename Elem<DT>::raw *__restrict__ res,
    uint64_t res_stride, const typename Elem<DT>::raw *__restrict__ weight, uint32_t n, uint32_t d, float eps,
    typename Elem<DT>::raw *__restrict__ h_out, typename Elem<DT>::raw *__restrict__ y_out, uint8_t *__restrict__ q,
    uint64_t q_stride, uint8_t *__restrict__ q_scale, uint64_t scale_stride, float *__restrict__ rstd_out)
{
    typedef typename Elem<DT>::vec8 V;
    constexpr bool AHEAD = kAhead<DT, IT, RES>;
    __shared__ float part[2][W];
    const uint32_t groups = W == 1 ? gridDim.x * 4u : gridDim.x;
    const uint32_t first = W == 1 ? blockIdx.x * 4u + (threadIdx.x >> 6) : blockIdx.x;
    const uint32_t lane = W == 1 ? threadIdx.x & 63u : threadIdx.x;
    if (first >= n) return;  // whole waves of a W == 1 workgroup, which has no barrier
    V vx[IT], vr[RES ? IT : 1], nx[IT], nr[RES ? IT : 1], vw[IT];
    const auto load = [&](uint32_t row, V *ax, V *ar) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            ax[i] = load8<DT>(x + row * x_stride, (i * W * 64u + lane) * 8u, d);
            if constexpr (RES) ar[i] = load8<DT>(res + row * res_stride, (i * W * 64u + lane) * 8u, d);
        }
    };
    const auto value = [&](int i, int e) {
        float h = Elem<DT>::get(vx[i][e]);
        if constexpr (RES) h += Elem<DT>::get(vr[i][e]);
        return h;
    };
    load(first, vx, vr);
    if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < IT; ++i) vw[i] = load8<DT>(weight, (i * W * 64u + lane) * 8u, d);
    }
    int flip = 0;
    uint32_t row = first;
    do {
        if (AHEAD && row + groups < n) load(row + groups, nx, nr);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = value(i, e);
                sum = fmaf(h, h, sum);
            }
        }
        sum = row_sum<W>(sum, part[flip]);  // two places in turn: a barrier a row
        flip ^= 1;
        const float rstd = rsqrtf(sum / (float)d + eps);
        if (rstd_out && lane == 0) rstd_out[row] = rstd;
        // from here the values are made from x and the residual again: kept,
        // they would take twice the registers
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            asm volatile("" : "+v"(vx[i]));
            if constexpr (RES) asm volatile("" : "+v"(vr[i]));
            if constexpr (AHEAD) asm volatile("" : "+v"(vw[i]));
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // one chunk's values at a time
            const uint32_t c = (i * W * 64u + lane) * 8u;
            if constexpr (RES) {
                float h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = value(i, e);
                if (h_out && c < d) store8<DT>(h_out + (uint64_t)row * d, c, d, h);
            }
            if (!AHEAD && (y_out || q)) vw[i] = load8<DT>(weight, c, d);
            if (!y_out && !q) continue;
            // (past the row's end, h and the weight are zero. Of 100 million
            // 8-bit values 45 to 65 lie so near a border that they fall on its
            // other side than in 64 bits. With a corrected root and one
            // rounding of the product they are 40 to 60, at 2 to 3 us more:
            // not kept; two products in 32 bits are what the formula says)
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = value(i, e) * rstd * Elem<DT>::get(vw[i][e]);
            if (y_out && c < d) store8<DT>(y_out + (uint64_t)row * d, c, d, y);
            if (q) put_group(y, c, d, q + row * q_stride, q_scale + row * scale_stride);
        }
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                vx[i] = nx[i];
                if constexpr (RES) vr[i] = nr[i];
            }
        }
        row += groups;
    } while (AHEAD && row < n);
}

// Rows too long for registers: the row is read twice.
constexpr int kLongWaves = 16;

template <int DT>
__global__ __launch_bounds__(kLongWaves * 64) void norm_long(
    const typename Elem<DT>::raw *__restrict__ x, uint64_t x_stride, const typename Elem<DT>::raw *__restrict__ res,
    uint64_t res_stride, const typename Elem<DT>::raw *__restrict__ weight, uint32_t d, float eps,
    typename Elem<DT>::raw *__restrict__ h_out, typename Elem<DT>::raw *__restrict__ y_out, uint8_t *__restrict__ q,
    uint64_t q_stride, uint8_t *__restrict__ q_scale, uint64_t scale_stride, float *__restrict__ rstd_out)
{
    __shared__ float part[kLongWaves];
    const uint64_t row = blockIdx.x;
    const uint32_t step = kLongWaves * 64u * 8u;
    float rstd = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        float sum = 0.0f;
        for (uint32_t c0 = 0; c0 < d; c0 += step) {  // all lanes, for put_group's maximum
            const uint32_t c = c0 + threadIdx.x * 8u;
            const typename Elem<DT>::vec8 vx = load8<DT>(x + row * x_stride, c, d);
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = Elem<DT>::get(vx[e]);
            if (res) {
                const typename Elem<DT>::vec8 vr = load8<DT>(res + row * res_stride, c, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] += Elem<DT>::get(vr[e]);
            }
            if (pass == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(h[e], h[e], sum);
            } else {
                if (h_out && c < d) store8<DT>(h_out + row * d, c, d, h);
                const typename Elem<DT>::vec8 w = load8<DT>(weight, c, d);
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = h[e] * rstd * Elem<DT>::get(w[e]);
                if (y_out && c < d) store8<DT>(y_out + row * d, c, d, y);
                if (q) put_group(y, c, d, q + row * q_stride, q_scale + row * scale_stride);
            }
        }
        if (pass == 0) {
            sum = row_sum<kLongWaves>(sum, part);
            rstd = rsqrtf(sum / (float)d + eps);
            if (rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
        }
    }
}

template <int DT, int W, int IT, bool RES>
void norm_launch(const NormArgs &a)
{
    typedef typename Elem<DT>::raw R;
    uint64_t blocks = W == 1 ? div_up(a.n, 4) : a.n;
    const uint64_t stay = kAheadWaves / (W == 1 ? 4 : W);
    if (kAhead<DT, IT, RES> && blocks > stay) blocks = stay;
    norm_rows<DT, W, IT, RES><<<(uint32_t)blocks, W == 1 ? 256 : W * 64, 0, a.stream>>>(
        (const R *)a.x, a.x_stride, (const R *)a.residual, a.residual_stride, (const R *)a.weight, (uint32_t)a.n,
        (uint32_t)a.d, a.eps, (R *)a.h, (R *)a.y, a.q, a.q_stride, a.q_scale, a.scale_stride, a.rstd);
}

template <int DT, bool RES>
hipError_t norm_of(const NormArgs &a)
{
    typedef typename Elem<DT>::raw R;
    const bool few = a.n <= 512;  // rows for two workgroups per compute unit at most: more waves per row
    if (a.d <= 512) norm_launch<DT, 1, 1, RES>(a);
    else if (a.d <= 1024) norm_launch<DT, 1, 2, RES>(a);
    else if (a.d <= 2048) norm_launch<DT, 4, 1, RES>(a);
    else if (a.d <= 4096) few ? norm_launch<DT, 8, 1, RES>(a) : norm_launch<DT, 4, 2, RES>(a);
    else if (a.d <= 8192) few ? norm_launch<DT, 16, 1, RES>(a) : norm_launch<DT, 8, 2, RES>(a);
    else if (a.d <= 16384) norm_launch<DT, 16, 2, RES>(a);
    else if (a.d <= 24576) norm_launch<DT, 16, 3, RES>(a);
    else if (a.d <= 32768) norm_launch<DT, 16, 4, RES>(a);
    else
        norm_long<DT><<<(uint32_t)a.n, kLongWaves * 64, 0, a.stream>>>(
            (const R *)a.x, a.x_stride, (const R *)a.residual, a.residual_stride, (const R *)a.weight, (uint32_t)a.d,
            a.eps, (R *)a.h, (R *)a.y, a.q, a.q_stride, a.q_scale, a.scale_stride, a.rstd);
    return hipGetLastError();
}

template <int DT>
hipError_t norm_type(const NormArgs &a)
{
    return a.residual ? norm_of<DT, true>(a) : norm_of<DT, false>(a);
}

// -------------------------------------------------------------- gradient

constexpr uint32_t kGradBlocks = 512;  // workgroups, each with its own rows and its own sum for dw

// Group g of W waves takes rows g, g + groups, ...; dw's sum over them goes
// to partial row g. Bound by memory: 8,192 bf16 rows of 4,096 with a residual
// take 50 us here and 5 for the sum of the partial rows, 4.9 TB/s (a copy: 5.0).
//
// Not so at two ends. 16 waves a row have 128 registers a lane, of which dw's
// sums take 8 IT: up to 24,576 columns 8 of them spill in bf16 and 214 in 32
// bits, up to 32,768 there are 173, 379 and, in fp16, 78. 4,096 rows of 24,576
// take 173 us in bf16 and 365 in 32 bits (3.5 and 3.3 TB/s), 2,048 of 32,768
// 379 and 406 (1.1 and 2.0 TB/s). And up to 512 rows have a partial row each,
// written and read again: 512 x 4,096 in bf16 take 11 us, 682 x 24,576 46.
template <int DT, int W, int IT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_grad_rows(
    const typename Elem<DT>::raw *__restrict__ dy, uint64_t dy_stride, const typename Elem<DT>::raw *__restrict__ x,
    uint64_t x_stride, const float *__restrict__ rstd, const typename Elem<DT>::raw *__restrict__ weight,
    const typename Elem<DT>::raw *__restrict__ dres, uint64_t dres_stride, uint32_t n, uint32_t d,
    typename Elem<DT>::raw *__restrict__ dx, float *__restrict__ partial)
{
    __shared__ float part[2][W];
    const uint32_t groups = W == 1 ? gridDim.x * 4u : gridDim.x;
    const uint32_t g = W == 1 ? blockIdx.x * 4u + (threadIdx.x >> 6) : blockIdx.x;
    const uint32_t lane = W == 1 ? threadIdx.x & 63u : threadIdx.x;
    typename Elem<DT>::vec8 w[IT];
    float dw[IT][8];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        w[i] = load8<DT>(weight, (i * W * 64u + lane) * 8u, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    int flip = 0;
    for (uint32_t row = g; row < n; row += groups) {
        const float rs = rstd[row];
        typename Elem<DT>::vec8 vy[IT], vx[IT], vr[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t c = (i * W * 64u + lane) * 8u;
            vy[i] = load8<DT>(dy + row * dy_stride, c, d);
            vx[i] = load8<DT>(x + row * x_stride, c, d);
            if (dres) vr[i] = load8<DT>(dres + row * dres_stride, c, d);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const bool in = (i * W * 64u + lane) * 8u < d;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float hat = Elem<DT>::get(vx[i][e]) * rs, y = Elem<DT>::get(vy[i][e]);
                if (in) dw[i][e] = fmaf(y, hat, dw[i][e]);
                if (in) sum = fmaf(y * Elem<DT>::get(w[i][e]), hat, sum);
            }
        }
        sum = row_sum<W>(sum, part[flip]);  // two places in turn: a barrier a row
        flip ^= 1;
        const float mean = sum / (float)d;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t c = (i * W * 64u + lane) * 8u;
            if (c >= d) continue;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float hat = Elem<DT>::get(vx[i][e]) * rs;
                o[e] = rs * (Elem<DT>::get(vy[i][e]) * Elem<DT>::get(w[i][e]) - hat * mean);
                if (dres) o[e] += Elem<DT>::get(vr[i][e]);
            }
            store8<DT>(dx + (uint64_t)row * d, c, d, o);
        }
    }
    if (partial) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t c = (i * W * 64u + lane) * 8u;
            if (c < d) store8<kF32>(partial + (uint64_t)g * d, c, d, dw[i]);
        }
    }
}

// Rows too long for registers, from row `first` on: dx alone, the row read twice.
template <int DT>
__global__ __launch_bounds__(kLongWaves * 64) void norm_grad_long(
    const typename Elem<DT>::raw *__restrict__ dy, uint64_t dy_stride, const typename Elem<DT>::raw *__restrict__ x,
    uint64_t x_stride, const float *__restrict__ rstd, const typename Elem<DT>::raw *__restrict__ weight,
    const typename Elem<DT>::raw *__restrict__ dres, uint64_t dres_stride, uint64_t first, uint32_t d,
    typename Elem<DT>::raw *__restrict__ dx)
{
    __shared__ float part[kLongWaves];
    const uint64_t row = first + blockIdx.x;
    const float rs = rstd[row];
    float mean = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        float sum = 0.0f;
        for (uint32_t c = threadIdx.x * 8u; c < d; c += kLongWaves * 64u * 8u) {
            const typename Elem<DT>::vec8 vy = load8<DT>(dy + row * dy_stride, c, d);
            const typename Elem<DT>::vec8 vx = load8<DT>(x + row * x_stride, c, d);
            const typename Elem<DT>::vec8 vw = load8<DT>(weight, c, d);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float hat = Elem<DT>::get(vx[e]) * rs, gg = Elem<DT>::get(vy[e]) * Elem<DT>::get(vw[e]);
                if (c + e < d) sum = fmaf(gg, hat, sum);
                o[e] = rs * (gg - hat * mean);
            }
            if (pass == 1) {
                if (dres) {
                    const typename Elem<DT>::vec8 vr = load8<DT>(dres + row * dres_stride, c, d);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += Elem<DT>::get(vr[e]);
                }
                store8<DT>(dx + row * d, c, d, o);
            }
        }
        if (pass == 0) mean = row_sum<kLongWaves>(sum, part) / (float)d;
    }
}

// The long rows' partial sums of dw: blockIdx.y takes every gridDim.y-th row.
template <int DT>
__global__ __launch_bounds__(256) void norm_grad_long_dw(const typename Elem<DT>::raw *__restrict__ dy,
                                                         uint64_t dy_stride,
                                                         const typename Elem<DT>::raw *__restrict__ x,
                                                         uint64_t x_stride, const float *__restrict__ rstd, uint32_t n,
                                                         uint32_t d, float *__restrict__ partial)
{
    const uint32_t c = (blockIdx.x * 256u + threadIdx.x) * 8u;
    if (c >= d) return;
    float dw[8] = {};
    for (uint32_t row = blockIdx.y; row < n; row += gridDim.y) {
        const typename Elem<DT>::vec8 vy = load8<DT>(dy + row * dy_stride, c, d);
        const typename Elem<DT>::vec8 vx = load8<DT>(x + row * x_stride, c, d);
        const float rs = rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(Elem<DT>::get(vy[e]), Elem<DT>::get(vx[e]) * rs, dw[e]);
    }
    store8<kF32>(partial + (uint64_t)blockIdx.y * d, c, d, dw);
}

// dw = the sum of the partial rows: 32 columns per workgroup (workgroup 0 has
// those from 32 first on), 32 threads a column, joined in a fixed order.
__global__ __launch_bounds__(1024) void sum_partials(const float *__restrict__ partial, uint32_t count,
                                                     uint32_t first, uint32_t d, float *__restrict__ dw)
{
    __shared__ float sums[32][33];
    const uint32_t lane = threadIdx.x & 31u, g = threadIdx.x >> 5;
    const uint32_t c = (first + blockIdx.x) * 32u + lane;
    float s = 0.0f;
    if (c < d) {
#pragma unroll 8
        for (uint32_t p = g; p < count; p += 32) s += partial[(uint64_t)p * d + c];
    }
    sums[g][lane] = s;
    __syncthreads();
    if (g == 0 && c < d) {
        s = 0.0f;
#pragma unroll
        for (int q = 0; q < 32; ++q) s += sums[q][lane];
        dw[c] = s;
    }
}

__global__ void zero_floats(float *p, uint64_t n)
{
    const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

constexpr uint64_t kGradRegColumns = 32768;  // longest row kept in registers

uint32_t grad_blocks(uint64_t n, uint64_t d)
{
    const uint64_t need = d <= 1024 ? div_up(n, 4) : n;
    return (uint32_t)(need < kGradBlocks ? need : kGradBlocks);
}

uint32_t grad_partials(uint64_t n, uint64_t d) { return grad_blocks(n, d) * (d <= 1024 ? 4u : 1u); }

template <int DT, int W, int IT>
void grad_launch(const NormGradArgs &a)
{
    typedef typename Elem<DT>::raw R;
    norm_grad_rows<DT, W, IT><<<grad_blocks(a.n, a.d), W == 1 ? 256 : W * 64, 0, a.stream>>>(
        (const R *)a.dy, a.dy_stride, (const R *)a.x, a.x_stride, a.rstd, (const R *)a.weight, (const R *)a.dres,
        a.dres_stride, (uint32_t)a.n, (uint32_t)a.d, (R *)a.dx, a.dw ? (float *)a.workspace : nullptr);
}

template <int DT>
hipError_t grad_of(const NormGradArgs &a)
{
    typedef typename Elem<DT>::raw R;
    if (a.n == 0) {
        if (a.dw) zero_floats<<<(uint32_t)div_up(a.d, 256), 256, 0, a.stream>>>(a.dw, a.d);
        return hipGetLastError();
    }
    if (a.d <= 512) grad_launch<DT, 1, 1>(a);
    else if (a.d <= 1024) grad_launch<DT, 1, 2>(a);
    else if (a.d <= 2048) grad_launch<DT, 4, 1>(a);
    else if (a.d <= 4096) grad_launch<DT, 8, 1>(a);
    else if (a.d <= 8192) grad_launch<DT, 8, 2>(a);
    else if (a.d <= 16384) grad_launch<DT, 16, 2>(a);
    else if (a.d <= 24576) grad_launch<DT, 16, 3>(a);
    else if (a.d <= kGradRegColumns) grad_launch<DT, 16, 4>(a);
    else {
        for (uint64_t row = 0; row < a.n; row += kMaxRows)
            norm_grad_long<DT><<<(uint32_t)(a.n - row < kMaxRows ? a.n - row : kMaxRows), kLongWaves * 64, 0, a.stream>>>(
                (const R *)a.dy, a.dy_stride, (const R *)a.x, a.x_stride, a.rstd, (const R *)a.weight, (const R *)a.dres,
                a.dres_stride, row, (uint32_t)a.d, (R *)a.dx);
        if (a.dw)
            norm_grad_long_dw<DT><<<dim3((uint32_t)div_up(a.d, 2048), grad_partials(a.n, a.d)), 256, 0, a.stream>>>(
                (const R *)a.dy, a.dy_stride, (const R *)a.x, a.x_stride, a.rstd, (uint32_t)a.n, (uint32_t)a.d,
                (float *)a.workspace);
    }
    if (a.dw) {
        const uint64_t blocks = div_up(a.d, 32);
        for (uint64_t b = 0; b < blocks; b += kMaxRows)
            sum_partials<<<(uint32_t)(blocks - b < kMaxRows ? blocks - b : kMaxRows), 1024, 0, a.stream>>>(
                (const float *)a.workspace, grad_partials(a.n, a.d), (uint32_t)b, (uint32_t)a.d, a.dw);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t rms_norm(const NormArgs &args)
{
    NormArgs a = args;
    const uint64_t es = dtype_bytes(a.dtype);
    for (uint64_t left = args.n; left > 0;) {
        a.n = left < kMaxRows ? left : kMaxRows;
        const hipError_t e = a.dtype == kF32    ? norm_type<kF32>(a)
                             : a.dtype == kBF16 ? norm_type<kBF16>(a)
                                                : norm_type<kF16>(a);
        if (e != hipSuccess) return e;
        left -= a.n;
        a.x = (const uint8_t *)a.x + a.n * a.x_stride * es;
        if (a.residual) a.residual = (const uint8_t *)a.residual + a.n * a.residual_stride * es;
        if (a.h) a.h = (uint8_t *)a.h + a.n * a.d * es;
        if (a.y) a.y = (uint8_t *)a.y + a.n * a.d * es;
        if (a.q) a.q += a.n * a.q_stride;
        if (a.q_scale) a.q_scale += a.n * a.scale_stride;
        if (a.rstd) a.rstd += a.n;
    }
    return hipSuccess;
}

uint64_t rms_norm_grad_workspace_bytes(uint64_t n, uint64_t d) { return 4ull * grad_partials(n, d) * d; }

hipError_t rms_norm_grad(const NormGradArgs &a)
{
    switch (a.dtype) {
    case kF32: return grad_of<kF32>(a);
    case kBF16: return grad_of<kBF16>(a);
    default: return grad_of<kF16>(a);
    }
}

}  // namespace cpk
