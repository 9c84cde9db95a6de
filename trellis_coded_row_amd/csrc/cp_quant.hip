// cp_quant.hip - the 8-bit form of a matrix, and of its transpose.
//
// A group of 128 values (or a block of 128 x 128) with largest finite
// magnitude A is stored as e4m3 values x / 2^e and the exponent e, the least
// with A / 2^e <= 448.
//
// Bound by memory: the matrix is read once, in tiles of 128 x 128 that hold
// whole groups of both directions, and both outputs are written from it.
// 4,096 x 24,576 bf16 in blocks, both ways: 81 to 87 us, 4.6 to 4.9 TB/s (a copy:
// 5.0 to 5.2). 1,000 x 2,050 (136 tiles, fewer than compute units) is a tile's
// latency: 6.7 us, where 256 threads a tile took 8.3 (a wave alone on its SIMD
// unit issues slowly) and testing each value for what is not finite, not the
// maxima, 9.8.
#include <type_traits>

#include "cp_ops_internal.h"

namespace cpk {

namespace {

constexpr uint32_t kTile = 128;
constexpr uint32_t kThreads = 512, kWaves = kThreads / 64;
constexpr int kRows = 4;  // of a thread

// 8 bytes of a row, or those of them before its end (left = bytes to there).
__device__ __forceinline__ void put8(uint8_t *p, u32x2 v, uint32_t left)
{
    if (left >= 8) {
        *reinterpret_cast<u32x2 *>(p) = v;
    } else {
        for (uint32_t e = 0; e < left; ++e) p[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3u)));
    }
}

// One tile per workgroup of 512 threads. Thread t has rows 4 (t / 16) + i and
// columns 8 (t % 16) + e, i < 4, e < 8: 16 neighbouring lanes hold a row's 128
// columns (a row of lanes, so its maximum needs no LDS), and a thread holds
// 4 or 8 values that follow one another in either direction.
//
// The transposed tile goes through LDS, 128 rows (the tile's columns) of 128
// bytes, in pieces of 8 bytes; piece p of row c stands at p ^ (c / 8 % 16),
// so that the 16 lanes that store together, with columns 8 apart, hit
// different banks.
template <int DT, bool BLOCKS, bool TRANS>
__global__ __launch_bounds__(kThreads) void quantize_tile(const typename Elem<DT>::raw *__restrict__ x, uint32_t n,
                                                     uint32_t d, uint64_t x_stride, uint32_t tiles_x,
                                                     uint8_t *__restrict__ q, uint64_t q_stride,
                                                     uint8_t *__restrict__ scale, uint64_t scale_stride,
                                                     uint8_t *__restrict__ qt, uint64_t qt_stride,
                                                     uint8_t *__restrict__ scale_t, uint64_t scale_t_stride)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[TRANS ? kTile * kTile : 16];
    __shared__ __attribute__((aligned(16))) uint32_t part[kWaves][kTile];
    const uint32_t tx = blockIdx.x % tiles_x, ty = blockIdx.x / tiles_x;
    const uint32_t cl = (threadIdx.x & 15u) * 8u, rl = (threadIdx.x >> 4) * kRows, wave = threadIdx.x >> 6;
    const uint32_t c0 = tx * kTile + cl, r0 = ty * kTile + rl;
    typename Elem<DT>::vec8 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (r0 + i < n) v[i] = load8<DT>(x + (r0 + i) * x_stride, c0, d);
        else v[i] = (typename Elem<DT>::raw)0;
    }
    // largest magnitudes: of each row's 8 columns and each column's 4 rows.
    // Where one of the thread's values is not finite, which its maxima then
    // are not either, it takes them again among those that are.
    uint32_t mr[kRows], mc[8];
    float fr[kRows], fc[8], most = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) fr[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) fc[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = __builtin_fabsf(Elem<DT>::get(v[i][e]));
            fr[i] = __builtin_elementwise_maximum(fr[i], f);
            if constexpr (TRANS && !BLOCKS) fc[e] = __builtin_elementwise_maximum(fc[e], f);
        }
        most = __builtin_elementwise_maximum(most, fr[i]);
        mr[i] = __float_as_uint(fr[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) mc[e] = __float_as_uint(fc[e]);
    const bool odd = !(most < __builtin_inff());
    if (odd) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mc[e] = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            mr[i] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = finite_bits(Elem<DT>::get(v[i][e]));
                mr[i] = mr[i] > b ? mr[i] : b;
                mc[e] = mc[e] > b ? mc[e] : b;
            }
        }
    }
    const auto four = [](auto check, float a, float b, float c, float d, float inv) {
        if constexpr (decltype(check)::value) return to_e4m3x4(a, b, c, d, inv);
        else return finite_to_e4m3x4(a, b, c, d, inv);
    };
    uint32_t byte_r[kRows], byte_c[8];
    if constexpr (BLOCKS) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = m > mr[i] ? m : mr[i];
        m = max_of_16(m);
        uint32_t o = (uint32_t)__shfl_xor((int)m, 16, 64);
        m = m > o ? m : o;
        o = (uint32_t)__shfl_xor((int)m, 32, 64);
        m = m > o ? m : o;
        if ((threadIdx.x & 63u) == 0) part[wave][0] = m;
        __syncthreads();
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) m = m > part[w][0] ? m : part[w][0];
        byte_r[0] = scale_byte(m);
        if (threadIdx.x == 0) {
            scale[ty * scale_stride + tx] = (uint8_t)byte_r[0];
            if constexpr (TRANS) scale_t[tx * scale_t_stride + ty] = (uint8_t)byte_r[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            byte_r[i] = scale_byte(max_of_16(mr[i]));
            if ((threadIdx.x & 15u) == 0 && r0 + i < n) scale[(r0 + i) * scale_stride + tx] = (uint8_t)byte_r[i];
        }
        if constexpr (TRANS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t o = (uint32_t)__shfl_xor((int)mc[e], 16, 64);
                mc[e] = mc[e] > o ? mc[e] : o;
                o = (uint32_t)__shfl_xor((int)mc[e], 32, 64);
                mc[e] = mc[e] > o ? mc[e] : o;
                if ((threadIdx.x & 63u) < 16) part[wave][cl + e] = mc[e];
            }
            __syncthreads();
            uint32_t m[8] = {};
#pragma unroll
            for (uint32_t w = 0; w < kWaves; ++w) {
#pragma unroll
                for (int e = 0; e < 8; ++e) m[e] = m[e] > part[w][cl + e] ? m[e] : part[w][cl + e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) byte_c[e] = scale_byte(m[e]);
            if (threadIdx.x < 16) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c0 + e < d) scale_t[(c0 + e) * scale_t_stride + ty] = (uint8_t)byte_c[e];
            }
        }
    }
    const uint32_t left = c0 < d ? d - c0 : 0;
    const auto convert = [&](auto check) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float inv = inverse_scale(byte_r[BLOCKS ? 0 : i]);
            u32x2 o;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o[h] = four(check, Elem<DT>::get(v[i][4 * h]), Elem<DT>::get(v[i][4 * h + 1]),
                            Elem<DT>::get(v[i][4 * h + 2]), Elem<DT>::get(v[i][4 * h + 3]), inv);
            if (r0 + i < n) put8(q + (r0 + i) * q_stride + c0, o, left);
        }
        if constexpr (TRANS) {
            // column e's 4 rows: half a piece of LDS row cl + e
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float inv = inverse_scale(BLOCKS ? byte_r[0] : byte_c[e]);
                const uint32_t o = four(check, Elem<DT>::get(v[0][e]), Elem<DT>::get(v[1][e]), Elem<DT>::get(v[2][e]),
                                        Elem<DT>::get(v[3][e]), inv);
                const uint32_t piece = (rl >> 3) ^ (cl >> 3);
                *reinterpret_cast<uint32_t *>(lds + (cl + e) * kTile + piece * 8u + (rl & 4u)) = o;
            }
        }
    };
    if (odd) convert(std::true_type{});
    else convert(std::false_type{});
    if constexpr (TRANS) {
        __syncthreads();
        // 8 lanes write an output row's 128 bytes, 16 at a time
#pragma unroll
        for (uint32_t i = 0; i < kTile * 8 / kThreads; ++i) {
            const uint32_t c = i * (kThreads / 8) + (threadIdx.x >> 3), p = (threadIdx.x & 7u) * 2u, sw = (c >> 3) & 15u;
            if (tx * kTile + c >= d) continue;
            const u32x2 a = *reinterpret_cast<const u32x2 *>(lds + c * kTile + (p ^ sw) * 8u);
            const u32x2 b = *reinterpret_cast<const u32x2 *>(lds + c * kTile + ((p + 1) ^ sw) * 8u);
            uint8_t *const to = qt + (uint64_t)(tx * kTile + c) * qt_stride + ty * kTile + p * 8u;
            const uint32_t at = ty * kTile + p * 8u;
            if (at + 16 <= n) {
                u32x4 o;
                o[0] = a[0];
                o[1] = a[1];
                o[2] = b[0];
                o[3] = b[1];
                *reinterpret_cast<u32x4 *>(to) = o;
            } else if (at < n) {
                put8(to, a, n - at);
                if (at + 8 < n) put8(to + 8, b, n - at - 8);
            }
        }
    }
}

// Tiles of one launch, at most: its threads are counted in 32 bits, and a
// launch of more than 2^32 runs the remainder alone, without an error.
constexpr uint64_t kLaunchTiles = 1ull << 22;
static_assert(kLaunchTiles * kThreads < (1ull << 32), "");

template <int DT, bool BLOCKS, bool TRANS>
hipError_t launch(const QuantArgs &a)
{
    const uint64_t tiles_x = div_up(a.d, kTile), tiles_y = div_up(a.n, kTile);
    const uint64_t step_x = tiles_x < kLaunchTiles ? tiles_x : kLaunchTiles, step_y = kLaunchTiles / step_x;
    for (uint64_t y = 0; y < tiles_y; y += step_y) {
        const uint64_t r = y * kTile, ny = tiles_y - y < step_y ? tiles_y - y : step_y;
        const uint64_t n = a.n - r < ny * kTile ? a.n - r : ny * kTile;
        for (uint64_t x = 0; x < tiles_x; x += step_x) {
            const uint64_t c = x * kTile, nx = tiles_x - x < step_x ? tiles_x - x : step_x;
            const uint64_t d = a.d - c < nx * kTile ? a.d - c : nx * kTile;
            quantize_tile<DT, BLOCKS, TRANS><<<(uint32_t)(ny * nx), kThreads, 0, a.stream>>>(
                (const typename Elem<DT>::raw *)a.x + r * a.x_stride + c, (uint32_t)n, (uint32_t)d, a.x_stride,
                (uint32_t)nx, a.q + r * a.q_stride + c, a.q_stride, a.scale + (BLOCKS ? y : r) * a.scale_stride + x,
                a.scale_stride, TRANS ? a.qt + c * a.qt_stride + r : nullptr, a.qt_stride,
                TRANS ? a.scale_t + (BLOCKS ? x : c) * a.scale_t_stride + y : nullptr, a.scale_t_stride);
        }
    }
    return hipGetLastError();
}

template <int DT>
hipError_t quant_of(const QuantArgs &a)
{
    if (a.blocks) return a.qt ? launch<DT, true, true>(a) : launch<DT, true, false>(a);
    return a.qt ? launch<DT, false, true>(a) : launch<DT, false, false>(a);
}

}  // namespace

hipError_t quantize_fp8(const QuantArgs &a)
{
    switch (a.dtype) {
    case kF32: return quant_of<kF32>(a);
    case kBF16: return quant_of<kBF16>(a);
    default: return quant_of<kF16>(a);
    }
}

}  // namespace cpk
