// cp_linear.hip - cp_linear's product: y[m][n] from rows of x and rows of w.
#include "cp_linear_tile.h"

namespace cpk {

namespace {

struct RowsParams {
    const void *x, *w;
    uint64_t x_stride, w_stride;  // bytes
    uint32_t m, n, k;
    uint32_t tiles, batches_per_wave;
    float *part;  // the splits' sums, [split][m][n], where k is split over workgroups
    Epilogue e;
};

template <int DT>
__device__ __forceinline__ f32x4 multiply16(i32x4 w, i32x4 x, f32x4 c)
{
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c,
                                                       0, 0, 0);
    else if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0,
                                                      0, 0);
    else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(w[e]), __int_as_float(x[e]), c, 0, 0, 0);
        return c;
    }
}

constexpr int kRowWaves = 8, kBatch = 8;                // waves of a workgroup; 64-byte pieces of a row read together
constexpr uint32_t kBatchBytes = kBatch * 64;

// Few rows of x: w is read once, straight into registers, and bounds the time:
// 8 x 4,096 x 24,576 in bf16 takes 41 us, 4.9 TB/s (a copy: 5.1), one row 37, 16
// rows 49, as each of the 256 workgroups reads all of x from L2. (The tiles take
// 51 for anything up to 64 rows. With a second fragment of x here 17 rows took
// 55, 32 rows 69; with four, 64 rows 111.) A workgroup has 16 columns of y; its waves take runs of
// batches of K (512 bytes of each row of w: a lane has row l % 16 and the
// 16-byte chunks l / 16 + 4 j of it) and add their sums through LDS. The next
// batch is read while one is multiplied: 16 KiB of w in flight for each wave.
template <int DT>
__global__ __launch_bounds__(kRowWaves * 64, 2) void linear_rows(RowsParams p)
{
    constexpr uint32_t ES = dtype_bytes(DT), EPC = 16 / ES;
    __shared__ float sums[kRowWaves][16][17];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 15u, g = lane >> 4;
    const uint32_t split = blockIdx.x / p.tiles, n0 = (blockIdx.x - split * p.tiles) * 16;
    const uint32_t batches = (p.k * ES + kBatchBytes - 1) / kBatchBytes;
    const uint32_t first = (split * kRowWaves + wave) * p.batches_per_wave;
    const uint32_t b0 = first < batches ? first : batches;
    const uint32_t b1 = b0 + p.batches_per_wave < batches ? b0 + p.batches_per_wave : batches;
    const uint32_t whole = p.k * ES / kBatchBytes;  // batches that do not reach past k
    // (rows past the end: the last one)
    const uint8_t *const pw = (const uint8_t *)p.w + (uint64_t)(n0 + r < p.n ? n0 + r : p.n - 1) * p.w_stride + g * 16;
    const uint8_t *const px = (const uint8_t *)p.x + (uint64_t)(r < p.m ? r : p.m - 1) * p.x_stride + g * 16;
    f32x4 acc = (f32x4)0.0f;

    const auto load = [&](const uint8_t *row, uint32_t batch, i32x4 *v) {
        const uint8_t *const at = row + (uint64_t)batch * kBatchBytes;
        if (batch < whole) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) v[j] = *reinterpret_cast<const unaligned_i32x4 *>(at + j * 64);
        } else {
            typedef typename Elem<DT>::raw raw;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const uint32_t c = batch * (kBatchBytes / ES) + j * 4 * EPC + g * EPC;
                v[j] = i32x4{0, 0, 0, 0};
                if (c + EPC <= p.k) {
                    v[j] = *reinterpret_cast<const unaligned_i32x4 *>(at + j * 64);
                } else if (c < p.k) {
                    raw e[EPC] = {};
#pragma unroll
                    for (uint32_t q = 0; q < EPC; ++q)
                        if (c + q < p.k) e[q] = ((const raw *)(at + j * 64))[q];
                    __builtin_memcpy(&v[j], e, 16);
                }
            }
        }
    };
    struct Batch {
        i32x4 w[kBatch], x[kBatch];
    };
    const auto turn = [&](uint32_t b, Batch &now, Batch &next) {
        if (b >= b1) return;
        if (b + 1 < b1) {
            load(pw, b + 1, next.w);
            load(px, b + 1, next.x);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) acc = multiply16<DT>(now.w[j], now.x[j], acc);
    };
    Batch u, v;
    if (b0 < b1) {
        load(pw, b0, u.w);
        load(px, b0, u.x);
    }
    for (uint32_t b = b0; b < b1; b += 2) {
        turn(b, u, v);
        turn(b + 1, v, u);
    }
    // lane l has row l % 16, columns 4 (l / 16) + e
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[wave][r][4 * g + e] = acc[e];
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const uint32_t row = threadIdx.x >> 1, c = (threadIdx.x & 1u) * 8;
    if (row >= p.m || n0 + c >= p.n) return;
    float f[8] = {};
#pragma unroll
    for (int q = 0; q < kRowWaves; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += sums[q][row][c + e];
    if (p.part) store8<kF32>(p.part + ((uint64_t)split * p.m + row) * p.n, n0 + c, p.n, f);
    else {
        float bias[8];
        bias8<DT>(p.e, n0 + c, p.n, bias);
        finish8<DT>(p.e, mask_of(p.e.drop), row, n0 + c, p.n, f, bias, residual8<DT>(p.e, row, n0 + c, p.n));
    }
}

constexpr uint64_t kFewRows = 16;  // a fragment of x

// Splits of K and a wave's batches for few rows.
Cut rows_cut(uint64_t n, uint64_t k, int dtype)
{
    const uint64_t batches = div_up(k * dtype_bytes(dtype), kBatchBytes), tiles = div_up(n, 16);
    uint64_t splits = 1;
    while (tiles * splits < 128 && batches >= 2 * splits * kRowWaves * 2) splits *= 2;
    const uint64_t per = div_up(batches, splits * kRowWaves);
    return Cut{0, (uint32_t)div_up(batches, per * kRowWaves), (uint32_t)per};
}

template <int DT>
hipError_t launch_rows(const LinearArgs &g)
{
    const Cut c = rows_cut(g.n, g.k, DT);
    RowsParams p{};
    p.x = g.a;
    p.w = g.b;
    p.x_stride = g.a_stride * dtype_bytes(DT);
    p.w_stride = g.b_stride * dtype_bytes(DT);
    p.m = (uint32_t)g.m;
    p.n = (uint32_t)g.n;
    p.k = (uint32_t)g.k;
    p.tiles = (uint32_t)div_up(g.n, 16);
    p.batches_per_wave = c.steps_per_split;
    p.part = c.splits > 1 ? (float *)g.workspace : nullptr;
    p.e = g.e;
    const uint32_t blocks = p.tiles * c.splits;
    linear_rows<DT><<<blocks, kRowWaves * 64, 0, g.stream>>>(p);
    if (c.splits > 1) return join<DT, DT>(g, c.splits);
    return hipGetLastError();
}

}  // namespace

uint64_t linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype)
{
    uint64_t most = m <= kFewRows ? workspace_of(rows_cut(n, k, dtype), m, n) : 0;
    for (Rows rows : {kWhole, kOdd, kShort}) {
        const uint64_t bytes = workspace_of(cut_of(m, n, k, dtype, rows), m, n);
        most = bytes > most ? bytes : most;
    }
    return most;
}

template <int DT>
static hipError_t rows_by_rows(const LinearArgs &a)
{
    if (a.m <= kFewRows && a.k > 0) return launch_rows<DT>(a);
    return launch_linear<DT, false, false, DT>(a);
}

hipError_t linear_rows_by_rows(const LinearArgs &a)
{
    if (a.dtype == kBF16) return rows_by_rows<kBF16>(a);
    if (a.dtype == kF16) return rows_by_rows<kF16>(a);
    return rows_by_rows<kF32>(a);
}

}  // namespace cpk
