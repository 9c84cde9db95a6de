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
// 8 x 4,096 x 24,576 in bf16 takes 40.5 us, 5.0 TB/s (a copy: 5.1), one row 37, 16
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
    // what the epilogue reads, by the threads that will write 8 values of y each
    const uint32_t row = threadIdx.x >> 1, c = (threadIdx.x & 1u) * 8;
    const bool writes = row < p.m && n0 + c < p.n;
    float bias[8];
    typename Elem<DT>::vec8 residual = {};
    Mask mask{};
    if (writes && !p.part) {
        bias8<DT>(p.e, n0 + c, p.n, bias);
        residual = residual8<DT>(p.e, row, n0 + c, p.n);
        mask = mask_of(p.e.drop);
    }

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
    if (!writes) return;
    float f[8] = {};
#pragma unroll
    for (int q = 0; q < kRowWaves; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += sums[q][row][c + e];
    if (p.part) store8<kF32>(p.part + ((uint64_t)split * p.m + row) * p.n, n0 + c, p.n, f);
    else finish8<DT>(p.e, mask, row, n0 + c, p.n, f, bias, residual);
}

// Up to four rows of x, where 16 columns a workgroup would leave compute units
// idle: the 4 x 4 instruction, whose 16 blocks take 16 neighbouring chunks of
// K. A workgroup has 8 columns; its waves go by the four columns and the quarter of
// K that they take. 1 x 1,024 x 4,096 in bf16: 5.6 us, call
// included (with 16 columns 7.2).
template <int DT>
__device__ __forceinline__ f32x4 multiply4(i32x4 w, i32x4 x, f32x4 c)
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_4x4x1f32(__int_as_float(w[e]), __int_as_float(x[e]), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const i32x2 a = {w[2 * e], w[2 * e + 1]}, b = {x[2 * e], x[2 * e + 1]};
            if constexpr (DT == kBF16)
                c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(i16x4, a), __builtin_bit_cast(i16x4, b), c, 0, 0, 0);
            else
                c = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0, 0);
        }
    }
    return c;
}

constexpr int kFourBatch = 4;                         // pieces of 256 bytes of a row that are read together
constexpr uint32_t kFourBatchBytes = kFourBatch * 256;

template <int DT>
__global__ __launch_bounds__(kRowWaves * 64, 2) void linear_four_rows(RowsParams p)
{
    constexpr uint32_t ES = dtype_bytes(DT), EPC = 16 / ES;
    __shared__ float sums[kRowWaves][4][4];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 3u, g = lane >> 2, half = wave & 1u, slice = wave >> 1;
    const uint32_t split = blockIdx.x / p.tiles, n0 = (blockIdx.x - split * p.tiles) * 8, column = n0 + half * 4 + r;
    const uint32_t batches = (p.k * ES + kFourBatchBytes - 1) / kFourBatchBytes;
    const uint32_t first = (split * (kRowWaves / 2) + slice) * p.batches_per_wave;
    const uint32_t b0 = first < batches ? first : batches;
    const uint32_t b1 = b0 + p.batches_per_wave < batches ? b0 + p.batches_per_wave : batches;
    // (rows past the end: the last one)
    const uint8_t *const pw = (const uint8_t *)p.w + (uint64_t)(column < p.n ? column : p.n - 1) * p.w_stride;
    const uint8_t *const px = (const uint8_t *)p.x + (uint64_t)(r < p.m ? r : p.m - 1) * p.x_stride;
    const bool writes = threadIdx.x < p.m;  // 8 values of a row of y
    float bias[8];
    typename Elem<DT>::vec8 residual = {};
    Mask mask{};
    if (writes && !p.part) {
        bias8<DT>(p.e, n0, p.n, bias);
        residual = residual8<DT>(p.e, threadIdx.x, n0, p.n);
        mask = mask_of(p.e.drop);
    }
    const auto load = [&](const uint8_t *row, uint32_t batch, i32x4 *v) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kFourBatch; ++j) {
            const uint32_t c = batch * (kFourBatchBytes / ES) + j * 16 * EPC + g * EPC;
            const typename Elem<DT>::raw *const at = (const typename Elem<DT>::raw *)row + c;
            v[j] = i32x4{0, 0, 0, 0};
            if (c + EPC <= p.k) {
                v[j] = *reinterpret_cast<const unaligned_i32x4 *>(at);
            } else if (c < p.k) {
                typename Elem<DT>::raw e[EPC] = {};
#pragma unroll
                for (uint32_t q = 0; q < EPC; ++q)
                    if (c + q < p.k) e[q] = at[q];
                __builtin_memcpy(&v[j], e, 16);
            }
        }
    };
    f32x4 acc = (f32x4)0.0f;
    i32x4 w[2][kFourBatch], x[2][kFourBatch];
    if (b0 < b1) {
        load(pw, b0, w[0]);
        load(px, b0, x[0]);
    }
    const auto turn = [&](uint32_t b, i32x4 *wn, i32x4 *xn, i32x4 *wl, i32x4 *xl) __attribute__((always_inline)) {
        if (b >= b1) return;
        if (b + 1 < b1) {
            load(pw, b + 1, wl);
            load(px, b + 1, xl);
        }
#pragma unroll
        for (int j = 0; j < kFourBatch; ++j) acc = multiply4<DT>(wn[j], xn[j], acc);
    };
    for (uint32_t b = b0; b < b1; b += 2) {
        turn(b, w[0], x[0], w[1], x[1]);
        turn(b + 1, w[1], x[1], w[0], x[0]);
    }
    // lane l has row l % 4 of x, this wave's four columns, of block l / 4
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int over = 4; over < 64; over *= 2) acc[e] += __shfl_xor(acc[e], over, 64);
        if (lane < 4) sums[wave][r][e] = acc[e];
    }
    __syncthreads();
    if (!writes) return;
    float f[8] = {};
#pragma unroll
    for (int q = 0; q < kRowWaves; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[(q & 1) * 4 + e] += sums[q][threadIdx.x][e];
    if (p.part) store8<kF32>(p.part + ((uint64_t)split * p.m + threadIdx.x) * p.n, n0, p.n, f);
    else finish8<DT>(p.e, mask, threadIdx.x, n0, p.n, f, bias, residual);
}

constexpr uint64_t kFewRows = 16;  // a fragment of x

// Whether few rows go by four: 16 columns a workgroup would leave compute units idle.
bool by_four(uint64_t m, uint64_t n) { return m <= 4 && n <= 16 * 255; }

// Splits of K over workgroups and a wave's batches for few rows: a second launch
// that joins them pays where it brings more of the chip in, and where each wave
// keeps two batches (four of the shorter ones) to read ahead. us, with a limit of
// 1 (no splits), 64, 128 and 256 workgroups: 8 x 512 x 20,000 in bf16 22.8, 15.6,
// 12.3, 12.4, in f32 59, 35, 21.2, 17.0; 4 x 512 x 20,000 in f32 36.8, 36.9, 23.2,
// 16.0; 8 x 2,048 x 24,576 in bf16 37.2, 37.2, 37.3, 24.4; 8 x 1,024 x 24,576 36,
// 36, 22, 15. (So 256 would serve a long K better; 512 is no faster than it: 27.6
// for 8 x 2,048 x 24,576.) With one batch a wave and 256: 8 x 512 x 20,000 in bf16
// 10.7, but 1 x 1,024 x 4,096 7.6 where it takes 5.2.
Cut rows_cut(uint64_t m, uint64_t n, uint64_t k, int dtype)
{
    const bool four = by_four(m, n);
    const uint64_t batches = div_up(k * dtype_bytes(dtype), four ? kFourBatchBytes : kBatchBytes);
    const uint64_t tiles = div_up(n, four ? 8 : 16), waves = four ? kRowWaves / 2 : kRowWaves;
    uint64_t splits = 1;
    while (tiles * splits < 128 && batches >= 2 * splits * waves * (four ? 4 : 2)) splits *= 2;
    const uint64_t per = div_up(batches, splits * waves);
    return Cut{0, (uint32_t)div_up(batches, per * waves), (uint32_t)per};
}

template <int DT>
hipError_t launch_rows(const LinearArgs &g)
{
    const Cut c = rows_cut(g.m, g.n, g.k, DT);
    const bool four = by_four(g.m, g.n);
    RowsParams p{};
    p.x = g.a;
    p.w = g.b;
    p.x_stride = g.a_stride * dtype_bytes(DT);
    p.w_stride = g.b_stride * dtype_bytes(DT);
    p.m = (uint32_t)g.m;
    p.n = (uint32_t)g.n;
    p.k = (uint32_t)g.k;
    p.tiles = (uint32_t)div_up(g.n, four ? 8 : 16);
    p.batches_per_wave = c.steps_per_split;
    p.part = c.splits > 1 ? (float *)g.workspace : nullptr;
    p.e = g.e;
    const uint32_t blocks = p.tiles * c.splits;
    if (four) linear_four_rows<DT><<<blocks, kRowWaves * 64, 0, g.stream>>>(p);
    else linear_rows<DT><<<blocks, kRowWaves * 64, 0, g.stream>>>(p);
    if (c.splits > 1) return join<DT, DT>(g, c.splits);
    return hipGetLastError();
}

}  // namespace

uint64_t linear_tile_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype)
{
    uint64_t most = 0;
    for (Rows rows : {kWhole, kOdd, kShort}) {
        const uint64_t bytes = workspace_of(cut_of(m, n, k, dtype, rows), m, n);
        most = bytes > most ? bytes : most;
    }
    return most;
}

uint64_t linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype)
{
    return m <= kFewRows ? workspace_of(rows_cut(m, n, k, dtype), m, n) : linear_tile_workspace_bytes(m, n, k, dtype);
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
