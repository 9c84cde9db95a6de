// cp_gemm.hip - out[m][n] = sum over k of A[m][k] B[n][k] for e4m3 operands
// with an e8m0 scale for each 128 values of k.
//
// 16-bit outputs use the scaled matrix instruction of gfx950 (16 x 16 outputs,
// 128 values of k): lane l carries row l % 16 and 32 of its 128 values, and
// every lane of a row is given that row's e8m0 scale for the group, so the
// scales cost no arithmetic. Which 32 values a lane carries does not matter
// as long as both operands agree: here 16 from the group's first half and 16
// from the second. That instruction adds its products in groups of 8 of
// neighbouring k, each cut, toward zero, to a multiple of 2^(E - 13), E the
// largest sum of the factors' exponents among them (measured with P - P + p).
// A product of two 4-bit significands has 8 bits, so only products more than 6
// binades below the group's largest lose any: with normal operands the error is
// 1.5e-5 of the result's rms at any k, and 1.2% of the bf16 outputs round to
// the neighbour of the value that a 32-bit sum rounds to. At worst it is 7
// times 2^-13 of each group's largest product, 2^-10 of the sum of magnitudes,
// half a bf16 rounding.
//
// 32-bit outputs are not to lose that, so there each value times its scale
// is converted to bf16 (e4m3 has 4 significant bits: exact) on the way from
// LDS to the bf16 matrix instruction (measured: 1e-8 to 2e-7 of the result's
// rms, the 32-bit sum's own rounding), at half the rate and with the
// conversions beside it.
//
// Reached: 4,096 x 4,096 x 24,576 to bf16 in 300 us, 2.75 PFLOP/s, where the
// vendor library's product of the same operands with one scale for each takes
// 250 in turn with it; 4,096 x 24,576 x 4,096 to 32 bits in 790 us, 1.04 PFLOP/s
// (its product of operands widened before, with a 16-bit output: 490); 8 x 4,096 x
// 24,576 in 22.6 us, 4.5 TB/s (a copy: 5.0 to 5.2). A run of long products lowers
// the clock for some milliseconds after a pause: 300 is 320 to 450 there, 790 up
// to 1,100. These sizes fill the chip with whole rounds of the largest tile;
// others are 1.5 to 5 times as far from the library's rate (see cut_of).
//
// The operands are passed swapped (B's rows as the instruction's rows), so
// that a lane's four results are neighbours in an output row.
#include <type_traits>

#include "cp_ops_internal.h"

namespace cpk {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr uint32_t kStep = 128;              // values of k per step (one scale group)
constexpr uint32_t kInside = 0x7FFFFFFFu;    // bytes of a buffer: any offset within a tile
constexpr uint32_t kOutside = 0x80000000u;   // an offset past it: loads give zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t size = kInside)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)size, 0x00020000);
}

// The scales are byte S of sb and sa.
template <int S>
__device__ __forceinline__ f32x4 mfma(i32x8 b, i32x8 a, f32x4 c, int sb, int sa)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, S, sb, S, sa);
}

// The same with the accumulator held in one place: left to itself, the
// compiler gives the largest tile's products a result register other than
// the one they add to, and with 256 accumulators there is none to spare.
// Bytes 0 and 1 only. The s_nop covers the wait that a preceding vector
// instruction's write to an operand needs, which the compiler does not count
// for assembly; it runs under the previous product. Results may be read
// after settle().
template <int S>
__device__ __forceinline__ void mfma_in_place(f32x4 &c, i32x8 b, i32x8 a, int sb, int sa)
{
    static_assert(S == 0 || S == 1, "");
    if constexpr (S == 0)
        asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                     : "+a"(c)
                     : "v"(b), "v"(a), "v"(sb), "v"(sa));
    else
        asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] "
                     "op_sel_hi:[0,0,0]"
                     : "+a"(c)
                     : "v"(b), "v"(a), "v"(sb), "v"(sa));
}

// Waits until the last product's result can be read.
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15"); }

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The float whose exponent is scale byte S of a dword (what the conversion
// reads of its scale).
template <int S>
__device__ __forceinline__ float scale_of(int scales)
{
    return __int_as_float(((scales >> (8 * S)) & 0xFF) << 23);
}

// 32 scaled e4m3 values in bf16.
struct Wide {
    bf16x8 v[4];
};

__device__ __forceinline__ Wide widen(i32x8 x, float scale)
{
    Wide w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], scale, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], scale, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], scale, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], scale, true);
        w.v[q] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    return w;
}

__device__ __forceinline__ f32x4 mfma_wide(const Wide &b, const Wide &a, f32x4 c)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[q], a.v[q], c, 0, 0, 0);
    return c;
}

// 8 neighbouring outputs of a row of n.
__device__ __forceinline__ void put_out(void *out, int dtype, uint64_t row, uint64_t stride, uint32_t c, uint32_t n,
                                        const float *f)
{
    if (c >= n) return;
    if (dtype == kBF16) store8<kBF16>((uint16_t *)out + row * stride, c, n, f);
    else if (dtype == kF16) store8<kF16>((uint16_t *)out + row * stride, c, n, f);
    else store8<kF32>((float *)out + row * stride, c, n, f);
}

struct TileParams {
    const uint8_t *a, *a_scale, *b, *b_scale;
    uint32_t a_stride, a_scale_stride, b_stride, b_scale_stride;
    uint32_t m, n, k;
    uint32_t tiles_m, tiles_n, steps_per_split;
    void *out;
    uint64_t out_stride, split_stride;  // split_stride: elements between the splits' outputs
    int out_dtype;
};

// A workgroup's tile and its steps of k.
struct TilePlace {
    uint32_t m0, n0, split, s0, s1;
};

__device__ __forceinline__ TilePlace place_of(const TileParams &p, uint32_t BM, uint32_t BN)
{
    // workgroup id -> tile: each of the 8 XCDs (ids taken in turn) gets a
    // contiguous run of tiles, which go down 8 tile rows at a time, so that
    // the operands an XCD reads at one time are few enough for its own L2
    const uint32_t ntiles = p.tiles_m * p.tiles_n, total = gridDim.x;
    const uint32_t xcd = blockIdx.x & 7u, per = total >> 3, extra = total & 7u;
    const uint32_t id = xcd * per + (xcd < extra ? xcd : extra) + (blockIdx.x >> 3);
    // (the quotients come out of vector registers: back to scalar ones)
    const uint32_t split = __builtin_amdgcn_readfirstlane(id / ntiles), tile = id - split * ntiles;
    const uint32_t band = __builtin_amdgcn_readfirstlane(tile / (8 * p.tiles_n)), band_m = band * 8;
    const uint32_t band_rows = p.tiles_m - band_m < 8 ? p.tiles_m - band_m : 8;
    const uint32_t in_band = tile - band * 8 * p.tiles_n;
    const uint32_t column = __builtin_amdgcn_readfirstlane(in_band / band_rows);
    TilePlace t;
    t.m0 = (band_m + in_band - column * band_rows) * BM;
    t.n0 = column * BN;
    const uint32_t all_steps = (p.k + kStep - 1) / kStep;
    t.split = split;
    t.s0 = split * p.steps_per_split;
    t.s1 = t.s0 + p.steps_per_split < all_steps ? t.s0 + p.steps_per_split : all_steps;
    return t;
}

// Tiles of 32 FM x 32 FN outputs; four waves, 2 x 2, each with FM x FN
// fragments of 16 x 16. A step's operands (128 values of k) are copied to
// LDS by loads that bypass the registers, one step ahead, into the other of
// two buffers. One barrier per step, before the last pair of A fragments is
// multiplied: by then every wave has read all it needs of this step and its
// own copies of the next have landed, so the first fragments of the next
// step are read, and the copies of the step after it start, under those
// products.
//
// SPREAD, for the largest tile: a compute unit takes in about 32 bytes of
// copies per cycle, so that a step's 64 KiB last as long as its products (32
// cycles each, 64 of them per wave) and are issued over all of it. A's go
// into the buffer that the barrier has freed, half of them in the next step's
// first group; B's a step earlier, behind a second barrier after the first
// group, when every wave holds its fragments of B. Issued together in the
// last group they took 2,160 cycles there, and a step 3,790.
//
// LDS: a row's 128 bytes are 8 chunks of 16; chunk c of the fragment row r
// stands at c ^ (r / 2). A 16-byte LDS read serves 16 lanes at a time, 8 of
// them with odd rows and 8 with even ones (which lie 128 bytes apart, in
// different halves of the banks); the exchange spreads each 8 over the 8
// chunks of a row. The copy to LDS writes lane after lane, so the exchange
// is made in the address that a lane loads from, inside one 128-byte line.
//
// B's fragment f has rows n = 4 FB (r / 4) + 4 f + r % 4 of a block of 16 FB
// (FB = up to 4 fragments): a lane's results from the FB fragments are then
// 4 FB neighbours in its output row.
template <int FM, int FN, bool BLOCKS, bool KTAIL, bool EXACT>
__global__ __launch_bounds__(256) void gemm_tile(TileParams p)
{
    constexpr uint32_t BM = 32 * FM, BN = 32 * FN;
    constexpr int FB = FN < 4 ? FN : 4, NG = FM / 2;
    constexpr bool IN_PLACE = !EXACT && FM * FN == 64;
    constexpr int LA = BM / 32, LB = BN / 32;  // copies of 8 rows per wave
    constexpr bool SPREAD = !EXACT && FM == 8 && FN == 8;
    __shared__ __attribute__((aligned(16))) uint8_t as0[BM * kStep], as1[BM * kStep], bs0[BN * kStep],
        bs1[BN * kStep];
    const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = w >> 1, wn = w & 1u, r = lane & 15u, g = lane >> 4;
    const TilePlace place = place_of(p, BM, BN);
    const uint32_t m0 = place.m0, n0 = place.n0, s0 = place.s0, s1 = place.s1;
    const uint32_t all_steps = (p.k + kStep - 1) / kStep;
    const uint32_t steps = s1 - s0;

    const uint8_t *const pa = p.a + (uint64_t)m0 * p.a_stride, *const pb = p.b + (uint64_t)n0 * p.b_stride;
    // where this lane's part of each copy comes from (rows past the end: the last one)
    uint32_t va[LA], vb[LB], ca[LA], cb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const uint32_t row = (w * LA + i) * 8 + (lane >> 3), in = m0 + row < p.m ? row : p.m - 1 - m0;
        ca[i] = ((lane & 7u) ^ ((row >> 1) & 7u)) * 16;
        va[i] = in * p.a_stride + ca[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const uint32_t row = (w * LB + i) * 8 + (lane >> 3), in = n0 + row < p.n ? row : p.n - 1 - n0;
        cb[i] = ((lane & 7u) ^ (((row / (4 * FB)) & 3u) << 1 | ((row >> 1) & 1u))) * 16;
        vb[i] = in * p.b_stride + cb[i];
    }
    // this wave's copies of 8 rows, j of FN shares
    const auto copy_share = [&](uint32_t s, uint8_t *as, uint8_t *bs, int j) {
        const uint32_t k0 = s * kStep;
        const uint32_t size = s < s1 ? kInside : 0;  // past the last step: zeros
        const auto ra = buffer_of(pa, size), rb = buffer_of(pb, size);
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            if (i % FN != j) continue;
            const uint32_t v = KTAIL && k0 + ca[i] >= p.k ? kOutside : va[i];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(as + (w * LA + i) * 1024), 16, v, k0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            if (i % FN != j) continue;
            const uint32_t v = KTAIL && k0 + cb[i] >= p.k ? kOutside : vb[i];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(bs + (w * LB + i) * 1024), 16, v, k0, 0, 0);
        }
    };
    // one of this wave's copies of 8 rows
    [[maybe_unused]] const auto copy_a = [&](uint32_t s, uint8_t *as, int i) {
        const uint32_t k0 = s * kStep, v = KTAIL && k0 + ca[i] >= p.k ? kOutside : va[i];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(pa, s < s1 ? kInside : 0),
                                                 (lds_void *)(as + (w * LA + i) * 1024), 16, v, k0, 0, 0);
    };
    [[maybe_unused]] const auto copy_b = [&](uint32_t s, uint8_t *bs, int i) {
        const uint32_t k0 = s * kStep, v = KTAIL && k0 + cb[i] >= p.k ? kOutside : vb[i];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(pb, s < s1 ? kInside : 0),
                                                 (lds_void *)(bs + (w * LB + i) * 1024), 16, v, k0, 0, 0);
    };
    const auto copy = [&](uint32_t s, uint8_t *as, uint8_t *bs) {
#pragma unroll
        for (int j = 0; j < FN; ++j) copy_share(s, as, bs, j);
    };
    // k ends inside a chunk: its bytes past k, which may hold anything, are
    // cleared in LDS
    const auto clear_tail = [&](uint8_t *as, uint8_t *bs) {
        const uint32_t chunk = (p.k % kStep) / 16, keep = p.k % 16;
        for (uint32_t row = threadIdx.x; row < BM + BN; row += 256) {
            uint8_t *at;
            if (row < BM) at = as + row * kStep + (chunk ^ ((row >> 1) & 7u)) * 16;
            else {
                const uint32_t rw = row - BM;
                at = bs + rw * kStep + (chunk ^ (((rw / (4 * FB)) & 3u) << 1 | ((rw >> 1) & 1u))) * 16;
            }
            for (uint32_t e = keep; e < 16; ++e) at[e] = 0;
        }
        __syncthreads();
    };
    const bool partial_chunk = KTAIL && p.k % 16 != 0 && s1 == all_steps;

    const uint32_t oa = (wm * FM * 16 + r) * kStep + (g ^ (r >> 1)) * 16;
    const uint32_t ob = (wn * FN * 16 + (r >> 2) * (4 * FB) + (r & 3u)) * kStep + (g ^ (r >> 1)) * 16;
    const auto read_a = [&](const uint8_t *as, int i) {
        return join(*reinterpret_cast<const i32x4 *>(as + oa + i * 16 * kStep),
                    *reinterpret_cast<const i32x4 *>(as + (oa ^ 64u) + i * 16 * kStep));
    };
    const auto read_b = [&](const uint8_t *bs, int f) {
        const uint32_t at = (f / FB) * 16 * FB * kStep + (f % FB) * 4 * kStep;
        return join(*reinterpret_cast<const i32x4 *>(bs + ob + at),
                    *reinterpret_cast<const i32x4 *>(bs + (ob ^ 64u) + at));
    };
    // scales: a dword has a row's bytes for four steps; one row of scales for
    // a wave's columns where they are for blocks
    constexpr int NB = BLOCKS ? 1 : FN;
    const uint8_t *const qa = p.a_scale + (uint64_t)m0 * p.a_scale_stride;
    const uint8_t *const qb = p.b_scale + (uint64_t)(BLOCKS ? n0 / 128 : n0) * p.b_scale_stride;
    uint32_t va_scale[FM], vb_scale[NB];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t row = wm * FM * 16 + i * 16 + r;
        va_scale[i] = (m0 + row < p.m ? row : p.m - 1 - m0) * p.a_scale_stride;
    }
#pragma unroll
    for (int f = 0; f < NB; ++f) {
        const uint32_t first = wn * FN * 16;
        uint32_t row = BLOCKS ? first : first + (f / FB) * 16 * FB + (r >> 2) * (4 * FB) + (f % FB) * 4 + (r & 3u);
        row = n0 + row < p.n ? row : p.n - 1 - n0;
        vb_scale[f] = (BLOCKS ? (n0 + row) / 128 - n0 / 128 : row) * p.b_scale_stride;
    }
    int sa[FM], sb[NB], ha[FM], hb[NB], na[FM], nb[NB];  // this pair of steps', these four steps', the next four's
    const auto load_scales = [&](uint32_t s, int *ta, int *tb) {
        const uint32_t at = s < s1 ? s : s0;
#pragma unroll
        for (int i = 0; i < FM; ++i) ta[i] = *reinterpret_cast<const int *>(qa + at + va_scale[i]);
#pragma unroll
        for (int f = 0; f < NB; ++f) tb[f] = *reinterpret_cast<const int *>(qb + at + vb_scale[f]);
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f) acc[i][f] = (f32x4)0.0f;
    i32x8 af[2][2], bf[FN];

    // step s, whose operands are in (as, bs) and the next one's in (an, bn)
    const auto step = [&](auto par, uint32_t s, uint8_t *as, uint8_t *bs, uint8_t *an, uint8_t *bn) {
        constexpr int S = decltype(par)::value;
#pragma unroll
        for (int ag = 0; ag < NG; ++ag) {
            constexpr int P0 = (S * NG) & 1;
            const int cur = (P0 + ag) & 1;
            if (ag + 1 < NG) {
                af[cur ^ 1][0] = read_a(as, 2 * ag + 2);
                af[cur ^ 1][1] = read_a(as, 2 * ag + 3);
            } else {
                // this wave's LDS reads and copies are done (where they are
                // spread: but for the last LB, of B's step after the next)
                if constexpr (SPREAD) {
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LB) : "memory");
                } else {
                    __builtin_amdgcn_s_waitcnt(0x0070);
                    __syncthreads();
                }
                if (partial_chunk && s + 2 == s1) clear_tail(an, bn);
                af[cur ^ 1][0] = read_a(an, 0);
                af[cur ^ 1][1] = read_a(an, 1);
            }
            // every wave holds its part of B: its place is free
            if (SPREAD && ag == 1) asm volatile("s_barrier" ::: "memory");
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if constexpr (SPREAD) {  // a copy before every other pair of products
                    if (f % 2 == 0) {
                        const int i = f / 2;
                        if (ag + 1 == NG) copy_a(s + 2, as, i);
                        else if (ag == 0) copy_a(s + 1, an, LA / 2 + i);
                        else copy_b(s + 2, bs, (ag - 1) * (LB / 2) + i);
                    }
                } else if (ag + 1 == NG) {
                    copy_share(s + 2, as, bs, f);  // one share before each pair of products
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 2 * ag + h;
                    if constexpr (IN_PLACE) mfma_in_place<S>(acc[i][f], bf[f], af[cur][h], sb[BLOCKS ? 0 : f], sa[i]);
                    else acc[i][f] = mfma<S>(bf[f], af[cur][h], acc[i][f], sb[BLOCKS ? 0 : f], sa[i]);
                }
                if (ag + 1 == NG) {
                    bf[f] = read_b(bn, f);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // keep the group's products here: left alone, the compiler moves
            // them down to the loop's end, with every operand live until there
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < FN; ++f) asm volatile("" : "+a"(acc[2 * ag + h][f]));
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The same step on widened operands: while a group's products run, the
    // next group's fragments are widened and those of the one after it read.
    [[maybe_unused]] Wide aw[2], bw[EXACT ? FN : 1];
    [[maybe_unused]] i32x8 raw[2];
    [[maybe_unused]] int pa_next[FM], pb_next[NB];  // the next pair of steps' scales
    [[maybe_unused]] const auto step_wide = [&](auto par, uint32_t s, uint8_t *as, uint8_t *bs, uint8_t *an,
                                                uint8_t *bn) {
        constexpr int S = decltype(par)::value;
        const auto next_a = [&](int i) { return S == 0 ? scale_of<1>(sa[i]) : scale_of<0>(pa_next[i]); };
        const auto next_b = [&](int f) { return S == 0 ? scale_of<1>(sb[f]) : scale_of<0>(pb_next[f]); };
#pragma unroll
        for (int ag = 0; ag < NG; ++ag) {
            i32x8 after[2], rb[FN];
            if (ag + 1 < NG) {
                if (ag + 2 < NG) {
                    after[0] = read_a(as, 2 * ag + 4);
                    after[1] = read_a(as, 2 * ag + 5);
                }
            } else {
                __builtin_amdgcn_s_waitcnt(0x0070);  // this wave's LDS reads and copies are done
                __syncthreads();
                if (partial_chunk && s + 2 == s1) clear_tail(an, bn);
                raw[0] = read_a(an, 0);
                raw[1] = read_a(an, 1);
#pragma unroll
                for (int f = 0; f < FN; ++f) rb[f] = read_b(bn, f);
                if constexpr (NG > 1) {
                    after[0] = read_a(an, 2);
                    after[1] = read_a(an, 3);
                }
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if (ag + 1 == NG) copy_share(s + 2, as, bs, f);
                acc[2 * ag][f] = mfma_wide(bw[f], aw[0], acc[2 * ag][f]);
                acc[2 * ag + 1][f] = mfma_wide(bw[f], aw[1], acc[2 * ag + 1][f]);
                if (ag + 1 == NG) bw[f] = widen(rb[f], next_b(BLOCKS ? 0 : f));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                aw[h] = widen(raw[h], ag + 1 < NG ? scale_of<S>(sa[(2 * ag + 2 + h) % FM]) : next_a(h));
                raw[h] = after[h];
            }
            // between products, their share of the conversions
            if (ag + 1 < NG) {
#pragma unroll
                for (int q = 0; q < 8 * FN; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, (32 + 8 * FN - 1) / (8 * FN), 0);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < FN; ++f) asm volatile("" : "+a"(acc[2 * ag + h][f]));
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    load_scales(s0, ha, hb);
    copy(s0, as0, bs0);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    if (partial_chunk && steps == 1) clear_tail(as0, bs0);
    if constexpr (SPREAD) {
#pragma unroll
        for (int i = 0; i < LB; ++i) copy_b(s0 + 1, bs1, i);
#pragma unroll
        for (int i = 0; i < LA / 2; ++i) copy_a(s0 + 1, as1, i);
    } else {
        copy(s0 + 1, as1, bs1);
    }
    if constexpr (EXACT) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            aw[h] = widen(read_a(as0, h), scale_of<0>(ha[h]));
            if constexpr (NG > 1) raw[h] = read_a(as0, 2 + h);
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) bw[f] = widen(read_b(bs0, f), scale_of<0>(hb[BLOCKS ? 0 : f]));
    } else {
        af[0][0] = read_a(as0, 0);
        af[0][1] = read_a(as0, 1);
#pragma unroll
        for (int f = 0; f < FN; ++f) bf[f] = read_b(bs0, f);
    }
    // two steps a turn, the second of an odd number on zeros; s0 is a multiple of 4
    uint32_t s = s0;
    do {
        if ((s & 2u) == 0) load_scales(s + 4, na, nb);
        // a step past k's end has no scale: 1 in place of what stands there
        const uint32_t shift = (s & 2u) * 8;
        const int keep = s + 1 < all_steps ? -1 : 0xFF, fill = s + 1 < all_steps ? 0 : 0x7F00;
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = ((ha[i] >> shift) & keep) | fill;
#pragma unroll
        for (int f = 0; f < NB; ++f) sb[f] = ((hb[f] >> shift) & keep) | fill;
        if constexpr (EXACT) {
#pragma unroll
            for (int i = 0; i < 2; ++i) pa_next[i] = (s & 2u) ? na[i] : ha[i] >> 16;
#pragma unroll
            for (int f = 0; f < NB; ++f) pb_next[f] = (s & 2u) ? nb[f] : hb[f] >> 16;
            step_wide(std::integral_constant<int, 0>{}, s, as0, bs0, as1, bs1);
            step_wide(std::integral_constant<int, 1>{}, s + 1, as1, bs1, as0, bs0);
        } else {
            step(std::integral_constant<int, 0>{}, s, as0, bs0, as1, bs1);
            step(std::integral_constant<int, 1>{}, s + 1, as1, bs1, as0, bs0);
        }
        if (s & 2u) {
#pragma unroll
            for (int i = 0; i < FM; ++i) ha[i] = na[i];
#pragma unroll
            for (int f = 0; f < NB; ++f) hb[f] = nb[f];
        }
        s += 2;
    } while (s < s1);
    __builtin_amdgcn_s_waitcnt(0x0070);  // the copies past the end (zeros) are in LDS while it is this workgroup's

    if constexpr (IN_PLACE) {
        settle();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) asm volatile("" : "+a"(acc[i][f]));
    }
    void *const out = p.out_dtype == kF32 ? (void *)((float *)p.out + place.split * p.split_stride) : p.out;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t row = m0 + wm * FM * 16 + i * 16 + r;
        if (row >= p.m) continue;
#pragma unroll
        for (int q = 0; q < FN / FB; ++q) {
            const uint32_t c = n0 + wn * FN * 16 + q * 16 * FB + g * 4 * FB;
#pragma unroll
            for (int h = 0; h < FB / 2; ++h) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = acc[i][q * FB + 2 * h + (e >> 2)][e & 3];
                put_out(out, p.out_dtype, row, p.out_stride, c + 8 * h, p.n, o);
            }
        }
    }
}

// 32-bit outputs of large matrices: tiles of 256 x 128 as above, with the
// 32 x 32 bf16 instruction (measured on one SIMD unit: 1,011 operations per
// cycle, the 16 x 16 one 600; the product above went from 927 to 811 us). Bound
// by a wave's issue: alone on its unit it issues a vector instruction every 8
// cycles (measured), so that a step's 192 conversions take 1,600 cycles beside
// 64 products of 32. Four waves, 2 x 2, each with 4 x 2 fragments of
// 32 x 32: lane l carries row l % 32 and the 16-byte chunks l / 32 + 2 j
// (j < 4) of its 128 values. A step goes by A's fragments, 16 products each;
// the next fragment is widened, and the one after it read, under them.
//
// LDS: chunk c of A's row r stands at c ^ (r / 2 % 8). B's fragment f has the
// rows n = 32 (r / 4 % 2) + 8 (r / 8) + 4 f + r % 4 of its wave's 64, so that a
// lane's results are 32 neighbours in its output row; chunk c of row n stands
// at c ^ (bits 1, 5 and 3 of n): the 16 lanes that a read serves together have
// each of the 8 values twice, with an even row and with an odd one.
struct Raw {
    i32x4 c[4];
};

// 64 scaled e4m3 values in bf16: piece k is half k % 2 of chunk k / 2.
struct Wide64 {
    bf16x8 v[8];
};

__device__ __forceinline__ bf16x8 widen_piece(const Raw &x, int k, float scale)
{
    const int lo = x.c[k >> 1][2 * (k & 1)], hi = x.c[k >> 1][2 * (k & 1) + 1];
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <bool BLOCKS, bool KTAIL>
__global__ __launch_bounds__(256) void gemm_wide(TileParams p)
{
    constexpr uint32_t BM = 256, BN = 128;
    constexpr int LA = BM / 32, LB = BN / 32;  // copies of 8 rows per wave
    __shared__ __attribute__((aligned(16))) uint8_t as0[BM * kStep], as1[BM * kStep], bs0[BN * kStep],
        bs1[BN * kStep];
    const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = w >> 1, wn = w & 1u, r = lane & 31u, g = lane >> 5;
    const TilePlace at = place_of(p, BM, BN);
    const uint32_t m0 = at.m0, n0 = at.n0, s0 = at.s0, s1 = at.s1;
    const uint32_t all_steps = (p.k + kStep - 1) / kStep;

    const uint8_t *const pa = p.a + (uint64_t)m0 * p.a_stride, *const pb = p.b + (uint64_t)n0 * p.b_stride;
    const auto key_a = [](uint32_t row) { return (row >> 1) & 7u; };
    const auto key_b = [](uint32_t row) { return ((row >> 1) & 1u) | ((row >> 4) & 2u) | ((row >> 1) & 4u); };
    // where this lane's part of each copy comes from (rows past the end: the last one)
    uint32_t va[LA], vb[LB], ca[LA], cb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const uint32_t row = (w * LA + i) * 8 + (lane >> 3), in = m0 + row < p.m ? row : p.m - 1 - m0;
        ca[i] = ((lane & 7u) ^ key_a(row)) * 16;
        va[i] = in * p.a_stride + ca[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const uint32_t row = (w * LB + i) * 8 + (lane >> 3), in = n0 + row < p.n ? row : p.n - 1 - n0;
        cb[i] = ((lane & 7u) ^ key_b(row)) * 16;
        vb[i] = in * p.b_stride + cb[i];
    }
    // one of this wave's copies of 8 rows; past the last step: zeros
    const auto copy_a = [&](uint32_t s, uint8_t *as, int i) {
        const uint32_t k0 = s * kStep, v = KTAIL && k0 + ca[i] >= p.k ? kOutside : va[i];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(pa, s < s1 ? kInside : 0),
                                                 (lds_void *)(as + (w * LA + i) * 1024), 16, v, k0, 0, 0);
    };
    const auto copy_b = [&](uint32_t s, uint8_t *bs, int i) {
        const uint32_t k0 = s * kStep, v = KTAIL && k0 + cb[i] >= p.k ? kOutside : vb[i];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(pb, s < s1 ? kInside : 0),
                                                 (lds_void *)(bs + (w * LB + i) * 1024), 16, v, k0, 0, 0);
    };
    // k ends inside a chunk: its bytes past k, which may hold anything, are
    // cleared in LDS
    const auto clear_tail = [&](uint8_t *as, uint8_t *bs) {
        const uint32_t chunk = (p.k % kStep) / 16, keep = p.k % 16;
        for (uint32_t row = threadIdx.x; row < BM + BN; row += 256) {
            uint8_t *const at = row < BM ? as + row * kStep + (chunk ^ key_a(row)) * 16
                                         : bs + (row - BM) * kStep + (chunk ^ key_b(row - BM)) * 16;
            for (uint32_t e = keep; e < 16; ++e) at[e] = 0;
        }
        __syncthreads();
    };
    const bool partial_chunk = KTAIL && p.k % 16 != 0 && s1 == all_steps;

    const uint32_t row_b = wn * 64 + 32 * ((r >> 2) & 1u) + 8 * (r >> 3) + (r & 3u);
    const uint32_t oa = (wm * 128 + r) * kStep + (g ^ key_a(r)) * 16;
    const uint32_t ob = row_b * kStep + (g ^ key_b(row_b)) * 16;
    const auto read_a = [&](const uint8_t *as, int i) {
        Raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x.c[j] = *reinterpret_cast<const i32x4 *>(as + (oa ^ (32u * j)) + i * 32 * kStep);
        return x;
    };
    const auto read_b = [&](const uint8_t *bs, int f) {
        Raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x.c[j] = *reinterpret_cast<const i32x4 *>(bs + (ob ^ (32u * j)) + f * 4 * kStep);
        return x;
    };
    // scales: a dword has a row's bytes for four steps
    constexpr int NB = BLOCKS ? 1 : 2;
    const uint8_t *const qa = p.a_scale + (uint64_t)m0 * p.a_scale_stride;
    const uint8_t *const qb = p.b_scale + (uint64_t)(BLOCKS ? n0 / 128 : n0) * p.b_scale_stride;
    uint32_t va_scale[4], vb_scale[NB];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = wm * 128 + i * 32 + r;
        va_scale[i] = (m0 + row < p.m ? row : p.m - 1 - m0) * p.a_scale_stride;
    }
#pragma unroll
    for (int f = 0; f < NB; ++f) {
        const uint32_t row = row_b + 4 * f;
        vb_scale[f] = BLOCKS ? 0 : (n0 + row < p.n ? row : p.n - 1 - n0) * p.b_scale_stride;  // n0 is a multiple of 128
    }
    int sa[4], sb[NB], ha[4], hb[NB], na[4], nb[NB];  // this pair of steps', these four steps', the next four's
    int pa_next[4], pb_next[NB];                      // the next pair of steps'
    const auto load_scales = [&](uint32_t s, int *ta, int *tb) {
        const uint32_t at = s < s1 ? s : s0;
#pragma unroll
        for (int i = 0; i < 4; ++i) ta[i] = *reinterpret_cast<const int *>(qa + at + va_scale[i]);
#pragma unroll
        for (int f = 0; f < NB; ++f) tb[f] = *reinterpret_cast<const int *>(qb + at + vb_scale[f]);
    };

    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f) acc[i][f] = (f32x16)0.0f;
    Wide64 aw, an_wide, bw[2];  // this fragment of A, the next one, B's
    Raw raw;                    // the fragment of A after aw

    // step s, whose operands are in (as, bs) and the next one's in (an, bn)
    const auto step = [&](auto par, uint32_t s, uint8_t *as, uint8_t *bs, uint8_t *an, uint8_t *bn) {
        constexpr int S = decltype(par)::value;
#pragma unroll
        for (int ag = 0; ag < 4; ++ag) {
            Raw after, rb[2];
            float scale_a, scale_b[2];
            if (ag < 3) {
                if (ag < 2) after = read_a(as, ag + 2);
                scale_a = scale_of<S>(sa[(ag + 1) & 3]);
            } else {
                // this wave's LDS reads are done, and its copies but the last
                // LB, of B's step after the next
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LB) : "memory");
                if (partial_chunk && s + 2 == s1) clear_tail(an, bn);
                raw = read_a(an, 0);
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    rb[f] = read_b(bn, f);
                    scale_b[f] = S == 0 ? scale_of<1>(sb[BLOCKS ? 0 : f]) : scale_of<0>(pb_next[BLOCKS ? 0 : f]);
                }
                after = read_a(an, 1);
                scale_a = S == 0 ? scale_of<1>(sa[0]) : scale_of<0>(pa_next[0]);
            }
            // every wave holds its part of B: its place is free
            if (ag == 1) asm volatile("s_barrier" ::: "memory");
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // a copy before every fourth product, B's every eighth
                if (k % 2 == 0) {
                    if (ag == 3) copy_a(s + 2, as, k / 2);
                    else if (ag == 0) copy_a(s + 1, an, LA / 2 + k / 2);
                    else if (k % 4 == 0) copy_b(s + 2, bs, (ag - 1) * (LB / 2) + k / 4);
                }
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    acc[ag][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bw[f].v[k], aw.v[k], acc[ag][f], 0, 0, 0);
                // (in the last group two places late: the reads take that long)
                const int late = ag == 3 ? 2 : 0;
                if (k >= late) {
                    an_wide.v[k - late] = widen_piece(raw, k - late, scale_a);
                    if (ag == 3) {
#pragma unroll
                        for (int f = 0; f < 2; ++f) bw[f].v[k - late] = widen_piece(rb[f], k - late, scale_b[f]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (ag == 3) {
#pragma unroll
                for (int k = 6; k < 8; ++k) {
                    an_wide.v[k] = widen_piece(raw, k, scale_a);
#pragma unroll
                    for (int f = 0; f < 2; ++f) bw[f].v[k] = widen_piece(rb[f], k, scale_b[f]);
                }
            }
            aw = an_wide;
            raw = after;
#pragma unroll
            for (int f = 0; f < 2; ++f) asm volatile("" : "+a"(acc[ag][f]));
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    load_scales(s0, ha, hb);
#pragma unroll
    for (int i = 0; i < LA; ++i) copy_a(s0, as0, i);
#pragma unroll
    for (int i = 0; i < LB; ++i) copy_b(s0, bs0, i);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    if (partial_chunk && s0 + 1 == s1) clear_tail(as0, bs0);
#pragma unroll
    for (int i = 0; i < LB; ++i) copy_b(s0 + 1, bs1, i);
#pragma unroll
    for (int i = 0; i < LA / 2; ++i) copy_a(s0 + 1, as1, i);
    {
        const Raw x = read_a(as0, 0), y[2] = {read_b(bs0, 0), read_b(bs0, 1)};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            aw.v[k] = widen_piece(x, k, scale_of<0>(ha[0]));
#pragma unroll
            for (int f = 0; f < 2; ++f) bw[f].v[k] = widen_piece(y[f], k, scale_of<0>(hb[BLOCKS ? 0 : f]));
        }
        raw = read_a(as0, 1);
    }
    // two steps a turn, the second of an odd number on zeros; s0 is a multiple of 4
    uint32_t s = s0;
    do {
        if ((s & 2u) == 0) load_scales(s + 4, na, nb);
        // a step past k's end has no scale: 1 in place of what stands there
        const uint32_t shift = (s & 2u) * 8;
        const int keep = s + 1 < all_steps ? -1 : 0xFF, fill = s + 1 < all_steps ? 0 : 0x7F00;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sa[i] = ((ha[i] >> shift) & keep) | fill;
            pa_next[i] = (s & 2u) ? na[i] : ha[i] >> 16;
        }
#pragma unroll
        for (int f = 0; f < NB; ++f) {
            sb[f] = ((hb[f] >> shift) & keep) | fill;
            pb_next[f] = (s & 2u) ? nb[f] : hb[f] >> 16;
        }
        step(std::integral_constant<int, 0>{}, s, as0, bs0, as1, bs1);
        step(std::integral_constant<int, 1>{}, s + 1, as1, bs1, as0, bs0);
        if (s & 2u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ha[i] = na[i];
#pragma unroll
            for (int f = 0; f < NB; ++f) hb[f] = nb[f];
        }
        s += 2;
    } while (s < s1);
    __builtin_amdgcn_s_waitcnt(0x0070);  // the copies past the end (zeros) are in LDS while it is this workgroup's

    float *const out = (float *)p.out + at.split * p.split_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = m0 + wm * 128 + i * 32 + r;
        if (row >= p.m) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = acc[i][e >> 2][4 * q + (e & 3)];
            put_out(out, kF32, row, p.out_stride, n0 + wn * 64 + 32 * g + 8 * q, p.n, o);
        }
    }
}

// The splits' partial products, joined in order.
__global__ __launch_bounds__(256) void join_splits(const float *__restrict__ part, uint32_t splits, uint64_t split_stride,
                                                   uint32_t n8, uint32_t n, uint64_t count, void *out,
                                                   uint64_t out_stride, int dtype)
{
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (uint64_t)gridDim.x * 256) {
        const uint64_t row = i / n8;
        const uint32_t c = (uint32_t)(i - row * n8) * 8;
        float f[8] = {};
        for (uint32_t s = 0; s < splits; ++s) {
            const auto v = load8<kF32>(part + s * split_stride + row * n, c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += v[e];
        }
        put_out(out, dtype, row, out_stride, c, n, f);
    }
}

// Few rows of A (16 MT at most): B is read once and, up to 16 rows, bounds the
// time. 32 rows of the product above take 39 us and 64 take 62: each of its 256
// workgroups reads all of A from L2, 0.2 and 0.4 GB together (and five of the
// eight forms of 64 rows spill 4 to 15 registers). A
// workgroup has 16 columns of the output; its W waves take runs of steps of
// k, straight into registers, and add their sums through LDS. A wave reads
// the next U steps while it multiplies U: 8 KiB of B in flight for each of
// a compute unit's eight waves. (A comes from L2; with 64 rows of it there
// is room for one U of them only.)
template <int MT, int W, bool BLOCKS, bool EXACT, bool KTAIL>
__global__ __launch_bounds__(W * 64, 2) void gemm_rows(TileParams p)
{
    constexpr int U = 4;  // steps read together: those of a dword of scales
    constexpr bool A_AHEAD = MT <= 2;
    __shared__ f32x4 sums[W][MT][64];
    const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 15u, g = lane >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t steps = (p.k + kStep - 1) / kStep;
    const uint32_t s0 = w * p.steps_per_split < steps ? w * p.steps_per_split : steps;
    const uint32_t s1 = s0 + p.steps_per_split < steps ? s0 + p.steps_per_split : steps;
    const uint8_t *const pb = p.b + (uint64_t)n0 * p.b_stride;
    const uint32_t nr = n0 + r < p.n ? r : p.n - 1 - n0;
    const uint32_t vb = nr * p.b_stride + g * 16;
    uint32_t va[MT];
    const uint8_t *psa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const uint32_t row = t * 16 + r < p.m ? t * 16 + r : p.m - 1;
        va[t] = row * p.a_stride + g * 16;
        psa[t] = p.a_scale + (uint64_t)row * p.a_scale_stride;
    }
    const uint8_t *const psb = p.b_scale + (uint64_t)(BLOCKS ? n0 / 128 : n0 + nr) * p.b_scale_stride;
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = (f32x4)0.0f;
    // 16 bytes at k of a row whose first byte this lane reads at offset v
    const auto load = [&](__amdgpu_buffer_rsrc_t rsrc, uint32_t v, uint32_t k0, uint32_t half) {
        const uint32_t k = k0 + half * 64 + g * 16;
        const uint32_t at = KTAIL && k >= p.k ? kOutside : v + half * 64;
        return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, k0, 0));
    };
    // bytes past k may hold anything
    const auto trim = [&](i32x8 x, uint32_t k0) {
        if constexpr (KTAIL) {
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q) {
                const uint32_t k = k0 + (q / 4) * 64 + g * 16 + (q % 4) * 4;
                if (k + 4 > p.k) x[q] &= k < p.k ? (int)((1u << (8 * (p.k - k))) - 1u) : 0;
            }
        }
        return x;
    };
    struct Batch {
        i32x8 b[U], a[U][MT];
        int sb, sa[MT];
    };
    const auto load_a = [&](uint32_t s, Batch &x) {
        const uint32_t at = s < s1 ? s : 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) x.sa[t] = *reinterpret_cast<const int *>(psa[t] + at);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const auto ra = buffer_of(p.a, s + u < s1 ? kInside : 0);
#pragma unroll
            for (int t = 0; t < MT; ++t)
                x.a[u][t] = join(load(ra, va[t], (s + u) * kStep, 0), load(ra, va[t], (s + u) * kStep, 1));
        }
    };
    const auto load_b = [&](uint32_t s, Batch &x) {
        x.sb = *reinterpret_cast<const int *>(psb + (s < s1 ? s : 0));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const auto rb = buffer_of(pb, s + u < s1 ? kInside : 0);  // past the wave's last step: nothing is read
            x.b[u] = join(load(rb, vb, (s + u) * kStep, 0), load(rb, vb, (s + u) * kStep, 1));
        }
    };
    const auto multiply = [&](uint32_t s, Batch &x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const i32x8 b = trim(x.b[u], (s + u) * kStep);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const i32x8 a = trim(x.a[u][t], (s + u) * kStep);
                if constexpr (EXACT)
                    acc[t] = mfma_wide(widen(b, scale_of<0>(x.sb >> (8 * u))), widen(a, scale_of<0>(x.sa[t] >> (8 * u))),
                                       acc[t]);
                else acc[t] = mfma<0>(b, a, acc[t], x.sb >> (8 * u), x.sa[t] >> (8 * u));
            }
        }
    };
    Batch x, y;
    const auto turn = [&](uint32_t s, Batch &now, Batch &next) {
        load_b(s + U, next);
        if constexpr (A_AHEAD) load_a(s + U, next);
        else load_a(s, now);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s, now);
        __builtin_amdgcn_sched_barrier(0);
    };
    load_b(s0, x);
    if constexpr (A_AHEAD) load_a(s0, x);
    for (uint32_t s = s0; s < s1; s += 2 * U) {
        turn(s, x, y);
        turn(s + U, y, x);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) sums[w][t][lane] = acc[t];
    __syncthreads();
    // lane l of fragment t has row 16 t + l % 16, columns 4 (l / 16) + e
    for (uint32_t i = threadIdx.x; i < MT * 256; i += W * 64) {
        const uint32_t t = i >> 8, row = t * 16 + ((i >> 4) & 15u), c = i & 15u;
        float f = 0.0f;
#pragma unroll
        for (int q = 0; q < W; ++q) f += sums[q][t][((c >> 2) << 4) | ((i >> 4) & 15u)][c & 3u];
        if (row < p.m && n0 + c < p.n) {
            const uint64_t at = row * p.out_stride + n0 + c;
            if (p.out_dtype == kBF16) ((uint16_t *)p.out)[at] = Elem<kBF16>::put(f);
            else if (p.out_dtype == kF16) ((uint16_t *)p.out)[at] = Elem<kF16>::put(f);
            else ((float *)p.out)[at] = f;
        }
    }
}

constexpr int kRowWaves = 8;

// How a product is cut: the rows kernel, or tiles of 32 f x 32 f and splits
// of k.
struct Cut {
    int rows;    // > 0: the rows kernel with this many fragments of A
    int fm, fn;  // else tiles of 32 fm x 32 fn
    uint32_t splits, steps_per_split;
};

Cut cut_of(uint64_t m, uint64_t n, uint64_t k, bool exact)
{
    const uint32_t steps = (uint32_t)div_up(k, kStep);
    Cut best{};
    if (m <= 64) {
        best.rows = m <= 16 ? 1 : m <= 32 ? 2 : 4;
        best.splits = 1;
        best.steps_per_split = (uint32_t)(div_up(div_up(steps, kRowWaves), 4) * 4);  // scales are read four steps at a time
        return best;
    }
    // time of each cut in cycles of one compute unit: rounds of workgroups
    // times their steps, the work of a step by tile size, a start and an end
    // per workgroup, and the pass that joins splits. (per_cu is what LDS allows
    // and the other figures were fitted with. The registers allow less in some
    // forms: one workgroup of the 128 x 128 tile with a 32-bit output or an end
    // of k inside a step, three of the 64 x 64 one with a 32-bit output. In a
    // sweep of 40 sizes the rule's cut took 3% more than the best of all on
    // average and 29% at most. With a 16-bit output, 128 x 128 tiles take
    // in a step's copies in twice the time of its products, so sizes that do
    // not fill the chip with 256 x 256 tiles run at half the rate or less:
    // 939 x 1,664 x 4,992 takes 25 us where the operations alone are 5.)
    double least = 0;
    struct Kind { int fm, fn; double step, ends; uint32_t per_cu; };
    static const Kind narrow[] = {{8, 8, 2430, 6000, 1}, {4, 4, 900, 4000, 2}, {2, 2, 330, 3000, 4}};
    static const Kind wide[] = {{8, 4, 2280, 6000, 1}, {4, 4, 1800, 4000, 2}, {2, 2, 660, 3000, 4}};
    const Kind *const kinds = exact ? wide : narrow;
    for (int q = 0; q < 3; ++q) {
        const Kind &t = kinds[q];
        const uint64_t tiles = div_up(m, 32u * t.fm) * div_up(n, 32u * t.fn);
        for (uint32_t want = 1; want <= 16; want *= 2) {
            const uint32_t per = (uint32_t)(div_up(div_up(steps, want), 4) * 4);
            const uint32_t splits = (uint32_t)div_up(steps, per);
            if (want > 1 && (per < 8 || splits != want)) continue;
            if (tiles * splits >= (1u << 24)) continue;  // a launch has fewer than 2^32 threads
            const uint64_t wgs = tiles * splits;
            const uint64_t full = wgs / (256 * t.per_cu), rest = wgs % (256 * t.per_cu);
            // a last round that does not fill the units runs fewer workgroups on each
            const double share = rest ? (double)div_up(rest, 256) : 0;
            double cost = (full * t.per_cu + share) * per * t.step + (full + (rest ? 1 : 0)) * t.ends;
            if (splits > 1) cost += 8000 + (double)m * n * 4 * (splits + 1) / 2000;
            if (best.fm == 0 || cost < least) {
                least = cost;
                best.fm = t.fm;
                best.fn = t.fn;
                best.splits = splits;
                best.steps_per_split = per;
            }
        }
    }
    return best;
}

template <int FM, int FN, bool BLOCKS, bool EXACT>
void launch_tile(const TileParams &p, uint32_t blocks, hipStream_t stream)
{
    if (p.k % kStep) gemm_tile<FM, FN, BLOCKS, true, EXACT><<<blocks, 256, 0, stream>>>(p);
    else gemm_tile<FM, FN, BLOCKS, false, EXACT><<<blocks, 256, 0, stream>>>(p);
}

template <int MT, bool BLOCKS, bool EXACT>
void launch_rows(const TileParams &p, uint32_t blocks, hipStream_t stream)
{
    if (p.k % kStep) gemm_rows<MT, kRowWaves, BLOCKS, EXACT, true><<<blocks, kRowWaves * 64, 0, stream>>>(p);
    else gemm_rows<MT, kRowWaves, BLOCKS, EXACT, false><<<blocks, kRowWaves * 64, 0, stream>>>(p);
}

template <bool BLOCKS, bool EXACT>
hipError_t launch_gemm(const GemmArgs &g)
{
    const Cut c = cut_of(g.m, g.n, g.k, EXACT);
    TileParams p{};
    p.a = g.a;
    p.a_scale = g.a_scale;
    p.b = g.b;
    p.b_scale = g.b_scale;
    p.a_stride = (uint32_t)g.a_stride;
    p.a_scale_stride = (uint32_t)g.a_scale_stride;
    p.b_stride = (uint32_t)g.b_stride;
    p.b_scale_stride = (uint32_t)g.b_scale_stride;
    p.m = (uint32_t)g.m;
    p.n = (uint32_t)g.n;
    p.k = (uint32_t)g.k;
    p.steps_per_split = c.steps_per_split;
    p.out = g.out;
    p.out_stride = g.out_stride;
    p.out_dtype = g.out_dtype;
    if (c.rows) {
        const uint32_t blocks = (uint32_t)div_up(g.n, 16);
        if (c.rows == 1) launch_rows<1, BLOCKS, EXACT>(p, blocks, g.stream);
        else if (c.rows == 2) launch_rows<2, BLOCKS, EXACT>(p, blocks, g.stream);
        else launch_rows<4, BLOCKS, EXACT>(p, blocks, g.stream);
        return hipGetLastError();
    }
    p.tiles_m = (uint32_t)div_up(g.m, 32u * c.fm);
    p.tiles_n = (uint32_t)div_up(g.n, 32u * c.fn);
    if (c.splits > 1) {
        p.out = g.workspace;
        p.out_stride = g.n;
        p.split_stride = g.m * g.n;
        p.out_dtype = kF32;
    }
    const uint32_t blocks = p.tiles_m * p.tiles_n * c.splits;
    if (c.fm == 4) launch_tile<4, 4, BLOCKS, EXACT>(p, blocks, g.stream);
    else if (c.fm == 2) launch_tile<2, 2, BLOCKS, EXACT>(p, blocks, g.stream);
    else if constexpr (EXACT) {
        if (p.k % kStep) gemm_wide<BLOCKS, true><<<blocks, 256, 0, g.stream>>>(p);
        else gemm_wide<BLOCKS, false><<<blocks, 256, 0, g.stream>>>(p);
    } else launch_tile<8, 8, BLOCKS, false>(p, blocks, g.stream);
    if (c.splits > 1) {
        const uint64_t n8 = div_up(g.n, 8), count = g.m * n8;
        const uint64_t wgs = div_up(count, 256);
        join_splits<<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, g.stream>>>(
            (const float *)g.workspace, c.splits, p.split_stride, (uint32_t)n8, (uint32_t)g.n, count, g.out,
            g.out_stride, g.out_dtype);
    }
    return hipGetLastError();
}

__global__ __launch_bounds__(256) void zero_out(void *out, int dtype, uint64_t stride, uint32_t n8, uint32_t n,
                                                uint64_t count)
{
    const float f[8] = {};
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (uint64_t)gridDim.x * 256)
        put_out(out, dtype, i / n8, stride, (uint32_t)(i % n8) * 8, n, f);
}

}  // namespace

uint64_t gemm_fp8_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int out_dtype)
{
    const Cut c = cut_of(m, n, k, out_dtype == kF32);
    return c.splits > 1 ? 4ull * c.splits * m * n : 0;
}

hipError_t gemm_fp8(const GemmArgs &g)
{
    if (g.k == 0) {  // an empty sum
        const uint64_t n8 = div_up(g.n, 8), count = g.m * n8, wgs = div_up(count, 256);
        zero_out<<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, g.stream>>>(g.out, g.out_dtype, g.out_stride,
                                                                           (uint32_t)n8, (uint32_t)g.n, count);
        return hipGetLastError();
    }
    if (g.out_dtype == kF32) return g.b_blocks ? launch_gemm<true, true>(g) : launch_gemm<false, true>(g);
    return g.b_blocks ? launch_gemm<true, false>(g) : launch_gemm<false, false>(g);
}

}  // namespace cpk
