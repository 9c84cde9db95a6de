// cp_linear_tile.h - the tiled product behind cp_linear, cp_linear_dx and
// cp_linear_dw: out[m][n] = sum over K of A B, each operand either rows of K or
// "across" (rows along K), in bf16, f16 or f32, summed in 32 bits.
#pragma once

#include <type_traits>

#include "cp_linear_internal.h"

namespace cpk {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int unaligned_i32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr uint32_t kStepBytes = 128;         // of each row or column of an operand, per step
constexpr uint32_t kInside = 0x7FFFFFFFu;    // bytes of a buffer: any offset within a tile
constexpr uint32_t kOutside = 0x80000000u;   // an offset past it: loads give zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t size)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)size, 0x00020000);
}

struct TileParams {
    const void *a, *b;
    uint64_t a_stride, b_stride;  // bytes
    uint32_t m, n, k;
    uint32_t tiles_m, tiles_n, steps_per_split;
    float *part;  // the splits' sums, [split][m][n], where k is split
    Epilogue e;
};

// A 16-byte piece of each operand: 8 values of K in 16 bits, 4 in 32.
template <int DT>
__device__ __forceinline__ f32x16 multiply(i32x4 b, i32x4 a, f32x16 c)
{
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c,
                                                       0, 0, 0);
    else if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0,
                                                      0, 0);
    else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(b[e]), __int_as_float(a[e]), c, 0, 0, 0);
        return c;
    }
}

// The same with the accumulator held in one place (16 bits). The s_nop covers
// the wait that a vector instruction's write to an operand needs, which the
// compiler does not count for assembly. Results may be read after settle().
template <int DT>
__device__ __forceinline__ void multiply_in_place(f32x16 &c, i32x4 b, i32x4 a)
{
    static_assert(DT == kBF16 || DT == kF16, "");
    if constexpr (DT == kBF16)
        asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
    else
        asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// Waits until the last product's result can be read.
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15"); }

// One operand's tile of W rows (or columns, where it is ACROSS), a step of K
// at a time, in LDS.
//
// Rows of K: a row's 128 bytes are 8 chunks of 16; chunk c of row r stands at
// c ^ (r / 2 % 8), as a 16-byte LDS read serves 16 lanes at a time, 8 with odd
// rows and 8 with even ones, which lie in different halves of the banks.
// ACROSS: a row of the step is the tile's W columns; a read that transposes
// takes 8 bytes of each of 4 rows for 16 lanes, 32 lanes at a time: 64-byte
// pieces of 4 rows, which change places within a row so that they lie in
// different banks. (32-bit columns are read one by one and stay in place.)
//
// The copy to LDS writes lane after lane, so the exchange is made in the
// address that a lane loads from.
// SHORT: rows of less than a chunk are read too.
template <int DT, bool ACROSS, int W, int F, bool DIRECT, bool SHORT>
struct Operand {
    static constexpr uint32_t ES = dtype_bytes(DT), EPC = 16 / ES;  // values of a 16-byte chunk
    static constexpr uint32_t KS = kStepBytes / ES;                 // values of K in a step
    static constexpr uint32_t RB = W * ES;                          // bytes of a row in LDS (ACROSS)
    static constexpr int COPIES = W / 32;                           // of 1 KiB, for each of four waves
    static constexpr uint32_t BYTES = W * kStepBytes;

    const uint8_t *base;     // of the tile at K = 0
    uint64_t stride;         // bytes between rows
    uint32_t from[COPIES];   // byte offset of this lane's chunk of each copy (its row, where not DIRECT; not of ACROSS then)
    uint32_t at[COPIES];     // its first value's place in K (ACROSS: its row's)
    uint32_t rows, width;    // all rows (ACROSS: columns), and those from the tile's first on
    uint32_t read[4];        // where this lane reads its fragments
    uint32_t w;

    // exchange of 64-byte pieces of row k of a step
    static __device__ __forceinline__ uint32_t piece(uint32_t k)
    {
        if constexpr (ES == 4) return 0;
        return W >= 128 ? k & 3u : (k >> 1) & 1u;
    }

    // `first`: the tile's first row or column of `rows_`; `part`: which of the
    // two waves along this operand reads
    __device__ __forceinline__ Operand(const void *p, uint64_t stride_, uint32_t first, uint32_t rows_, uint32_t part)
    {
        const uint32_t lane = threadIdx.x & 63u;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        stride = stride_;
        rows = rows_;
        width = rows - first;
        base = (const uint8_t *)p + (ACROSS ? (uint64_t)first * ES : (uint64_t)first * stride);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            if constexpr (!ACROSS) {
                const uint32_t row = (w * COPIES + i) * 8 + (lane >> 3), in = row < width ? row : width - 1;
                const uint32_t c = ((lane & 7u) ^ ((row >> 1) & 7u)) * 16;
                from[i] = in * (uint32_t)stride + (DIRECT ? c : 0);
                at[i] = c / ES;
            } else {
                at[i] = ((w * COPIES + i) * 1024 + lane * 16) / RB;
                const uint32_t c = column(i);
                // past the last column: the last chunk (DIRECT: columns are whole chunks)
                if constexpr (DIRECT) from[i] = at[i] * (uint32_t)stride + (c >= width ? width - EPC : c) * ES;
            }
        }
        const uint32_t r = lane & 31u, h = lane >> 5;
        if constexpr (!ACROSS) {
            const uint32_t o = (part * F * 32 + r) * kStepBytes + (h ^ ((r >> 1) & 7u)) * 16;
#pragma unroll
            for (int q = 0; q < 4; ++q) read[q] = o ^ (q * 32);
        } else if constexpr (ES == 2) {
            const uint32_t j = (lane & 15u) >> 2, g = lane & 3u, b = (lane >> 4) & 1u;
#pragma unroll
            for (int i = 0; i < F; ++i)
                read[i] = (8 * h + j) * RB + (((part * F + i) ^ piece(j)) * 64) + 32 * b + 8 * g;
        } else {
            read[0] = 4 * h * RB + (part * F * 32 + r) * 4;
        }
    }

    // copy i of the step at K = k0; zeros from k on (DIRECT)
    __device__ __forceinline__ void copy(uint8_t *lds, int i, uint32_t k0, uint32_t k) const
    {
        const auto rsrc = buffer_of(base + (ACROSS ? (uint64_t)k0 * stride : (uint64_t)k0 * ES), k0 < k ? kInside : 0);
        const uint32_t v = at[i] < k - k0 ? from[i] : kOutside;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(lds + (w * COPIES + i) * 1024), 16, v, 0, 0, 0);
    }

    // The same by way of a register, for rows at any alignment (of at least a
    // chunk, where not SHORT): a chunk that
    // reaches past the end of its row is read from the row's last 16 bytes
    // and moved into place by fix(), which has to be called where may_reach()
    // says so. (ACROSS, those may begin before the tile's first column.) `end`
    // is at least 1.
    __device__ __forceinline__ i32x4 load(int i, uint32_t k0, uint32_t end) const
    {
        if constexpr (ACROSS) {
            const uint32_t first = k0 < end ? k0 : end - 1, last = end - 1 - first;  // (rows past the end: the last one)
            const uint32_t row = at[i] < last ? at[i] : last;
            const int c = (int)column(i), most = (int)width - (int)EPC;
            const uint8_t *const p = base + (uint64_t)first * stride + (uint64_t)__umul24(row, (uint32_t)stride / ES) * ES;
            return SHORT && rows < EPC ? piecewise(p + c * (int)ES, row == at[i] && k0 < end && c < (int)width ? width - c : 0)
                                       : *reinterpret_cast<const unaligned_i32x4 *>(p + (int64_t)((c < most ? c : most) * (int)ES));
        } else {
            const uint32_t c = k0 + at[i], most = end - EPC;
            return SHORT && end < EPC ? piecewise(base + from[i] + c * ES, c < end ? end - c : 0)
                                      : *reinterpret_cast<const unaligned_i32x4 *>(base + (from[i] + (c < most ? c : most) * ES));
        }
    }

    // `have` values of a chunk
    static __device__ __forceinline__ i32x4 piecewise(const uint8_t *p, uint32_t have)
    {
        typename Elem<DT>::raw e[EPC] = {};
#pragma unroll
        for (uint32_t q = 0; q < EPC; ++q)
            if (q < have) e[q] = ((const typename Elem<DT>::raw *)p)[q];
        i32x4 v;
        __builtin_memcpy(&v, e, 16);
        return v;
    }

    // ACROSS: the column of this lane's chunk of copy i
    __device__ __forceinline__ uint32_t column(int i) const
    {
        const uint32_t in = ((w * COPIES + i) * 1024 + (threadIdx.x & 63u) * 16) % RB;
        return (((in / 64) ^ piece(at[i])) * 64 + in % 64) / ES;
    }

    __device__ __forceinline__ bool may_reach(uint32_t k0, uint32_t end) const
    {
        return k0 + KS > end || (ACROSS && width < W);
    }

    __device__ __forceinline__ i32x4 fix(int i, i32x4 v, uint32_t k0, uint32_t end) const
    {
        if (SHORT && (ACROSS ? rows < EPC : end < EPC)) return v;  // (read piece by piece)
        const int c = ACROSS ? (int)column(i) : (int)(k0 + at[i]), most = (int)(ACROSS ? width : end) - (int)EPC;
        const uint32_t by = c > most ? (uint32_t)(c - most) : 0;  // values to move by
        if (by & (EPC / 2)) v = i32x4{v[2], v[3], 0, 0};
        if (by & (EPC / 4)) v = i32x4{v[1], v[2], v[3], 0};
        if (ES == 2 && (by & 1u)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (int)((uint32_t)v[e] >> 16 | (e < 3 ? (uint32_t)v[e + 1] << 16 : 0u));
        }
        const bool none = by >= EPC || (ACROSS && k0 + at[i] >= end);
        return none ? i32x4{0, 0, 0, 0} : v;
    }

    __device__ __forceinline__ void put(uint8_t *lds, int i, i32x4 v) const
    {
        *reinterpret_cast<i32x4 *>(lds + (w * COPIES + i) * 1024 + (threadIdx.x & 63u) * 16) = v;
    }

    // fragment i of quarter q of the step: lane l has row (or column) l % 32,
    // the chunk 2 q + l / 32 of it
    __device__ __forceinline__ i32x4 fragment(const uint8_t *lds, int q, int i) const
    {
        if constexpr (!ACROSS) {
            return *reinterpret_cast<const i32x4 *>(lds + read[q] + i * 32 * kStepBytes);
        } else if constexpr (ES == 2) {
            const uint8_t *const from_ = lds + read[i] + q * 16 * RB;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(from_));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(from_ + 4 * RB));
            return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            i32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const int *>(lds + read[0] + (q * 8 + e) * RB + i * 128);
            return v;
        }
    }
};

// A workgroup's tile and its steps of K.
struct TilePlace {
    uint32_t m0, n0, split, s0, s1;
};

// Each of the 8 XCDs (workgroup ids taken in turn) gets a contiguous run of
// tiles, which go down 8 tile rows at a time, so that the operands an XCD
// reads at one time are few enough for its own L2.
__device__ __forceinline__ TilePlace place_of(const TileParams &p, uint32_t BM, uint32_t BN, uint32_t ks)
{
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
    const uint32_t all = (p.k + ks - 1) / ks;
    t.split = split;
    t.s0 = split * p.steps_per_split;
    t.s1 = t.s0 + p.steps_per_split < all ? t.s0 + p.steps_per_split : all;
    return t;
}

// Tiles of 64 FM x 64 FN outputs; four waves, 2 x 2, each with FM x FN
// fragments of 32 x 32. B's columns are the instruction's rows, so that a lane
// holds 4 neighbours of an output row (row l % 32, columns 8 a + 4 (l / 32) +
// 0 .. 3 for a < 4). A step's operands are copied to LDS by loads that bypass
// the registers: one step ahead into the other of two buffers, three steps
// ahead into four (DEEP), or, with 4 x 4 fragments, one to two steps ahead into
// five places of one operand's step each. One barrier per step, before its
// last quarter is multiplied: by then every wave has read all it needs of this
// step and its own copies of the next have landed.
//
// A step of 4 x 4 fragments reads 8 of them for 16 products, which LDS hides
// behind the products; its accumulators leave one wave for each SIMD, so the
// next fragments are read between the products of the present ones. 4,096 x
// 4,096 x 24,576 in bf16: cp_linear 571 to 610 us (1.35 to 1.44 PFLOP/s; the
// vendor library's product 542 to 628), cp_linear_dx 640 to 659 (618 to 722),
// cp_linear_dw 665 to 678 (709 to 824 for a 16-bit output). Its matrix units
// are busy 83% of the cycles (71 and 68% where operands are read across, at two LDS
// reads a fragment), at a clock that gives way to the power they draw: with
// zeros for operands the same launches take 458, 498 and 495 us.
//
// DIRECT needs both operands' rows to start on 16 bytes and to be whole
// chunks of 16 along their rows; others come by way of registers.
template <int DT, bool AX, bool BX, int OUT, int FM, int FN, bool DIRECT, bool DEEP = false, bool SHORT = false>
__global__ __launch_bounds__(256, FM *FN == 16 || DEEP ? 1 : FM *FN == 4 ? 2 : 4) void linear_tile(TileParams p)
{
    constexpr int BM = 64 * FM, BN = 64 * FN;
    typedef Operand<DT, AX, BM, FM, DIRECT, SHORT> OpA;
    typedef Operand<DT, BX, BN, FN, DIRECT, SHORT> OpB;
    constexpr bool IN_PLACE = FM * FN == 16;
    constexpr uint32_t STAGES = DEEP ? 4 : 2;
    constexpr bool FIVE = IN_PLACE && DIRECT;
    static_assert(!DEEP || (DIRECT && FM * FN < 16), "");
    constexpr int COPIES = OpA::COPIES + OpB::COPIES;
    constexpr uint32_t KS = OpA::KS;
    // an epilogue's slab of 32 rows of a wave has its place in one of them
    constexpr uint32_t SLAB_ROW = FN * 128 + 16;
    // (an array for each step: the compiler then knows which of them a copy
    // writes, and waits for no other)
    constexpr uint32_t BYTES = FIVE ? OpA::BYTES : OpA::BYTES + OpB::BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t l0[BYTES], l1[BYTES], l2[FIVE || DEEP ? BYTES : 16],
        l3[FIVE || DEEP ? BYTES : 16], l4[FIVE ? BYTES : 16];
    static_assert(FM == FN && 32 * SLAB_ROW <= OpA::BYTES, "");
    const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = w >> 1, wn = w & 1u;
    const TilePlace place = place_of(p, BM, BN, KS);
    const uint32_t s1 = place.s1, end = s1 * KS < p.k ? s1 * KS : p.k;  // of this split's part of K
    const OpA A(p.a, p.a_stride, place.m0, p.m, wm);
    const OpB B(p.b, p.b_stride, place.n0, p.n, wn);

    f32x16 acc[FM][FN];
    i32x4 a[2][FM], b[2][FN];
    // steps that are on their way in registers (not DIRECT)
    // (with four of them cp_linear_dx took 25.4 us against 24.9 for 1,000 x 1,030 from 2,050 in f16, 183 against
    // 158 for 2,001^3 in f32)
    constexpr int SETS = FM * FN == 16 ? 1 : 2;
    [[maybe_unused]] i32x4 ra[SETS][OpA::COPIES], rb[SETS][OpB::COPIES];
    [[maybe_unused]] const auto load = [&](int set, uint32_t s) {
#pragma unroll
        for (int i = 0; i < OpA::COPIES; ++i) ra[set][i] = A.load(i, s * KS, end);
#pragma unroll
        for (int i = 0; i < OpB::COPIES; ++i) rb[set][i] = B.load(i, s * KS, end);
    };
    [[maybe_unused]] const auto put = [&](int set, uint32_t s, uint8_t *as, uint8_t *bs) {
        if (A.may_reach(s * KS, end)) {
#pragma unroll
            for (int i = 0; i < OpA::COPIES; ++i) ra[set][i] = A.fix(i, ra[set][i], s * KS, end);
        }
        if (B.may_reach(s * KS, end)) {
#pragma unroll
            for (int i = 0; i < OpB::COPIES; ++i) rb[set][i] = B.fix(i, rb[set][i], s * KS, end);
        }
#pragma unroll
        for (int i = 0; i < OpA::COPIES; ++i) A.put(as, i, ra[set][i]);
#pragma unroll
        for (int i = 0; i < OpB::COPIES; ++i) B.put(bs, i, rb[set][i]);
    };

    const auto read = [&](const uint8_t *as, const uint8_t *bs, int q, int into) {
#pragma unroll
        for (int i = 0; i < FM; ++i) a[into][i] = A.fragment(as, q, i);
#pragma unroll
        for (int f = 0; f < FN; ++f) b[into][f] = B.fragment(bs, q, f);
    };
    // Step s, whose operands are in (as, bs) and the next one's in (an, bn); bb
    // held B's of the step before. Past the last step there are zeros.
    const auto step = [&](auto odd, uint32_t s, uint8_t *as, uint8_t *bs, uint8_t *an, uint8_t *bn, uint8_t *bb) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int cur = q & 1;
            const uint8_t *const ra_ = q < 3 ? as : an, *const rb_ = q < 3 ? bs : bn;
            const int rq = q < 3 ? q + 1 : 0;
            if (q == 3) {
                // this wave's LDS reads and its copies of the next step are done
                if constexpr (DIRECT)
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(FIVE ? OpA::COPIES : (STAGES - 2) * COPIES)
                                 : "memory");
                else  // (loads on their way are not waited for)
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            }
            if constexpr (!IN_PLACE) read(ra_, rb_, rq, cur ^ 1);
            if constexpr (!DIRECT) {
                constexpr int next = (odd + 1) % SETS;
                if (q == 1) put(next, s + 1, an, bn);
                if (q == 2) load(next, s + 1 + SETS);
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if constexpr (DIRECT && !FIVE) {
#pragma unroll
                    for (int i = f * (OpA::COPIES / FN); i < (f + 1) * (OpA::COPIES / FN); ++i) {
                        if (q == 0) B.copy(bb, i, (s - 1 + STAGES) * KS, end);
                        if (q == 3) A.copy(as, i, (s + STAGES) * KS, end);
                    }
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    if constexpr (IN_PLACE) {
                        // the next quarter's fragments and the copies one by one between the products
                        multiply_in_place<DT>(acc[i][f], b[cur][f], a[cur][i]);
                        const int slot = f * 4 + i;
                        if (slot == 2) b[cur ^ 1][0] = B.fragment(rb_, rq, 0);
                        else if (slot == 0) a[cur ^ 1][0] = A.fragment(ra_, rq, 0);
                        else if (slot < 10 && slot % 2 == 0) a[cur ^ 1][slot / 2 - 1] = A.fragment(ra_, rq, slot / 2 - 1);
                        else if (slot % 2 == 0) b[cur ^ 1][slot / 2 - 4] = B.fragment(rb_, rq, slot / 2 - 4);
                        if constexpr (FIVE) {
                            if (i == 1) {
                                if (q == 3) B.copy(as, f, (s + 2) * KS, end);
                                if (q == 0) B.copy(bn, 4 + f, (s + 1) * KS, end);
                                if (q == 1) A.copy(bb, f, (s + 2) * KS, end);
                                if (q == 2) A.copy(bb, 4 + f, (s + 2) * KS, end);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    } else {
                        acc[i][f] = multiply<DT>(b[cur][f], a[cur][i], acc[i][f]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // (while the first copies are on their way)
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                acc[i][f] = (f32x16)0.0f;
                if constexpr (IN_PLACE) asm volatile("" : "+a"(acc[i][f]));  // (once, not on each way past the loops)
            }
    };
    [[maybe_unused]] const auto copy_a = [&](uint8_t *as, uint32_t s) {
#pragma unroll
        for (int i = 0; i < OpA::COPIES; ++i) A.copy(as, i, s * KS, end);
    };
    [[maybe_unused]] const auto copy_b = [&](uint8_t *bs, uint32_t s) {
#pragma unroll
        for (int i = 0; i < OpB::COPIES; ++i) B.copy(bs, i, s * KS, end);
    };

    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    uint32_t s = place.s0;
    // (in the loops whole turns first: with a way out inside the turn the
    // compiler waits for copies that just began, as on the ways out)
    if constexpr (FIVE) {
        copy_a(l0, s);
        copy_b(l1, s);
        copy_a(l2, s + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) B.copy(l3, i, (s + 1) * KS, end);
        clear();
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(OpA::COPIES + 4) : "memory");
        read(l0, l1, 0, 0);
        for (; s + 5 <= s1; s += 5) {
            step(even, s, l0, l1, l2, l3, l4);
            step(even, s + 1, l2, l3, l4, l0, l1);
            step(even, s + 2, l4, l0, l1, l2, l3);
            step(even, s + 3, l1, l2, l3, l4, l0);
            step(even, s + 4, l3, l4, l0, l1, l2);
        }
        if (s < s1) {
            step(even, s, l0, l1, l2, l3, l4);
            if (s + 1 < s1) {
                step(even, s + 1, l2, l3, l4, l0, l1);
                if (s + 2 < s1) {
                    step(even, s + 2, l4, l0, l1, l2, l3);
                    if (s + 3 < s1) step(even, s + 3, l1, l2, l3, l4, l0);
                }
            }
        }
    } else if constexpr (DEEP) {
        uint8_t *const b0 = l0 + OpA::BYTES, *const b1 = l1 + OpA::BYTES, *const b2 = l2 + OpA::BYTES,
                *const b3 = l3 + OpA::BYTES;
        copy_a(l0, s);
        copy_b(b0, s);
        copy_a(l1, s + 1);
        copy_b(b1, s + 1);
        copy_a(l2, s + 2);
        copy_b(b2, s + 2);
        copy_a(l3, s + 3);
        clear();
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * COPIES + OpA::COPIES) : "memory");
        read(l0, b0, 0, 0);
        for (; s + 4 <= s1; s += 4) {
            step(even, s, l0, b0, l1, b1, b3);
            step(even, s + 1, l1, b1, l2, b2, b0);
            step(even, s + 2, l2, b2, l3, b3, b1);
            step(even, s + 3, l3, b3, l0, b0, b2);
        }
        if (s < s1) {
            step(even, s, l0, b0, l1, b1, b3);
            if (s + 1 < s1) {
                step(even, s + 1, l1, b1, l2, b2, b0);
                if (s + 2 < s1) step(even, s + 2, l2, b2, l3, b3, b1);
            }
        }
    } else {
        uint8_t *const b0 = l0 + OpA::BYTES, *const b1 = l1 + OpA::BYTES;
        if constexpr (DIRECT) {
            copy_a(l0, s);
            copy_b(b0, s);
            copy_a(l1, s + 1);
            clear();
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(OpA::COPIES) : "memory");
        } else {
            load(0, s);
            clear();
            put(0, s, l0, b0);
#pragma unroll
            for (uint32_t t = 1; t <= SETS; ++t) load(t % SETS, s + t);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        read(l0, b0, 0, 0);
        for (; s + 2 <= s1; s += 2) {
            step(even, s, l0, b0, l1, b1, b1);
            step(odd, s + 1, l1, b1, l0, b0, b0);
        }
        if (s < s1) step(even, s, l0, b0, l1, b1, b1);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // the copies past the end (zeros) are in LDS
    __syncthreads();                     // and every wave's last reads are done

    if constexpr (IN_PLACE) {
        settle();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) asm volatile("" : "+a"(acc[i][f]));
    }
    // by way of LDS, so that 8 neighbours meet in a lane and rows are written
    // in long pieces
    constexpr uint32_t HALF = FIVE ? 0 : OpA::BYTES;
    uint8_t *const slab = FIVE ? (w == 0 ? l0 : w == 1 ? l1 : w == 2 ? l2 : l3) : (w & 1u ? l1 : l0) + (w >> 1) * HALF;
    Epilogue e = p.e;
    if (p.part) e = Epilogue{};  // the sums alone, of 32 bits
    const Mask mask = mask_of(e.drop);
    constexpr uint32_t GROUPS = 4 * FN, ROWS = 64 / GROUPS;  // groups of 8 in a slab's row; rows at a time
    constexpr uint32_t TURNS = 32 / ROWS;
    const uint32_t r = lane & 31u, h = lane >> 5, group = lane % GROUPS, slab_row = lane / GROUPS;
    const uint32_t m_first = place.m0 + wm * FM * 32 + slab_row, n = place.n0 + wn * FN * 32 + group * 8;
    float bias[8];
    bias8<DT>(e, n, p.n, bias);  // (a lane's columns are the same in all rows)
    const auto take = [&](uint32_t t, float *o) {  // turn t of the slab
        const uint8_t *const at = slab + (t * ROWS + slab_row) * SLAB_ROW + group * 32;
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(at), hi = *reinterpret_cast<const f32x4 *>(at + 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            o[q] = lo[q];
            o[4 + q] = hi[q];
        }
    };
    constexpr uint32_t AHEAD = TURNS < 4 ? TURNS : 4;  // turns that the residual is read ahead
    typename Elem<OUT>::vec8 ahead[AHEAD];
    const auto look = [&](uint32_t turn) {
        const uint32_t m = m_first + turn * ROWS;
        return turn < FM * TURNS && m < p.m && n < p.n ? residual8<OUT>(e, m, n, p.n) : typename Elem<OUT>::vec8{};
    };
    if (e.residual) {
#pragma unroll
        for (uint32_t t = 0; t < AHEAD; ++t) ahead[t] = look(t);
    }
#pragma unroll 1
    for (uint32_t i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            if ((int)i != j) continue;
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4 *>(slab + r * SLAB_ROW + (32 * f + 8 * q + 4 * h) * 4) =
                        f32x4{acc[j][f][4 * q], acc[j][f][4 * q + 1], acc[j][f][4 * q + 2], acc[j][f][4 * q + 3]};
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (a wave's own: its LDS accesses stay in order)
        if (!e.residual) {
            // (apart: where loads are waited for, so are the stores before them)
#pragma unroll 1
            for (uint32_t t = 0; t < TURNS; ++t) {
                float o[8];
                take(t, o);
                const uint32_t m = m_first + (i * TURNS + t) * ROWS;
                if (m < p.m && n < p.n) {
                    if (p.part) store8<kF32>(p.part + ((uint64_t)place.split * p.m + m) * p.n, n, p.n, o);
                    else finish8<OUT>(e, mask, m, n, p.n, o, bias, typename Elem<OUT>::vec8{});
                }
            }
        } else {
#pragma unroll 1
            for (uint32_t t = 0; t < TURNS; t += AHEAD) {
#pragma unroll
                for (uint32_t u = 0; u < AHEAD; ++u) {
                    float o[8];
                    take(t + u, o);
                    const uint32_t m = m_first + (i * TURNS + t + u) * ROWS;
                    if (m < p.m && n < p.n) finish8<OUT>(e, mask, m, n, p.n, o, bias, ahead[u]);
                    ahead[u] = look(i * TURNS + t + u + AHEAD);
                }
            }
        }
        asm volatile("" ::: "memory");
    }
}

// The splits' sums, joined in order, through the epilogue (none: zeros).
template <int DT, int OUT>
__global__ __launch_bounds__(256) void join_parts(const float *__restrict__ part, uint32_t splits, uint32_t n8,
                                                  uint32_t m, uint32_t n, Epilogue e)
{
    const Mask mask = mask_of(e.drop);
    const uint64_t count = (uint64_t)m * n8;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (uint64_t)gridDim.x * 256) {
        const uint32_t row = (uint32_t)(i / n8), c = (uint32_t)(i - (uint64_t)row * n8) * 8;
        float f[8] = {};
        for (uint32_t s = 0; s < splits; ++s) {
            const auto v = load8<kF32>(part + ((uint64_t)s * m + row) * n, c, n);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] += v[q];
        }
        float bias[8];
        bias8<DT>(e, c, n, bias);
        finish8<OUT>(e, mask, row, c, n, f, bias, residual8<OUT>(e, row, c, n));
    }
}

// How a product is cut: tiles of 64 f x 64 f, and splits of K.
struct Cut {
    int f;
    uint32_t splits, steps_per_split;
};

// How an operand's rows lie: whole chunks of 16 bytes, at any alignment, or
// shorter than a chunk.
enum Rows { kWhole = 0, kOdd = 1, kShort = 2 };

Cut cut_of(uint64_t m, uint64_t n, uint64_t k, int dtype, Rows rows)
{
    // us, fitted to measured times of every form: a step of a workgroup that has
    // its compute unit to itself, and of each where there are more for a unit;
    // launch, first loads and epilogue; each further workgroup of a unit. Large
    // tiles read less, small ones and splits fill the chip: 4,096 x 4,096 x
    // 24,576 takes 571 us with f = 4 and 779 with 2, 2,000^3 takes 35, 26 and 46
    // with 1, 2 and 4, 256 x 1,024 x 1,024 takes 6.5, 11 and 28; 64 x 4,096 x
    // 24,576 with f = 1 takes 121, 72, 53 and 50 in 1, 2, 4 and 8 splits, 8,192 x
    // 1,024 x 512 with f = 2 takes 15 whole and 41 in 2.
    struct Kind { int f; double alone, each, ends, more; };
    static const Kind narrow[] = {{1, 0.15, 0.20, 4.7, 0.6}, {2, 0.29, 0.51, 7.4, 2.8}, {4, 1.52, 1.52, 18.0, 20.0}};
    static const Kind odd[] = {{1, 0.46, 0.38, 4.8, 0.8}, {2, 0.80, 0.75, 7.5, 4.0}, {4, 2.0, 1.85, 22.0, 18.0}};
    static const Kind wide[] = {{1, 0.43, 0.58, 4.6, 1.0}, {2, 1.82, 2.12, 8.0, 3.6}};
    const Kind *const kinds = dtype == kF32 ? wide : rows == kWhole ? narrow : odd;
    const uint32_t steps = (uint32_t)div_up(k * dtype_bytes(dtype), kStepBytes);
    Cut best{};
    double least = 0;
    for (int q = 0; q < (dtype == kF32 ? 2 : 3); ++q) {
        const Kind &t = kinds[q];
        if (t.f > 1 && rows == kShort) continue;
        const uint64_t tiles = div_up(m, 64u * t.f) * div_up(n, 64u * t.f);
        for (uint32_t want = 1; want <= 16; want *= 2) {
            const uint32_t per = (uint32_t)div_up(steps, want), splits = (uint32_t)div_up(steps, per);
            if (want > 1 && (per < 4 || splits != want)) continue;
            const uint64_t wgs = tiles * splits;
            if (wgs >= (1u << 24)) continue;  // a launch has fewer than 2^32 threads
            // workgroups of a compute unit: between the mean and the most
            const double load = 0.5 * ((double)div_up(wgs, 256) + wgs / 256.0);
            const double step = t.alone > load * t.each ? t.alone : load * t.each;
            double cost = t.ends + per * step + (load > 1 ? t.more * (load - 1) : 0);
            if (splits > 1) cost += 3.4 + 0.13e-6 * 4 * (double)m * n * (splits + 1);
            if (best.f == 0 || cost < least) {
                least = cost;
                best = Cut{t.f, splits, per};
            }
        }
    }
    return best;
}

inline uint64_t workspace_of(const Cut &c, uint64_t m, uint64_t n) { return c.splits > 1 ? 4ull * c.splits * m * n : 0; }

template <int DT, int OUT>
hipError_t join(const LinearArgs &g, uint32_t splits)
{
    const uint64_t n8 = div_up(g.n, 8), wgs = div_up(g.m * n8, 256);
    join_parts<DT, OUT><<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, g.stream>>>(
        (const float *)g.workspace, splits, (uint32_t)n8, (uint32_t)g.m, (uint32_t)g.n, g.e);
    return hipGetLastError();
}

// Whether an operand's rows can be copied to LDS in chunks of 16 bytes.
inline bool whole_chunks(const void *p, uint64_t stride_bytes, uint64_t row_bytes)
{
    return ((uintptr_t)p | stride_bytes | row_bytes) % 16 == 0;
}

template <int DT, bool AX, bool BX, int OUT>
hipError_t launch_linear(const LinearArgs &g)
{
    if (g.k == 0) return join<DT, OUT>(g, 0);
    constexpr uint64_t es = dtype_bytes(DT);
    const uint64_t a_row = (AX ? g.m : g.k) * es, b_row = (BX ? g.n : g.k) * es;
    const bool direct = whole_chunks(g.a, g.a_stride * es, a_row) && whole_chunks(g.b, g.b_stride * es, b_row);
    const Rows rows = direct ? kWhole : a_row < 16 || b_row < 16 ? kShort : kOdd;
    const Cut c = cut_of(g.m, g.n, g.k, DT, rows);
    TileParams p{};
    p.a = g.a;
    p.b = g.b;
    p.a_stride = g.a_stride * es;
    p.b_stride = g.b_stride * es;
    p.m = (uint32_t)g.m;
    p.n = (uint32_t)g.n;
    p.k = (uint32_t)g.k;
    p.tiles_m = (uint32_t)div_up(g.m, 64u * c.f);
    p.tiles_n = (uint32_t)div_up(g.n, 64u * c.f);
    p.steps_per_split = c.steps_per_split;
    p.part = c.splits > 1 ? (float *)g.workspace : nullptr;
    p.e = g.e;
    const uint32_t blocks = p.tiles_m * p.tiles_n * c.splits;
    if (direct) {
        // four steps' buffers where no compute unit has two workgroups: 64 x 4,096
        // x 24,576 in 4 splits 53 us, with two 82; 2,000^3 26 and 31. Where one
        // has, the other hides the copies, and twice the LDS keeps it out: 8,192 x
        // 1,024 x 512 takes 19 us with four and 15 with two.
        const bool deep = blocks <= 256;
        if (c.f == 1 && deep) linear_tile<DT, AX, BX, OUT, 1, 1, true, true><<<blocks, 256, 0, g.stream>>>(p);
        else if (c.f == 1) linear_tile<DT, AX, BX, OUT, 1, 1, true><<<blocks, 256, 0, g.stream>>>(p);
        else if (c.f == 2 && deep) linear_tile<DT, AX, BX, OUT, 2, 2, true, true><<<blocks, 256, 0, g.stream>>>(p);
        else if (c.f == 2) linear_tile<DT, AX, BX, OUT, 2, 2, true><<<blocks, 256, 0, g.stream>>>(p);
        else if constexpr (DT != kF32) linear_tile<DT, AX, BX, OUT, 4, 4, true><<<blocks, 256, 0, g.stream>>>(p);
    } else {
        // (a form of its own: with a way around each load the compiler waits for later loads too. 1,000 x
        // 1,030 from 2,050 in f16 25 us against 28, 33 x 8,001 from 1,001 11 against 14)
        if (rows == kShort) linear_tile<DT, AX, BX, OUT, 1, 1, false, false, true><<<blocks, 256, 0, g.stream>>>(p);
        else if (c.f == 1) linear_tile<DT, AX, BX, OUT, 1, 1, false><<<blocks, 256, 0, g.stream>>>(p);
        else if (c.f == 2) linear_tile<DT, AX, BX, OUT, 2, 2, false><<<blocks, 256, 0, g.stream>>>(p);
        else if constexpr (DT != kF32) linear_tile<DT, AX, BX, OUT, 4, 4, false><<<blocks, 256, 0, g.stream>>>(p);
    }
    if (c.splits > 1) return join<DT, OUT>(g, c.splits);
    return hipGetLastError();
}

}  // namespace

}  // namespace cpk
