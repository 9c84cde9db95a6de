// cp_embed.hip - the uncompressed row table: lookup, plan of a batch's
// gradient (a stable sort of its ids), gradient.
//
//   lookup:   out[j] = scale * table[ids[j]]
//   gradient: grad[r] = scale * sum over {j: ids[j] = r} of dout[j]
//
// All three move data and are bound by it. The gradient's sums run over the
// lookups of a row in batch order, which the sort keeps, so that equal calls
// give equal bits (an atomic sum would not).
#include "cp_ops_internal.h"

namespace cpk {

namespace {

constexpr uint32_t kMaxBlocks = 1u << 22;  // workgroups of one launch, at most

// Lanes that share a row of d elements, 8 elements each: a power of two.
int row_lanes_log2(uint64_t d)
{
    int s = 0;
    while (s < 6 && (8ull << s) < d) ++s;
    return s;
}

// ---------------------------------------------------------------- lookup

// 2^gs lanes take a row, 8 elements each per step; a thread has U rows'
// loads in flight.
template <int TI, int TO, int U>
__global__ __launch_bounds__(256) void lookup_rows(const typename Elem<TI>::raw *__restrict__ table, uint64_t rows,
                                                   uint32_t d, uint64_t stride, const int64_t *__restrict__ ids,
                                                   uint32_t n, float scale, typename Elem<TO>::raw *__restrict__ out,
                                                   int32_t *__restrict__ bad_id, int gs)
{
    const uint32_t lane = threadIdx.x & ((1u << gs) - 1u);
    const uint32_t per = 256u >> gs;
    const uint64_t j0 = (uint64_t)blockIdx.x * (U * per) + (threadIdx.x >> gs);
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = j0 + u * per < n ? ids[j0 + u * per] : -1;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (id[u] >= 0 && (uint64_t)id[u] >= rows) {
            bad = true;
            id[u] = -1;
        }
    }
    if (bad && bad_id) *bad_id = 1;
    for (uint32_t c = lane * 8u; c < d; c += 8u << gs) {
        typename Elem<TI>::vec8 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (id[u] >= 0) v[u] = load8<TI>(table + (uint64_t)id[u] * stride, c, d);
            else v[u] = (typename Elem<TI>::raw)0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u * per >= n) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = id[u] >= 0 ? Elem<TI>::get(v[u][e]) * scale : 0.0f;
            store8<TO, true>(out + (j0 + u * per) * d, c, d, f);
        }
    }
}

template <int TI, int TO>
hipError_t launch_lookup(const EmbedLookupArgs &a)
{
    typedef typename Elem<TI>::raw RI;
    typedef typename Elem<TO>::raw RO;
    const int gs = row_lanes_log2(a.d);
    const uint32_t per = 256u >> gs;
    // four rows in flight per thread once that still leaves the chip several
    // workgroups per compute unit
    const bool four = a.n >= 4ull * per * 2048;
    const uint64_t step = (uint64_t)kMaxBlocks * per * (four ? 4 : 1);
    for (uint64_t j = 0; j < a.n; j += step) {  // a launch has fewer than 2^32 threads
        const uint32_t n = (uint32_t)(a.n - j < step ? a.n - j : step);
        RO *out = (RO *)a.out + j * a.d;
        if (four)
            lookup_rows<TI, TO, 4><<<(uint32_t)div_up(n, 4ull * per), 256, 0, a.stream>>>(
                (const RI *)a.table, a.rows, (uint32_t)a.d, a.row_stride, a.ids + j, n, a.scale, out, a.bad_id, gs);
        else
            lookup_rows<TI, TO, 1><<<(uint32_t)div_up(n, per), 256, 0, a.stream>>>(
                (const RI *)a.table, a.rows, (uint32_t)a.d, a.row_stride, a.ids + j, n, a.scale, out, a.bad_id, gs);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------------ plan

constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortRounds = 4;                            // keys per thread
constexpr uint32_t kSortTile = kSortThreads * kSortRounds;     // keys per workgroup
constexpr int kDigitBits = 9;                                  // bits sorted by one pass, at most
constexpr uint32_t kDigits = 1u << kDigitBits;
static_assert(kDigits <= kSortThreads, "a thread per digit");

// The sort key of an id: the id, or `rows` (above every valid key) when it
// is outside [0, rows).
template <typename K>
__device__ __forceinline__ K key_of(int64_t id, uint64_t rows)
{
    return (uint64_t)id < rows ? (K)id : (K)rows;
}

// Lanes of the wave whose digit (of `bits` bits) equals this lane's, among
// the lanes of `valid`.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, uint64_t valid)
{
    uint64_t m = valid;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1u);
        m &= ((digit >> b) & 1u) ? set : ~set;
    }
    return m;
}

__device__ __forceinline__ uint64_t lanes_below() { return (1ull << (threadIdx.x & 63u)) - 1ull; }

// Inclusive prefix sum over a workgroup of WAVES waves; *total = all.
template <int WAVES>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t *wave_sum, uint32_t *total)
{
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const uint32_t up = (uint32_t)__shfl_up((int)v, (unsigned)k, 64);
        if (lane >= (uint32_t)k) v += up;
    }
    if (lane == 63) wave_sum[w] = v;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
        if (q < (int)w) before += wave_sum[q];
        all += wave_sum[q];
    }
    __syncthreads();
    *total = all;
    return before + v;
}

// hist[digit][tile] = keys of the tile with that digit.
template <typename K, bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count(const int64_t *__restrict__ ids, uint64_t rows,
                                                           const K *__restrict__ keys, uint32_t n, int shift,
                                                           uint32_t digits, uint32_t ntiles,
                                                           uint32_t *__restrict__ hist)
{
    __shared__ uint32_t cnt[kDigits];
    if (threadIdx.x < digits) cnt[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * kSortTile + threadIdx.x;
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * kSortThreads;
        if (i < n) {
            K k;
            if constexpr (FIRST) k = key_of<K>(ids[i], rows);
            else k = keys[i];
            atomicAdd(&cnt[(uint32_t)(k >> shift) & (digits - 1u)], 1u);
        }
    }
    __syncthreads();
    if (threadIdx.x < digits) hist[(uint64_t)threadIdx.x * ntiles + blockIdx.x] = cnt[threadIdx.x];
}

// Per digit: hist[digit][tile] becomes the count of the tiles before it,
// totals[digit] the count of all.
__global__ __launch_bounds__(256) void sort_scan(uint32_t *__restrict__ hist, uint32_t ntiles,
                                                 uint32_t *__restrict__ totals)
{
    __shared__ uint32_t wave_sum[4];
    uint32_t *const h = hist + (uint64_t)blockIdx.x * ntiles;
    uint32_t run = 0;
    for (uint32_t t0 = 0; t0 < ntiles; t0 += 256) {
        const uint32_t t = t0 + threadIdx.x;
        const uint32_t v = t < ntiles ? h[t] : 0;
        uint32_t all;
        const uint32_t incl = block_prefix<4>(v, wave_sum, &all);
        if (t < ntiles) h[t] = run + incl - v;
        run += all;
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// Each key to its place: the keys of smaller digits, the same digit's in
// earlier tiles, in earlier waves' parts of this tile, and in this wave
// before it. Wave w has keys [w, w + 1) * 64 * kSortRounds of the tile.
template <typename K, bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_scatter(const int64_t *__restrict__ ids, uint64_t rows,
                                                             const K *__restrict__ keys,
                                                             const int32_t *__restrict__ vals, uint32_t n, int shift,
                                                             int bits, uint32_t ntiles,
                                                             const uint32_t *__restrict__ hist,
                                                             const uint32_t *__restrict__ totals,
                                                             K *__restrict__ keys_out, int32_t *__restrict__ vals_out)
{
    __shared__ uint32_t cnt[kSortWaves][kDigits];
    __shared__ uint32_t wave_sum[kSortWaves];
    const uint32_t digits = 1u << bits;
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
    for (uint32_t i = threadIdx.x; i < kSortWaves * kDigits; i += kSortThreads) (&cnt[0][0])[i] = 0;
    const uint32_t base = blockIdx.x * kSortTile + w * (64 * kSortRounds) + lane;
    K key[kSortRounds];
    int32_t val[kSortRounds];
    uint32_t rank[kSortRounds];
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * 64;
        key[r] = 0;
        val[r] = 0;
        if (i < n) {
            if constexpr (FIRST) {
                key[r] = key_of<K>(ids[i], rows);
                val[r] = (int32_t)i;
            } else {
                key[r] = keys[i];
                val[r] = vals[i];
            }
        }
    }
    uint32_t before = 0, total = 0;
    if (threadIdx.x < digits) {
        before = hist[(uint64_t)threadIdx.x * ntiles + blockIdx.x];
        total = totals[threadIdx.x];
    }
    uint32_t all;
    before += block_prefix<kSortWaves>(total, wave_sum, &all) - total;  // holds the barrier for cnt too
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        const bool in = base + r * 64 < n;
        const uint32_t digit = (uint32_t)(key[r] >> shift) & (digits - 1u);
        const uint64_t peers = same_digit(digit, bits, __ballot(in));
        const uint32_t prev = cnt[w][digit];
        rank[r] = prev + (uint32_t)__popcll(peers & lanes_below());
        __builtin_amdgcn_wave_barrier();
        if (in && (peers & lanes_below()) == 0) cnt[w][digit] = prev + (uint32_t)__popcll(peers);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (threadIdx.x < digits) {
        uint32_t run = before;
#pragma unroll
        for (uint32_t q = 0; q < kSortWaves; ++q) {
            const uint32_t c = cnt[q][threadIdx.x];
            cnt[q][threadIdx.x] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        if (base + r * 64 < n) {
            const uint32_t p = cnt[w][(uint32_t)(key[r] >> shift) & (digits - 1u)] + rank[r];
            keys_out[p] = key[r];
            vals_out[p] = val[r];
        }
    }
}

// tile_heads[tile] = how many of its keys begin a row's run.
template <typename K>
__global__ __launch_bounds__(kSortThreads) void count_heads(const K *__restrict__ keys, uint64_t rows, uint32_t n,
                                                            uint32_t *__restrict__ tile_heads)
{
    __shared__ uint32_t sum;
    if (threadIdx.x == 0) sum = 0;
    __syncthreads();
    uint32_t c = 0;
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        const uint32_t i = blockIdx.x * kSortTile + r * kSortThreads + threadIdx.x;
        bool head = false;
        if (i < n) {
            const K k = keys[i];
            head = k < rows && (i == 0 || keys[i - 1] != k);
        }
        c += (uint32_t)__popcll(__ballot(head));
    }
    if ((threadIdx.x & 63u) == 0) atomicAdd(&sum, c);
    __syncthreads();
    if (threadIdx.x == 0) tile_heads[blockIdx.x] = sum;
}

template <typename K>
__global__ __launch_bounds__(kSortThreads) void write_runs(const K *__restrict__ keys, uint64_t rows, uint32_t n,
                                                           const uint32_t *__restrict__ tile_heads,
                                                           int32_t *__restrict__ slot, int64_t *__restrict__ unique,
                                                           int32_t *__restrict__ starts, int64_t *__restrict__ count)
{
    __shared__ uint32_t wave_sum[kSortWaves];
    uint32_t mine = 0, base, all;
    for (uint32_t t = threadIdx.x; t < blockIdx.x; t += kSortThreads) mine += tile_heads[t];
    (void)block_prefix<kSortWaves>(mine, wave_sum, &base);
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
        const uint32_t i = blockIdx.x * kSortTile + r * kSortThreads + threadIdx.x;
        const bool in = i < n;
        const K k = in ? keys[i] : (K)rows;
        const bool valid = in && k < rows;
        const bool head = valid && (i == 0 || keys[i - 1] != k);
        const uint32_t u = base + block_prefix<kSortWaves>(head ? 1u : 0u, wave_sum, &all) - 1u;
        base += all;
        if (valid) slot[i] = (int32_t)u;
        if (head) {
            unique[u] = (int64_t)k;
            starts[u] = (int32_t)i;
        }
        if (valid && (i + 1 == n || keys[i + 1] >= rows)) {  // the last lookup that takes part
            *count = (int64_t)u + 1;
            starts[u + 1] = (int32_t)i + 1;
        }
        if (in && i == 0 && !valid) {
            *count = 0;
            starts[0] = 0;
        }
    }
}

__global__ void empty_plan(int32_t *starts, int64_t *count)
{
    *count = 0;
    starts[0] = 0;
}

struct PlanLayout {
    uint64_t keys0, keys1, vals0, vals1, hist, totals, heads, total;
};

PlanLayout plan_layout(uint64_t n, uint64_t rows)
{
    const uint64_t kb = rows < (1ull << 32) ? 4 : 8, tiles = div_up(n, kSortTile);
    PlanLayout L{};
    uint64_t off = 0;
    const auto take = [&off](uint64_t bytes) {
        const uint64_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L.keys0 = take(kb * n);
    L.keys1 = take(kb * n);
    L.vals0 = take(4 * n);
    L.vals1 = take(4 * n);
    L.hist = take(4 * kDigits * tiles);
    L.totals = take(4 * kDigits);
    L.heads = take(4 * tiles);
    L.total = off;
    return L;
}

template <typename K>
hipError_t launch_plan(const EmbedPlanArgs &a)
{
    const PlanLayout L = plan_layout(a.n, a.rows);
    const uint32_t n = (uint32_t)a.n, ntiles = (uint32_t)div_up(a.n, kSortTile);
    uint32_t *const hist = reinterpret_cast<uint32_t *>(a.workspace + L.hist);
    uint32_t *const totals = reinterpret_cast<uint32_t *>(a.workspace + L.totals);
    uint32_t *const heads = reinterpret_cast<uint32_t *>(a.workspace + L.heads);
    K *keys[2] = {reinterpret_cast<K *>(a.workspace + L.keys0), reinterpret_cast<K *>(a.workspace + L.keys1)};
    int32_t *vals[2] = {reinterpret_cast<int32_t *>(a.workspace + L.vals0),
                        reinterpret_cast<int32_t *>(a.workspace + L.vals1)};
    int key_bits = 1;
    while (key_bits < 64 && (a.rows >> key_bits) != 0) ++key_bits;
    const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
    const int bits = (key_bits + passes - 1) / passes;
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        const K *in = keys[(p + 1) & 1];
        K *out = keys[p & 1];
        int32_t *vout = p + 1 == passes ? a.order : vals[p & 1];
        if (p == 0) {
            sort_count<K, true><<<ntiles, kSortThreads, 0, a.stream>>>(a.ids, a.rows, nullptr, n, shift, 1u << bits,
                                                                       ntiles, hist);
            sort_scan<<<1u << bits, 256, 0, a.stream>>>(hist, ntiles, totals);
            sort_scatter<K, true><<<ntiles, kSortThreads, 0, a.stream>>>(a.ids, a.rows, nullptr, nullptr, n, shift,
                                                                         bits, ntiles, hist, totals, out, vout);
        } else {
            sort_count<K, false><<<ntiles, kSortThreads, 0, a.stream>>>(nullptr, a.rows, in, n, shift, 1u << bits,
                                                                        ntiles, hist);
            sort_scan<<<1u << bits, 256, 0, a.stream>>>(hist, ntiles, totals);
            sort_scatter<K, false><<<ntiles, kSortThreads, 0, a.stream>>>(nullptr, a.rows, in, vals[(p + 1) & 1], n,
                                                                          shift, bits, ntiles, hist, totals, out, vout);
        }
    }
    const K *sorted = keys[(passes - 1) & 1];
    count_heads<K><<<ntiles, kSortThreads, 0, a.stream>>>(sorted, a.rows, n, heads);
    write_runs<K><<<ntiles, kSortThreads, 0, a.stream>>>(sorted, a.rows, n, heads, a.slot, a.unique, a.starts, a.count);
    return hipGetLastError();
}

// -------------------------------------------------------------- gradient

// Sorted lookups per chunk: a chunk is summed by one group of lanes.
uint32_t grad_chunk(uint64_t n)
{
    uint32_t c = 8;
    while (c < 64 && n / c > 4096) c <<= 1;
    return c;
}

// A row with more than kLongChunks chunks' worth of lookups is summed by
// chunks (partial sums, joined afterwards); any other by the chunk in which
// its run begins.
constexpr uint32_t kLongChunks = 4;

// Row s's sum goes to grad row `rows ? unique[s] : s`.
__device__ __forceinline__ float *grad_row(float *grad, const int64_t *unique, uint64_t rows, int32_t s, uint64_t d)
{
    return grad + (rows ? (uint64_t)unique[s] : (uint64_t)(uint32_t)s) * d;
}

// Chunk c: sorted lookups [c C, c C + C). Its group of 2^gs lanes sums the
// runs that begin in it, reading past its end for a short last run, and its
// own part of a long run into partial[2 c] (begun in an earlier chunk) or
// partial[2 c + 1] (begun in this one). blockIdx.y: a slice of 8 << gs columns.
template <int DT>
__global__ __launch_bounds__(256) void grad_chunks(const int32_t *__restrict__ order, const int32_t *__restrict__ slot,
                                                   const int64_t *__restrict__ unique,
                                                   const int32_t *__restrict__ starts,
                                                   const int64_t *__restrict__ count, uint64_t rows,
                                                   const typename Elem<DT>::raw *__restrict__ dout, uint32_t d,
                                                   uint64_t stride, float scale, float *__restrict__ grad,
                                                   float *__restrict__ partial, uint32_t C, int gs)
{
    constexpr int U = 8;  // rows' loads in flight
    const uint32_t lane = threadIdx.x & ((1u << gs) - 1u);
    const uint32_t chunk = blockIdx.x * (256u >> gs) + (threadIdx.x >> gs);
    const uint32_t c = (blockIdx.y * (1u << gs) + lane) * 8u;
    const uint64_t c0 = (uint64_t)chunk * C;
    const int32_t nrows = (int32_t)*count;
    const uint32_t nv = (uint32_t)starts[nrows];
    if (c0 >= nv) return;
    const uint32_t L = kLongChunks * C;
    uint32_t lo = (uint32_t)c0, hi = (uint32_t)(c0 + C < nv ? c0 + C : nv);
    // the run that covers the first lookup, and the one that covers the last
    const int32_t sf = slot[lo], sl = slot[hi - 1];
    const uint32_t fb = (uint32_t)starts[sf], fe = (uint32_t)starts[sf + 1];
    const uint32_t lb = (uint32_t)starts[sl], le = (uint32_t)starts[sl + 1];
    const bool first_long = fe - fb > L, last_long = le - lb > L;
    const bool from_before = fb < lo;
    if (from_before && !first_long) lo = fe;  // an earlier chunk sums it
    if (!last_long) hi = le;
    if (lo >= hi || c >= d) return;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    for (uint32_t i = lo; i < hi; i += U) {
        int32_t s[U + 1];
        typename Elem<DT>::vec8 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t iu = i + u < hi ? i + u : hi - 1;
            const int32_t t = order[iu];
            s[u] = slot[iu];
            v[u] = load8<DT>(dout + (uint64_t)(uint32_t)t * stride, c, d);
        }
        s[U] = i + U < hi ? slot[i + U] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u < hi) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += Elem<DT>::get(v[u][e]);
                if (i + u + 1 == hi || s[u + 1] != s[u]) {
                    float *row;
                    if (s[u] == sf && first_long) row = partial + (2ull * chunk + (from_before ? 0 : 1)) * d;
                    else if (s[u] == sl && last_long) row = partial + (2ull * chunk + 1) * d;
                    else row = grad_row(grad, unique, rows, s[u], d);
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] = acc[e] * scale;
                        acc[e] = 0.0f;
                    }
                    store8<kF32>(row, c, d, f);
                }
            }
        }
    }
}

// The long runs: a run that begins in a chunk of this workgroup and spans more than
// kLongChunks chunks' worth is the sum of its partial sums. 32 lanes take
// 128 columns; the workgroup's 8 such groups every eighth partial sum.
__global__ __launch_bounds__(256) void grad_join(const int32_t *__restrict__ slot, const int64_t *__restrict__ unique,
                                                 const int32_t *__restrict__ starts,
                                                 const int64_t *__restrict__ count, uint64_t rows, uint32_t d,
                                                 const float *__restrict__ partial, float *__restrict__ grad,
                                                 uint32_t C)
{
    __shared__ float sums[8][128];
    const uint32_t nv = (uint32_t)starts[*count];
    const uint32_t lane = threadIdx.x & 31u, g = threadIdx.x >> 5;
    const uint32_t col = blockIdx.y * 128u + lane * 4u;
    for (uint32_t chunk = blockIdx.x; (uint64_t)chunk * C < nv; chunk += gridDim.x) {
        const uint64_t c0 = (uint64_t)chunk * C;
        const uint32_t end = (uint32_t)(c0 + C < nv ? c0 + C : nv);
        const int32_t s = slot[end - 1];
        const uint32_t b = (uint32_t)starts[s], e = (uint32_t)starts[s + 1];
        if (e - b <= kLongChunks * C || b < c0) continue;
        const uint32_t parts = (e - 1) / C - chunk + 1;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (uint32_t k = g; k < parts; k += 8) {  // part 0 is this chunk's
            const float *p = partial + (2ull * (chunk + k) + (k == 0 ? 1 : 0)) * d;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] += col + q < d ? p[col + q] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[g][lane * 4 + q] = acc[q];
        __syncthreads();
        if (threadIdx.x < 128) {
            const uint32_t cc = blockIdx.y * 128u + threadIdx.x;
            float t = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) t += sums[q][threadIdx.x];
            if (cc < d) grad_row(grad, unique, rows, s, d)[cc] = t;
        }
        __syncthreads();
    }
}

// Zeros in the rows of the whole gradient that no lookup has. A workgroup
// takes R rows, marks those that appear in unique, and fills the others.
constexpr uint32_t kZeroRowsMax = 1024;

__device__ __forceinline__ uint32_t lower_bound(const int64_t *__restrict__ a, uint32_t n, int64_t v)
{
    // the wave probes 64 places at a time: three rounds cover 2^18 entries
    uint32_t lo = 0, hi = n;  // a[lo - 1] < v <= a[hi]
    while (lo < hi) {
        const uint32_t step = (hi - lo + 63) / 64;
        const uint64_t at = (uint64_t)lo + (uint64_t)(threadIdx.x & 63u) * step;
        const bool less = at < hi && a[at] < v;
        const uint32_t k = (uint32_t)__popcll(__ballot(less));  // a prefix of the lanes
        if (k == 0) return lo;
        const uint64_t nlo = (uint64_t)lo + (uint64_t)(k - 1) * step + 1;
        const uint64_t nhi = (uint64_t)lo + (uint64_t)k * step;
        lo = (uint32_t)nlo;
        hi = (uint32_t)(nhi < hi ? nhi : hi);
    }
    return lo;
}

template <int W>
__global__ __launch_bounds__(256) void grad_zero(const int64_t *__restrict__ unique,
                                                 const int64_t *__restrict__ count, uint64_t rows, uint32_t d,
                                                 float *__restrict__ grad, uint32_t R)
{
    __shared__ uint32_t seen[kZeroRowsMax / 32];
    if (threadIdx.x < kZeroRowsMax / 32) seen[threadIdx.x] = 0;
    const uint64_t r0 = (uint64_t)blockIdx.x * R;
    const uint32_t nr = (uint32_t)(rows - r0 < R ? rows - r0 : R);
    const uint32_t nu = (uint32_t)*count;
    const uint32_t u0 = lower_bound(unique, nu, (int64_t)r0);
    __syncthreads();
    for (uint32_t u = u0 + threadIdx.x; u < nu; u += 256) {
        const uint64_t r = (uint64_t)unique[u] - r0;
        if (r >= nr) break;
        atomicOr(&seen[r >> 5], 1u << (r & 31u));
    }
    __syncthreads();
    const uint32_t per = d / W;  // W divides d
    for (uint32_t f = threadIdx.x; f < nr * per; f += 256) {
        const uint32_t r = f / per;
        if (!((seen[r >> 5] >> (r & 31u)) & 1u)) {
            float *p = grad + (r0 + r) * d + (uint64_t)(f - r * per) * W;
            if constexpr (W == 4) {
                typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
                __builtin_nontemporal_store((v4)0.0f, reinterpret_cast<v4 *>(p));
            } else {
                __builtin_nontemporal_store(0.0f, p);
            }
        }
    }
}

template <int DT>
hipError_t launch_grad(const EmbedGradArgs &a)
{
    const uint32_t C = grad_chunk(a.n), d = (uint32_t)a.d;
    const uint32_t chunks = (uint32_t)div_up(a.n, C);
    const int gs = row_lanes_log2(a.d);
    float *const partial = reinterpret_cast<float *>(a.workspace);
    if (a.rows) {
        uint32_t R = 65536u / d;  // about 256 KiB of gradient per workgroup
        R = R < 1 ? 1 : R > kZeroRowsMax ? kZeroRowsMax : R;
        const uint32_t blocks = (uint32_t)div_up(a.rows, R);
        if (d % 4 == 0) grad_zero<4><<<blocks, 256, 0, a.stream>>>(a.unique, a.count, a.rows, d, a.grad, R);
        else grad_zero<1><<<blocks, 256, 0, a.stream>>>(a.unique, a.count, a.rows, d, a.grad, R);
    }
    if (a.n == 0) return hipGetLastError();
    grad_chunks<DT><<<dim3((uint32_t)div_up(chunks, 256u >> gs), (uint32_t)div_up(a.d, 8ull << gs)), 256, 0,
                      a.stream>>>(a.order, a.slot, a.unique, a.starts, a.count, a.rows,
                                  (const typename Elem<DT>::raw *)a.dout, d, a.stride, a.scale, a.grad, partial, C, gs);
    if (a.n > (uint64_t)kLongChunks * C)
        grad_join<<<dim3(chunks < 65536u ? chunks : 65536u, (uint32_t)div_up(a.d, 128)), 256, 0, a.stream>>>(
            a.slot, a.unique, a.starts, a.count, a.rows, d, partial, a.grad, C);
    return hipGetLastError();
}

}  // namespace

hipError_t embed_lookup(const EmbedLookupArgs &a)
{
    switch (a.table_dtype * 3 + a.out_dtype) {
    case 0: return launch_lookup<0, 0>(a);
    case 1: return launch_lookup<0, 1>(a);
    case 2: return launch_lookup<0, 2>(a);
    case 3: return launch_lookup<1, 0>(a);
    case 4: return launch_lookup<1, 1>(a);
    case 5: return launch_lookup<1, 2>(a);
    case 6: return launch_lookup<2, 0>(a);
    case 7: return launch_lookup<2, 1>(a);
    default: return launch_lookup<2, 2>(a);
    }
}

uint64_t embed_plan_workspace_bytes(uint64_t n, uint64_t rows) { return n ? plan_layout(n, rows).total : 0; }

hipError_t embed_plan(const EmbedPlanArgs &a)
{
    if (a.n == 0) {
        empty_plan<<<1, 1, 0, a.stream>>>(a.starts, a.count);
        return hipGetLastError();
    }
    return a.rows < (1ull << 32) ? launch_plan<uint32_t>(a) : launch_plan<uint64_t>(a);
}

uint64_t embed_grad_workspace_bytes(uint64_t n, uint64_t d) { return 2 * div_up(n, grad_chunk(n)) * d * 4; }

hipError_t embed_grad(const EmbedGradArgs &a)
{
    switch (a.dtype) {
    case kF32: return launch_grad<kF32>(a);
    case kBF16: return launch_grad<kBF16>(a);
    default: return launch_grad<kF16>(a);
    }
}

}  // namespace cpk
