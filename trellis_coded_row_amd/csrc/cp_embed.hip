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

// What a kernel only reads: from here the compiler may use scalar loads.
typedef const __attribute__((address_space(4))) int32_t *const_i32;
typedef const __attribute__((address_space(4))) int64_t *const_i64;

// Lanes that share a row of d elements, 8 elements each: a power of two.
int row_lanes_log2(uint64_t d)
{
    int s = 0;
    while (s < 6 && (8ull << s) < d) ++s;
    return s;
}

// ---------------------------------------------------------------- lookup

// 2^gs lanes take a row, 8 elements each; blockIdx.y + slice0: a slice of
// 8 << gs columns. A thread has U rows' loads in flight. WAVE: gs is 6, so
// that the ids are the same in all of a wave's lanes and go through scalar
// registers and loads.
//
// Bound by the rows' way from HBM and the stores. 393,216 lookups of 1 KiB
// into a 4 GiB table: 110 us where the rows come from HBM, 4.5 TB/s of what
// has to move (82 us where the last level cache holds them; a copy reaches 5.0
// TB/s). Eight rows a thread in workgroups that end with them: with one row
// 123 us, with four 113; workgroups that stay and read ahead 121; stores that
// are not marked as streaming 116 (four rows).
template <int TI, int TO, int U, bool WAVE>
__global__ __launch_bounds__(256) void lookup_rows(const typename Elem<TI>::raw *__restrict__ table, uint64_t rows,
                                                   uint32_t d, uint64_t stride, const_i64 ids, uint32_t n, float scale,
                                                   typename Elem<TO>::raw *__restrict__ out,
                                                   int32_t *__restrict__ bad_id, int gs, uint32_t slice0)
{
    if constexpr (WAVE) gs = 6;
    const uint32_t per = 256u >> gs;
    const uint32_t c = (((slice0 + blockIdx.y) << gs) + (threadIdx.x & ((1u << gs) - 1u))) * 8u;
    uint32_t j = blockIdx.x * (U * per) + (threadIdx.x >> gs);
    if constexpr (WAVE) j = __builtin_amdgcn_readfirstlane(j);
    if (c >= d) return;
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = j + u * per < n ? ids[j + u * per] : -1;
    typename Elem<TI>::vec8 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (id[u] >= 0 && (uint64_t)id[u] >= rows) {
            id[u] = -1;
            if (bad_id) *bad_id = 1;
        }
        if (id[u] >= 0) v[u] = load8<TI>(table + (uint64_t)id[u] * stride, c, d);
        else v[u] = (typename Elem<TI>::raw)0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (j + u * per >= n) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = id[u] < 0 ? 0.0f : Elem<TI>::get(v[u][e]) * scale;  // padding: +0 for any scale
        store8<TO, true>(out + (uint64_t)(j + u * per) * d, c, d, f);
    }
}

constexpr uint32_t kLookupBlocks = 1u << 22;  // workgroups of one launch, at most
constexpr uint32_t kManyRows = 8;             // rows of a thread where there are many

template <int TI, int TO>
hipError_t launch_lookup(const EmbedLookupArgs &a)
{
    typedef typename Elem<TI>::raw RI;
    typedef typename Elem<TO>::raw RO;
    const int gs = row_lanes_log2(a.d);
    const uint32_t per = 256u >> gs;
    const uint64_t slices = div_up(a.d, 8ull << gs);
    // many rows per thread once that still leaves the chip several
    // workgroups per compute unit
    const bool many = a.n >= (uint64_t)kManyRows * per * 2048;
    const uint32_t each = (many ? kManyRows : 1) * per;
    // a launch has fewer than 2^32 threads, and fewer than 2^16 workgroups along y
    const uint64_t step_y = slices < 16384 ? slices : 16384, step = kLookupBlocks / step_y * each;
    for (uint64_t y = 0; y < slices; y += step_y) {
        for (uint64_t j = 0; j < a.n; j += step) {
            const uint32_t n = (uint32_t)(a.n - j < step ? a.n - j : step);
            const dim3 grid((uint32_t)div_up(n, each), (uint32_t)(slices - y < step_y ? slices - y : step_y));
            const auto launch = [&](auto kernel) {
                kernel<<<grid, 256, 0, a.stream>>>((const RI *)a.table, a.rows, (uint32_t)a.d, a.row_stride,
                                                   (const_i64)(a.ids + j), n, a.scale, (RO *)a.out + j * a.d, a.bad_id, gs,
                                                   (uint32_t)y);
            };
            if (gs == 6) many ? launch(lookup_rows<TI, TO, kManyRows, true>) : launch(lookup_rows<TI, TO, 1, true>);
            else many ? launch(lookup_rows<TI, TO, kManyRows, false>) : launch(lookup_rows<TI, TO, 1, false>);
        }
    }
    return hipGetLastError();
}

// ------------------------------------------------------------------ plan

constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortRounds = 2;                            // keys per thread
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

// Where the count of a tile's keys with a digit stands: for few tiles, by
// tile (a scatter adds up the earlier tiles' counts by itself, a launch
// less); else by digit (sort_scan adds them up). The threshold keeps those
// loads in flight together.
constexpr uint32_t kDirectTiles = 32;

template <bool DIRECT>
__device__ __forceinline__ uint64_t count_at(uint32_t tile, uint32_t digit, uint32_t ntiles, uint32_t digits)
{
    return DIRECT ? (uint64_t)tile * digits + digit : (uint64_t)digit * ntiles + tile;
}

// (Counting a pass's keys where the pass before puts them, by atomics, was
// slower than this launch: 25 to 50 us, as frequent rows' keys meet.)
template <typename K, bool FIRST, bool DIRECT>
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
    if (threadIdx.x < digits) hist[count_at<DIRECT>(blockIdx.x, threadIdx.x, ntiles, digits)] = cnt[threadIdx.x];
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

// A pass is bound by the latency of its dependent steps, so tiles are small
// (1,024 keys; with 2,048 a vocabulary's plan took 7 us more) and fill the
// chip early. In a profile: 5 us a count, 3 a scan, 9 to 12 a scatter.
//
// Each key to its place: the keys of smaller digits, the same digit's in
// earlier tiles, in earlier waves' parts of this tile, and in this wave
// before it. Wave w has keys [w, w + 1) * 64 * kSortRounds of the tile.
template <typename K, bool FIRST, bool DIRECT>
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
        if constexpr (DIRECT) {
            constexpr uint32_t B = 8;  // loads in flight
            for (uint32_t t0 = 0; t0 < ntiles; t0 += B) {
                uint32_t c[B];
#pragma unroll
                for (uint32_t q = 0; q < B; ++q) c[q] = t0 + q < ntiles ? hist[(t0 + q) * digits + threadIdx.x] : 0;
#pragma unroll
                for (uint32_t q = 0; q < B; ++q) {
                    total += c[q];
                    before += t0 + q < blockIdx.x ? c[q] : 0;
                }
            }
        } else {
            before = hist[(uint64_t)threadIdx.x * ntiles + blockIdx.x];
            total = totals[threadIdx.x];
        }
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
        if (in) slot[i] = valid ? (int32_t)u : -1;
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

// The whole plan of a batch that fits one workgroup's LDS, in one launch:
// the same sort, its passes divided by barriers, R keys per thread. In a
// graph, for 131,072 rows: 8 us for 1,024 ids and 14 us for 4,096, where the
// launches below take 22 us; with 16 keys per thread it spills (8,192 ids:
// 200 us).
constexpr uint32_t kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;

template <typename K, int R>
__global__ __launch_bounds__(kSmallThreads) void plan_small(const int64_t *__restrict__ ids, uint64_t rows, uint32_t n,
                                                            int passes, int bits, int32_t *__restrict__ order,
                                                            int32_t *__restrict__ slot, int64_t *__restrict__ unique,
                                                            int32_t *__restrict__ starts, int64_t *__restrict__ count)
{
    __shared__ K keys[kSmallThreads * R];
    __shared__ uint16_t vals[kSmallThreads * R];
    __shared__ uint32_t cnt[kSmallWaves][kDigits];
    __shared__ uint32_t wave_sum[kSmallWaves];
    const uint32_t digits = 1u << bits;
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
    const uint32_t base = w * (64 * R) + lane;  // wave w has keys [w, w + 1) * 64 R
    K key[R];
    uint32_t val[R], rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = base + r * 64;
        key[r] = i < n ? key_of<K>(ids[i], rows) : (K)0;
        val[r] = i;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        for (uint32_t i = threadIdx.x; i < kSmallWaves * kDigits; i += kSmallThreads) (&cnt[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
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
        uint32_t total = 0, all;
        if (threadIdx.x < digits) {
#pragma unroll
            for (uint32_t q = 0; q < kSmallWaves; ++q) total += cnt[q][threadIdx.x];
        }
        uint32_t run = block_prefix<kSmallWaves>(total, wave_sum, &all) - total;
        if (threadIdx.x < digits) {
#pragma unroll
            for (uint32_t q = 0; q < kSmallWaves; ++q) {
                const uint32_t c = cnt[q][threadIdx.x];
                cnt[q][threadIdx.x] = run;
                run += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (base + r * 64 < n) {
                const uint32_t to = cnt[w][(uint32_t)(key[r] >> shift) & (digits - 1u)] + rank[r];
                keys[to] = key[r];
                vals[to] = (uint16_t)val[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t i = base + r * 64;
            if (i < n) {
                key[r] = keys[i];
                val[r] = vals[i];
            }
        }
    }
    // the runs: heads before this wave's keys, then before each key
    uint32_t heads = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = base + r * 64;
        const bool head = i < n && key[r] < rows && (i == 0 || keys[i - 1] != key[r]);
        const uint64_t set = __ballot(head);
        rank[r] = heads + (uint32_t)__popcll(set & lanes_below()) + (head ? 1u : 0u);
        heads += (uint32_t)__popcll(set);
    }
    if (lane == 0) wave_sum[w] = heads;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (uint32_t q = 0; q < kSmallWaves; ++q) before += q < w ? wave_sum[q] : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = base + r * 64;
        if (i >= n) continue;
        const bool valid = key[r] < rows;
        const uint32_t u = before + rank[r] - 1u;
        order[i] = (int32_t)val[r];
        slot[i] = valid ? (int32_t)u : -1;
        if (valid && (i == 0 || keys[i - 1] != key[r])) {
            unique[u] = (int64_t)key[r];
            starts[u] = (int32_t)i;
        }
        if (valid && (i + 1 == n || keys[i + 1] >= rows)) {  // the last lookup that takes part
            *count = (int64_t)u + 1;
            starts[u + 1] = (int32_t)i + 1;
        }
        if (i == 0 && !valid) {
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

template <typename K, bool FIRST, bool DIRECT>
void launch_pass(const EmbedPlanArgs &a, const PlanLayout &L, const K *keys, const int32_t *vals, int shift, int bits,
                 K *keys_out, int32_t *vals_out)
{
    const uint32_t n = (uint32_t)a.n, ntiles = (uint32_t)div_up(a.n, kSortTile);
    uint32_t *const hist = reinterpret_cast<uint32_t *>(a.workspace + L.hist);
    uint32_t *const totals = reinterpret_cast<uint32_t *>(a.workspace + L.totals);
    sort_count<K, FIRST, DIRECT><<<ntiles, kSortThreads, 0, a.stream>>>(a.ids, a.rows, keys, n, shift, 1u << bits,
                                                                        ntiles, hist);
    if constexpr (!DIRECT) sort_scan<<<1u << bits, 256, 0, a.stream>>>(hist, ntiles, totals);
    sort_scatter<K, FIRST, DIRECT><<<ntiles, kSortThreads, 0, a.stream>>>(a.ids, a.rows, keys, vals, n, shift, bits,
                                                                          ntiles, hist, totals, keys_out, vals_out);
}

template <typename K>
hipError_t launch_plan(const EmbedPlanArgs &a)
{
    const PlanLayout L = plan_layout(a.n, a.rows);
    const uint32_t n = (uint32_t)a.n, ntiles = (uint32_t)div_up(a.n, kSortTile);
    uint32_t *const heads = reinterpret_cast<uint32_t *>(a.workspace + L.heads);
    K *keys[2] = {reinterpret_cast<K *>(a.workspace + L.keys0), reinterpret_cast<K *>(a.workspace + L.keys1)};
    int32_t *vals[2] = {reinterpret_cast<int32_t *>(a.workspace + L.vals0),
                        reinterpret_cast<int32_t *>(a.workspace + L.vals1)};
    int key_bits = 1;
    while (key_bits < 64 && (a.rows >> key_bits) != 0) ++key_bits;
    const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
    const int bits = (key_bits + passes - 1) / passes;
    if (n <= 4 * kSmallThreads) {
        const auto launch = [&](auto kernel) {
            kernel<<<1, kSmallThreads, 0, a.stream>>>(a.ids, a.rows, n, passes, bits, a.order, a.slot, a.unique, a.starts,
                                                      a.count);
        };
        if (n <= kSmallThreads) launch(plan_small<K, 1>);
        else launch(plan_small<K, 4>);
        return hipGetLastError();
    }
    const bool direct = ntiles <= kDirectTiles;
    for (int p = 0; p < passes; ++p) {
        const K *in = keys[(p + 1) & 1];
        K *out = keys[p & 1];
        const int32_t *vin = vals[(p + 1) & 1];
        int32_t *vout = p + 1 == passes ? a.order : vals[p & 1];
        if (p == 0) {
            if (direct) launch_pass<K, true, true>(a, L, nullptr, nullptr, 0, bits, out, vout);
            else launch_pass<K, true, false>(a, L, nullptr, nullptr, 0, bits, out, vout);
        } else {
            if (direct) launch_pass<K, false, true>(a, L, in, vin, p * bits, bits, out, vout);
            else launch_pass<K, false, false>(a, L, in, vin, p * bits, bits, out, vout);
        }
    }
    const K *sorted = keys[(passes - 1) & 1];
    count_heads<K><<<ntiles, kSortThreads, 0, a.stream>>>(sorted, a.rows, n, heads);
    write_runs<K><<<ntiles, kSortThreads, 0, a.stream>>>(sorted, a.rows, n, heads, a.slot, a.unique, a.starts, a.count);
    return hipGetLastError();
}

// -------------------------------------------------------------- gradient

// Sorted lookups per chunk: a chunk is summed by one group of lanes. Few, so
// that no group's rows, read a few at a time, outlast the others'.
uint32_t grad_chunk(uint64_t n)
{
    uint32_t c = 8;
    while ((c < 32 && n / c > 4096) || n / c > (1u << 24)) c <<= 1;  // (a launch has fewer than 2^32 threads)
    return c;
}

// A row with more lookups than a chunk (a long run) is summed by chunks
// (partial sums, joined afterwards); any other by the chunk in which its run
// begins.

// Row s's sum goes to grad row `rows ? unique[s] : s`.
template <typename P>
__device__ __forceinline__ float *grad_row(float *grad, P unique, uint64_t rows, int32_t s, uint64_t d)
{
    return grad + (rows ? (uint64_t)unique[s] : (uint64_t)(uint32_t)s) * d;
}

struct GradParams {
    const_i32 order, slot;
    const_i64 unique;
    const_i32 starts;
    const_i64 count;
    uint64_t rows;
    const void *dout;
    uint32_t n, d;
    uint64_t stride;
    float scale;
    float *grad, *partial;
    uint32_t C;  // lookups per chunk
    int gs;      // 2^gs lanes per chunk
};

// Chunk c: sorted lookups [c C, c C + C). Its group of 2^gs lanes sums the
// runs that begin in it, reading past its end for a short last run, and its
// own part of a long run into partial[2 c] (begun in an earlier chunk) or
// partial[2 c + 1] (begun in this one). blockIdx.y: a slice of 8 << gs
// columns. WAVE: gs is 6, so that everything but the row's values is the same
// in all of a wave's lanes and goes through scalar registers and loads.
//
// Bound by the rows' bytes: 393,216 rows of 512 bf16 into 110,000 sums take 142
// us, 4.4 TB/s. A group's rows come one after the other, so what costs is the
// longest group: with chunks of 64 and runs of up to 256 in one group, 245 us.
template <int DT, bool WAVE>
__global__ __launch_bounds__(256) void grad_rows(GradParams p)
{
    constexpr int U = 8;  // rows' loads in flight
    const int gs = WAVE ? 6 : p.gs;
    const uint32_t d = p.d, C = p.C;
    const uint32_t lane = threadIdx.x & ((1u << gs) - 1u);
    uint32_t chunk = blockIdx.x * (256u >> gs) + (threadIdx.x >> gs);
    if constexpr (WAVE) chunk = __builtin_amdgcn_readfirstlane(chunk);
    const uint32_t c = (blockIdx.y * (1u << gs) + lane) * 8u;
    const uint64_t c0 = (uint64_t)chunk * C;
    if (c0 >= p.n) return;
    uint32_t lo = (uint32_t)c0, hi = (uint32_t)(c0 + C < p.n ? c0 + C : p.n);
    // the run that covers the first lookup, and the one that covers the last
    const int32_t sf = p.slot[lo];
    int32_t sl = p.slot[hi - 1];
    if (sf < 0) return;  // lookups that take no part are the last ones
    if (sl < 0) {
        hi = (uint32_t)p.starts[*p.count];
        sl = p.slot[hi - 1];
    }
    const uint32_t fb = (uint32_t)p.starts[sf], fe = (uint32_t)p.starts[sf + 1];
    const uint32_t lb = (uint32_t)p.starts[sl], le = (uint32_t)p.starts[sl + 1];
    const bool first_long = fe - fb > C, last_long = le - lb > C;
    const bool from_before = fb < lo;
    if (from_before && !first_long) lo = fe;  // an earlier chunk sums it
    if (!last_long) hi = le;
    if (lo >= hi || c >= d) return;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    // the next rows' places are read while the present rows' values arrive
    int32_t t[U], s[U + 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t iu = lo + u < hi ? lo + u : hi - 1;
        t[u] = p.order[iu];
        s[u] = p.slot[iu];
    }
    for (uint32_t i = lo; i < hi; i += U) {
        typename Elem<DT>::vec8 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = load8<DT>((const typename Elem<DT>::raw *)p.dout + (uint64_t)(uint32_t)t[u] * p.stride, c, d);
        int32_t tn[U], sn[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t iu = i + U + u < hi ? i + U + u : hi - 1;
            tn[u] = p.order[iu];
            sn[u] = p.slot[iu];
        }
        s[U] = sn[0];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u < hi) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += Elem<DT>::get(v[u][e]);
                if (i + u + 1 == hi || s[u + 1] != s[u]) {
                    float *row;
                    if (s[u] == sf && first_long) row = p.partial + (2ull * chunk + (from_before ? 0 : 1)) * d;
                    else if (s[u] == sl && last_long) row = p.partial + (2ull * chunk + 1) * d;
                    else row = grad_row(p.grad, p.unique, p.rows, s[u], d);
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] = acc[e] * p.scale;
                        acc[e] = 0.0f;
                    }
                    store8<kF32>(row, c, d, f);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = tn[u];
            s[u] = sn[u];
        }
    }
}

// Zeros in the whole gradient, before the sums are written: bound by the
// stores. One of 16 bytes for each thread of a workgroup that ends then is
// the fastest (131,072 x 1,024: 79 us, 6.8 TB/s; workgroups that clear 64 KiB
// each 99 us), faster than leaving out the rows that sums go to, which has to
// look each up (107 us).
constexpr uint32_t kZeroFloats = 1024;  // of a workgroup

__global__ __launch_bounds__(256) void grad_zero(float *__restrict__ grad, uint64_t count)
{
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    for (uint64_t at = (uint64_t)blockIdx.x * kZeroFloats + threadIdx.x * 4u; at < count;
         at += (uint64_t)gridDim.x * kZeroFloats) {
        if (at + 4 <= count) {
            *reinterpret_cast<v4 *>(grad + at) = (v4)0.0f;
        } else {
            for (uint64_t q = at; q < count; ++q) grad[q] = 0.0f;
        }
    }
}

typedef float float4_any __attribute__((ext_vector_type(4), aligned(4)));

// Columns [c, c + 4) of a row of d floats, zeros past its end.
__device__ __forceinline__ float4_any load4(const float *row, uint32_t c, uint32_t d)
{
    if (c + 4 <= d) return *reinterpret_cast<const float4_any *>(row + c);
    float4_any v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = c + q < d ? row[c + q] : 0.0f;
    return v;
}

// The long runs: each is the sum of its partial sums. A workgroup looks for
// those that begin in its kJoinChunks chunks; 16 lanes take 64 columns, the
// workgroup's 16 such groups every 16th partial sum. 24 to 27 us for the batch
// above, whose most frequent row has 1,200 partial sums: the time is theirs.
constexpr uint32_t kJoinChunks = 16, kJoinColumns = 64;

__global__ __launch_bounds__(256) void grad_join(const int32_t *__restrict__ slot, const int64_t *__restrict__ unique,
                                                 const int32_t *__restrict__ starts, uint64_t rows, uint32_t n,
                                                 uint32_t d, const float *__restrict__ partial,
                                                 float *__restrict__ grad, uint32_t C)
{
    __shared__ float sums[16][kJoinColumns];
    __shared__ uint32_t found, run_chunk[kJoinChunks], run_parts[kJoinChunks];
    __shared__ int32_t run_slot[kJoinChunks];
    const uint32_t lane = threadIdx.x & 15u, g = threadIdx.x >> 4;
    const uint32_t col = blockIdx.y * kJoinColumns + lane * 4u;
    if (threadIdx.x < 64) {
        const uint32_t chunk = blockIdx.x * kJoinChunks + (threadIdx.x & (kJoinChunks - 1u));
        const uint64_t c0 = (uint64_t)chunk * C;
        bool begins = false;
        int32_t s = -1;
        uint32_t e = 0;
        // a long run that begins in a chunk covers its last lookup
        if (threadIdx.x < kJoinChunks && c0 + C <= n) s = slot[c0 + C - 1];
        if (s >= 0) {
            const uint32_t b = (uint32_t)starts[s];
            e = (uint32_t)starts[s + 1];
            begins = e - b > C && b >= c0;
        }
        const uint64_t set = __ballot(begins);
        if (begins) {
            const uint32_t at = (uint32_t)__popcll(set & lanes_below());
            run_chunk[at] = chunk;
            run_parts[at] = (e - 1) / C - chunk + 1;
            run_slot[at] = s;
        }
        if (threadIdx.x == 0) found = (uint32_t)__popcll(set);
    }
    __syncthreads();
    for (uint32_t r = 0; r < found; ++r) {
        const uint32_t chunk = run_chunk[r], parts = run_parts[r];
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 16
        for (uint32_t k = g; k < parts; k += 16) {  // part 0 is this chunk's
            const auto v = load4(partial + (2ull * (chunk + k) + (k == 0 ? 1 : 0)) * d, col, d);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] += v[q];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[g][lane * 4 + q] = acc[q];
        __syncthreads();
        const uint32_t cc = blockIdx.y * kJoinColumns + threadIdx.x;
        if (threadIdx.x < kJoinColumns && cc < d) {
            float t = 0.0f;
#pragma unroll
            for (int q = 0; q < 16; ++q) t += sums[q][threadIdx.x];
            grad_row(grad, unique, rows, run_slot[r], d)[cc] = t;
        }
        __syncthreads();
    }
}

template <int DT>
hipError_t launch_grad(const EmbedGradArgs &a)
{
    GradParams p{};
    p.order = (const_i32)a.order;
    p.slot = (const_i32)a.slot;
    p.unique = (const_i64)a.unique;
    p.starts = (const_i32)a.starts;
    p.count = (const_i64)a.count;
    p.rows = a.rows;
    p.dout = a.dout;
    p.n = (uint32_t)a.n;
    p.d = (uint32_t)a.d;
    p.stride = a.stride;
    p.scale = a.scale;
    p.grad = a.grad;
    p.partial = reinterpret_cast<float *>(a.workspace);
    p.C = grad_chunk(a.n);
    p.gs = row_lanes_log2(a.d);
    const uint64_t chunks = div_up(a.n, p.C);
    const uint32_t slices = (uint32_t)div_up(a.d, 8ull << p.gs);
    if (a.rows) {
        const uint64_t count = a.rows * a.d, blocks = div_up(count, kZeroFloats);
        // (a launch has fewer than 2^32 threads)
        grad_zero<<<(uint32_t)(blocks < (1u << 23) ? blocks : 1u << 23), 256, 0, a.stream>>>(a.grad, count);
    }
    if (a.n == 0) return hipGetLastError();
    const dim3 grid((uint32_t)div_up(chunks, 256u >> p.gs), slices);
    if (p.gs == 6) grad_rows<DT, true><<<grid, 256, 0, a.stream>>>(p);
    else grad_rows<DT, false><<<grid, 256, 0, a.stream>>>(p);
    if (a.n > p.C)
        grad_join<<<dim3((uint32_t)div_up(chunks, kJoinChunks), (uint32_t)div_up(a.d, kJoinColumns)), 256, 0,
                    a.stream>>>(a.slot, a.unique, a.starts, a.rows, p.n, p.d, p.partial, a.grad, p.C);
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
