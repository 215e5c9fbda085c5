// embedding.hip -- token embedding (rows of a table by token id, scaled) and
// the gradient of the table.
//
//   out[i] = scale * table[ids[i]]                 (zero where ids[i] is no row)
//   grad[v] = scale * sum over i with ids[i] = v of dout[i]    (+ grad[v])
//
// Up to 128 tokens the gradient is one launch. Above, it goes by sorted tokens:
// the positions i are put in order of their token (equal tokens in input
// order), so that each row's terms are consecutive, and are then summed in that
// order: no atomics on the sums, and the same bits on every run.
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

// ---------------------------------------------------------------------------
// Lookup. `lanes` lanes (a power of two) stand side by side on one row, 64 /
// lanes rows at once, 16 bytes per lane and step; a wave takes ROWS such groups
// of rows and holds STEPS steps of each in flight. Outputs are written past the
// cache: nothing here reads them again, and rows of frequent tokens stay in it.
// 65,536 tokens of 2,048 bf16: 64-66 us, 351 MB at 5.4 TB/s (one group of rows
// in flight: 77; with cached stores 79, with past-cache loads 85).
// ---------------------------------------------------------------------------
template <typename T, typename ID, int STEPS, int ROWS>
__global__ __launch_bounds__(kThreads) void embedding_kernel(const T* __restrict__ table, int64_t rows, int64_t dim,
                                                             int64_t table_stride, const ID* __restrict__ ids,
                                                             int64_t n, float scale, T* __restrict__ out,
                                                             int64_t out_stride, int lanes)
{
    constexpr int N = Vec16<T>::kN;
    const int per_wave = kWave / lanes, mine = lane_id() % lanes;
    const int64_t wave = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    const int64_t first = wave * (per_wave * ROWS) + lane_id() / lanes;
    const T* src[ROWS];
    bool there[ROWS], live[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t i = first + r * per_wave;
        there[r] = i < n;
        const int64_t id = there[r] ? (int64_t)ids[i] : -1;
        live[r] = id >= 0 && id < rows;
        src[r] = table + (live[r] ? id : 0) * table_stride;
    }
    const int64_t step = (int64_t)lanes * N, vecs = dim / N * N;
    for (int64_t c = (int64_t)mine * N; c < vecs; c += step * STEPS) {
        u32x4 v[ROWS][STEPS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                v[r][k] = u32x4{0u, 0u, 0u, 0u};
                if (live[r] && c + k * step < vecs)
                    v[r][k] = *reinterpret_cast<const typename Vec16<T>::type*>(src[r] + c + k * step);
            }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            T* dst = out + (first + r * per_wave) * out_stride + c;
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                T t[N];
                __builtin_memcpy(t, &v[r][k], sizeof(t));
#pragma unroll
                for (int j = 0; j < N; ++j) t[j] = live[r] ? (T)((float)t[j] * scale) : (T)0.0f;
                u32x4 w;
                __builtin_memcpy(&w, t, sizeof(w));
                if (there[r] && c + k * step < vecs)
                    __builtin_nontemporal_store(w, reinterpret_cast<typename Vec16<T>::type*>(dst + k * step));
            }
        }
    }
    // the last, partial vector of the rows
    for (int64_t e = vecs + mine; e < dim; e += lanes)
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (there[r])
                out[(first + r * per_wave) * out_stride + e] = live[r] ? (T)((float)src[r][e] * scale) : (T)0.0f;
}

// ---------------------------------------------------------------------------
// Clearing of a whole new gradient, by workgroups that ride along in the
// launches. A sort's launches wait on latency and leave the memory idle, so
// each clears its first rows whatever their tokens; the launch of the sums
// clears the rest but for the rows that have tokens.
// ---------------------------------------------------------------------------
struct ClearArgs {
    char* grad;
    int64_t row_bytes, stride_bytes;
    int64_t first, last;  // rows
    int skip;             // workgroups before the clearing ones
    int per_wave;         // rows of a wave
};

__device__ __forceinline__ void clear_span(char* p, int64_t bytes)
{
    int64_t c = (int64_t)lane_id() * kVecBytes;
    for (; c + kVecBytes <= bytes; c += kWave * kVecBytes)
        __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4_a2*>(p + c));
    for (; c < bytes && c + kVecBytes > bytes; c += 2) *reinterpret_cast<uint16_t*>(p + c) = 0;
}

template <int THREADS>
__device__ __forceinline__ int64_t clear_wave(const ClearArgs& a)
{
    return (int64_t)(blockIdx.x - a.skip) * (THREADS / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}

// Rows without gaps are cleared in pieces of kPiece bytes that begin at
// multiples of it, so that no cache line is written by two waves.
constexpr int64_t kPiece = 4096;

template <int THREADS>
__device__ __forceinline__ void clear_rows(const ClearArgs& a)
{
    const int64_t wave = clear_wave<THREADS>(a);
    if (a.stride_bytes == a.row_bytes) {
        const int64_t first = a.first * a.row_bytes, last = a.last * a.row_bytes, at = (first / kPiece + wave) * kPiece;
        const int64_t from = at > first ? at : first, to = at + kPiece < last ? at + kPiece : last;
        if (from < to) clear_span(a.grad + from, to - from);
        return;
    }
    const int64_t r0 = a.first + wave * a.per_wave, r1 = r0 + a.per_wave < a.last ? r0 + a.per_wave : a.last;
    for (int64_t r = r0; r < r1; ++r) clear_span(a.grad + r * a.stride_bytes, a.row_bytes);
}

// The same but for rows among the sorted keys: each half of the wave looks,
// with 32 probes at a time, for one end of the keys of the wave's rows, then
// lane l looks for row r0 + l among them. (Seventeen dependent reads for 65,536
// keys become four and a few.)
template <int THREADS>
__device__ __forceinline__ void clear_other_rows(const ClearArgs& a, const uint32_t* __restrict__ keys, int64_t n)
{
    const int64_t r0 = a.first + clear_wave<THREADS>(a) * a.per_wave, mine = r0 + lane_id();
    const int64_t end = r0 + lane_id() / 32 * a.per_wave;
    int64_t low = 0, size = n;  // the first key that is not below `end` is among low .. low + size
    while (readlane((int)(size > 0), 0) | readlane((int)(size > 0), 32)) {
        const int64_t step = size / 32 + 1, at = low + (lane_id() % 32) * step;
        const bool below = at < low + size && (int64_t)keys[at] < end;
        const uint32_t which = (uint32_t)(ballot(below) >> (lane_id() / 32 * 32));
        const int count = __builtin_popcount(which);  // probes below `end`: the first ones
        if (count == 0) {
            size = 0;
        } else {
            const int64_t from = low + (count - 1) * step + 1, to = low + count * step;
            size = (to < low + size ? to : low + size) - from;
            low = from;
        }
    }
    const int64_t last = readlane(low, 32);
    low = readlane(low, 0);
    for (int64_t high = last; low < high;) {
        const int64_t mid = (low + high) / 2;
        if ((int64_t)keys[mid] < mine) low = mid + 1;
        else high = mid;
    }
    const uint64_t has = ballot(low < last && (int64_t)keys[low < last ? low : 0] == mine);
    for (int i = 0; i < a.per_wave && r0 + i < a.last; ++i)
        if (!((has >> i) & 1u)) clear_span(a.grad + (r0 + i) * a.stride_bytes, a.row_bytes);
}

// ---------------------------------------------------------------------------
// Sorting the tokens. Keys are row numbers; what is no row gets the key
// `rows`, which sorts last and is left out of the sums.
// ---------------------------------------------------------------------------
template <typename ID>
__device__ __forceinline__ uint32_t token_key(ID id, int64_t rows)
{
    return (int64_t)id >= 0 && (int64_t)id < rows ? (uint32_t)id : (uint32_t)rows;
}

// 8,000 tokens of 256 columns: 26.8 us for a whole gradient call by rank, 29.4
// by the passes below; 9,000: 29.1 and 28.3.
constexpr int64_t kRankSortMax = 8192;
constexpr int kRankParts = 16;                     // lanes that count for one token
constexpr int kRankTokens = kThreads / kRankParts; // tokens per workgroup

// place(i) = #{j : key_j < key_i} + #{j < i : key_j = key_i}. Every workgroup
// holds all keys in LDS; 16 lanes share one token's count.
template <typename ID>
__global__ __launch_bounds__(kThreads) void token_rank_sort_kernel(const ID* __restrict__ ids, uint32_t n,
                                                                   int64_t rows, uint32_t* __restrict__ keys,
                                                                   uint32_t* __restrict__ places,
                                                                   uint32_t* __restrict__ crossing, ClearArgs clear)
{
    extern __shared__ __align__(16) uint32_t s_key[];  // n rounded up to 64 keys
    if (blockIdx.x >= (uint32_t)clear.skip) return clear_rows<kThreads>(clear);
    if (blockIdx.x == 0 && threadIdx.x == 0) crossing[0] = 0;
    const uint32_t padded = (n + 63u) & ~63u;
    constexpr uint32_t kAt = 8;  // ids in flight per thread
    for (uint32_t j0 = threadIdx.x; j0 < padded; j0 += kAt * kThreads) {
        ID id[kAt];
#pragma unroll
        for (uint32_t q = 0; q < kAt; ++q) id[q] = ids[j0 + q * kThreads < n ? j0 + q * kThreads : 0];
#pragma unroll
        for (uint32_t q = 0; q < kAt; ++q) {
            const uint32_t j = j0 + q * kThreads;
            if (j < padded) s_key[j] = j < n ? token_key(id[q], rows) : 0xFFFFFFFFu;
        }
    }
    __syncthreads();
    const uint32_t i = blockIdx.x * kRankTokens + threadIdx.x / kRankParts, part = threadIdx.x % kRankParts;
    const uint32_t key = i < n ? s_key[i] : 0u;
    uint32_t below = 0;
    // the workgroup's tokens lie in one block of 64: before it equal keys count, after it they do not
    static_assert(64 % kRankTokens == 0 && kRankParts * 4 == 64, "a step is a block of 64 keys");
    const uint32_t own = blockIdx.x * kRankTokens / 64 * 64;
    const auto count = [&](uint32_t from, uint32_t to, uint32_t limit) {
#pragma unroll 4
        for (uint32_t j = from + part * 4; j < to; j += 64) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(s_key + j);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) below += k[q] < limit ? 1u : 0u;
        }
    };
    count(0, own, key + 1);
    {
        const uint32_t j = own + part * 4;
        const u32x4 k = *reinterpret_cast<const u32x4*>(s_key + j);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) below += k[q] < key + (j + q < i ? 1u : 0u) ? 1u : 0u;
    }
    count(own + 64, padded, key);
    below += dpp<0x111>(below);  // sums over the row of 16 lanes: row_shr 1, 2, 4, 8
    below += dpp<0x112>(below);
    below += dpp<0x114>(below);
    below += dpp<0x118>(below);
    if (part == kRankParts - 1 && i < n) {
        keys[below] = key;
        places[below] = i;
    }
}

// From kRankSortMax to kTileSortMax tokens: stable counting passes over digits
// of up to 9 bits, two for up to 2^18 - 1 rows, each a launch that counts the
// digit in every tile and one that places the keys. There is no scan in
// between: each workgroup of a pass sums the table up for itself (at most 128
// tiles to a digit, read from the cache, tile by tile so that a wave reads
// whole lines). For 65,536 tokens the four launches
// take 5 us each, where the library's general passes with a scan launch each
// took 36 us in all; one launch less, with the second digit counted by atomics
// in the first pass, took 11 us more (its words are shared by all XCDs).
constexpr int64_t kTileSortMax = 262144;
constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;
constexpr int kDigitBits = 9;
static_assert(1 << kDigitBits == kTileThreads, "one digit per thread");

struct TileSort {
    uint32_t n;
    int64_t rows;
    int bits, digits;          // of a digit; digits of a key
    int items;                 // keys per thread: tiles of kTileThreads * items
    int tiles;
    uint32_t* table;           // [tiles][1 << bits]
};

// Counts digit `digit` of every tile. The first launch has the ids and writes
// the keys; the others (ids null) have the keys.
template <typename ID>
__global__ __launch_bounds__(kTileThreads) void token_count_kernel(const ID* __restrict__ ids, TileSort a, int digit,
                                                                   uint32_t* __restrict__ keys,
                                                                   uint32_t* __restrict__ crossing, ClearArgs clear)
{
    __shared__ uint32_t s_count[kTileThreads];
    if (blockIdx.x >= (uint32_t)clear.skip) return clear_rows<kTileThreads>(clear);
    if (blockIdx.x == 0 && threadIdx.x == 0) crossing[0] = 0;
    const uint32_t size = 1u << a.bits;
    s_count[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * (uint32_t)(kTileThreads * a.items);
    for (int k = 0; k < a.items; ++k) {
        const uint32_t i = first + k * kTileThreads + threadIdx.x;
        if (i < a.n) {
            const uint32_t key = ids ? token_key(ids[i], a.rows) : keys[i];
            if (ids) keys[i] = key;
            atomicAdd(&s_count[(key >> (digit * a.bits)) & (size - 1)], 1u);
        }
    }
    __syncthreads();
    if (threadIdx.x < size) a.table[(blockIdx.x << a.bits) + threadIdx.x] = s_count[threadIdx.x];
}

// Pass `digit`: keys (and their positions; null: keys are in input order) to
// their places by that digit.
template <int ITEMS>
__global__ __launch_bounds__(kTileThreads) void token_pass_kernel(const uint32_t* __restrict__ keys,
                                                                  const uint32_t* __restrict__ index, TileSort a,
                                                                  int digit, uint32_t* __restrict__ keys_out,
                                                                  uint32_t* __restrict__ index_out, ClearArgs clear)
{
    __shared__ uint32_t s_count[kTileWaves][kTileThreads];  // of each wave, then of the waves before it
    __shared__ uint32_t s_base[kTileThreads];
    __shared__ uint32_t s_wave[kTileWaves];
    if (blockIdx.x >= (uint32_t)clear.skip) return clear_rows<kTileThreads>(clear);
    const int lane = lane_id(), wave = (int)(threadIdx.x / kWave), tile = blockIdx.x;
    const uint32_t size = 1u << a.bits, shift = (uint32_t)(digit * a.bits);
    // this thread's keys, in input order along the wave's segment of the tile
    const uint32_t seg = (uint32_t)tile * (kTileThreads * ITEMS) + wave * (kWave * ITEMS) + lane;
    uint32_t key[ITEMS], pos[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const uint32_t i = seg + k * kWave;
        key[k] = i < a.n ? keys[i] : 0u;
        pos[k] = i < a.n && index ? index[i] : i;
    }
    // digit d = this thread: keys of smaller digits and, of its own, those of the tiles before
    uint32_t total = 0, before = 0;
    if (threadIdx.x < size) {
        for (int t0 = 0; t0 < a.tiles; t0 += 16) {
            uint32_t c[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) c[q] = a.table[((t0 + q < a.tiles ? t0 + q : 0) << a.bits) + threadIdx.x];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const uint32_t v = t0 + q < a.tiles ? c[q] : 0u;
                total += v;
                before += t0 + q < tile ? v : 0u;
            }
        }
    }
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) s_count[w][threadIdx.x] = 0;
    const uint32_t incl = wave_inclusive_scan(total);
    if (lane == kWave - 1) s_wave[wave] = incl;
    __syncthreads();
    uint32_t start = incl - total + before;
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) start += w < wave ? s_wave[w] : 0u;
    // rank among the wave's keys of the same digit that come before
    uint32_t rank[ITEMS], d[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const bool live = seg + k * kWave < a.n;
        d[k] = (key[k] >> shift) & (size - 1);
        uint64_t same = ballot(live);
        for (int b = 0; b < a.bits; ++b) {
            const bool bit = (d[k] >> b) & 1u;
            const uint64_t set = ballot(bit);
            same &= bit ? set : ~set;
        }
        const uint32_t below = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u));
        const uint32_t run = s_count[wave][d[k]];
        if (live && below == 0) s_count[wave][d[k]] = run + (uint32_t)__builtin_popcountll(same);
        rank[k] = run + below;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next key's lanes read what these lanes wrote
    }
    __syncthreads();
    uint32_t sum = start;
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) {
        const uint32_t c = s_count[w][threadIdx.x];
        s_count[w][threadIdx.x] = sum;
        sum += c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        if (seg + k * kWave < a.n) {
            const uint32_t to = s_count[wave][d[k]] + rank[k];
            keys_out[to] = key[k];
            index_out[to] = pos[k];
        }
    }
}

// Above kTileSortMax tokens: keys and positions for the radix passes.
template <typename ID>
__global__ __launch_bounds__(kThreads) void token_keys_kernel(const ID* __restrict__ ids, int64_t n, int64_t rows,
                                                              uint32_t* __restrict__ keys, uint32_t* __restrict__ index,
                                                              uint32_t* __restrict__ crossing, ClearArgs clear)
{
    if (blockIdx.x >= (uint32_t)clear.skip) return clear_rows<kThreads>(clear);
    if (blockIdx.x == 0 && threadIdx.x == 0) crossing[0] = 0;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    keys[i] = token_key(ids[i], rows);
    index[i] = (uint32_t)i;
}

// ---------------------------------------------------------------------------
// Sums. The sorted positions are cut into chunks of `chunk` (8 to 64), the
// columns into slabs of one 16-byte access per lane (of the wider of the two types); a wave adds up one chunk
// of one slab, run by run. A run that lies inside its chunk is a whole row of
// the gradient. The part of a run that crosses a chunk's edge goes to
// `partial` (two 32-bit rows per chunk: 0 for a run that began in an earlier
// chunk, 1 for one that begins here and goes on), the chunk in which such a
// run begins to the list `crossing`, and embedding_join_kernel adds the parts
// up in order.
// ---------------------------------------------------------------------------
struct GradArgs {
    const uint32_t* keys;   // sorted
    const uint32_t* index;  // position of each sorted token in the input
    int64_t n, rows, dim, dout_stride, grad_stride;
    int chunk;
    float scale;
    float* partial;  // [chunks][2][dim rounded up to whole slabs]
    int64_t partial_stride;
    uint32_t* crossing;  // count, then chunks in any order
};

__device__ __forceinline__ uint32_t key_at(const GradArgs& a, int64_t p)
{
    return p >= 0 && p < a.n ? a.keys[p] : 0xFFFFFFFFu;
}

// N elements of T, 8 or 16 bytes, as loaded: one access at any alignment.
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
template <typename T, int N> struct Pack {
    static constexpr int kWords = N * (int)sizeof(T) / 4;
    uint32_t w[kWords];
};

// Elements at .. at + N - 1 of `base`, moved down where they would pass `limit`
// elements (the buffer's end): element j is then at place j + shift. limit >= N.
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_window(const T* __restrict__ base, int64_t at, int64_t limit)
{
    const T* p = base + (at + N <= limit ? at : limit - N);
    Pack<T, N> r;
    if constexpr (Pack<T, N>::kWords == 4) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const typename Vec16<T>::type*>(p));
        __builtin_memcpy(&r, &v, sizeof(r));
    } else {
        const u32x2_a2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a2*>(p));
        __builtin_memcpy(&r, &v, sizeof(r));
    }
    return r;
}

template <typename T, int N>
__device__ __forceinline__ void shift_down(Pack<T, N>& v, int elems)
{
    constexpr int kWords = Pack<T, N>::kWords;
    const int bytes = elems * (int)sizeof(T);
#pragma unroll
    for (int by = 2; by >= 1; by /= 2)
        if (bytes & (by * 4)) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) v.w[i] = i + by < kWords ? v.w[i + by] : 0u;
        }
    if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) v.w[i] = v.w[i] >> 16 | (i + 1 < kWords ? v.w[i + 1] << 16 : 0u);
    }
}

// Columns per lane: 16 bytes of the wider of the two types.
template <typename T, typename O> struct GradCols {
    static constexpr int value = Vec16<O>::kN < Vec16<T>::kN ? Vec16<O>::kN : Vec16<T>::kN;
};

// ADD: the rows that end in the chunk are loaded with the terms, not when the
// run's sum is ready: a load behind every run is what bounded this otherwise.
// Their stores are non-temporal; those of a new gradient are not (65,536
// tokens of 2,048: 142 us against 127). Terms are read once and loaded
// non-temporally (127 us against 138). WHOLE: no lane of the wave has a row's
// last, partial vector.
template <typename T, typename O, bool ADD, bool WHOLE>
__device__ __forceinline__ void sum_chunk_of_slab(const T* __restrict__ dout, O* __restrict__ grad, const GradArgs& a,
                                                  int64_t chunk, int64_t c, bool first_slab)
{
    constexpr int N = GradCols<T, O>::value;
    constexpr int kAhead = 8;  // rows in flight
    using Vec = typename Vec16<O>::type;
    const int lane = lane_id();
    const int64_t p0 = chunk * a.chunk;
    const bool mine = lane < a.chunk;
    const uint32_t key = mine ? key_at(a, p0 + lane) : 0xFFFFFFFFu;
    const uint32_t next = mine ? key_at(a, p0 + lane + 1) : 0xFFFFFFFFu;
    const uint32_t before = key_at(a, p0 - 1);
    const uint32_t index = mine && p0 + lane < a.n ? a.index[p0 + lane] : 0u;
    const int count = __builtin_popcountll(ballot(key < (uint32_t)a.rows));
    if (count == 0) return;
    const uint64_t ends = ballot(key != next);  // the run ends at this position
    bool opened = readlane(key, 0) == before;   // the current run began in an earlier chunk
    const bool live = c < a.dim;
    const int64_t col = live ? c : 0, valid = a.dim - col;
    const int64_t limit = (a.n - 1) * a.dout_stride + a.dim;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    for (int i0 = 0; i0 < count; i0 += kAhead) {
        Pack<T, N> x[kAhead];
        u32x4 was[ADD ? kAhead : 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t row = (int64_t)readlane(index, i0 + i < count ? i0 + i : count - 1) * a.dout_stride;
            if (WHOLE || limit >= N) {
                x[i] = load_window<T, N>(dout, row + col, WHOLE ? INT64_MAX : limit);
            } else {  // fewer than N elements in all
                T t[N];
#pragma unroll
                for (int j = 0; j < N; ++j) t[j] = j < valid ? dout[row + col + j] : (T)0.0f;
                __builtin_memcpy(&x[i], t, sizeof(t));
            }
        }
        if constexpr (ADD) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i0 + i < count && ((ends >> (i0 + i)) & 1u)) {
                    const O* p = grad + (int64_t)readlane(key, i0 + i) * a.grad_stride + col;
                    if (WHOLE || valid >= N) {
                        was[i] = *reinterpret_cast<const Vec*>(p);
                    } else {
                        O t[N];
#pragma unroll
                        for (int j = 0; j < N; ++j) t[j] = j < valid ? p[j] : (O)0.0f;
                        __builtin_memcpy(&was[i], t, sizeof(t));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i < count) {  // uniform
                if constexpr (!WHOLE) {
                    const int64_t over =
                        limit < N ? 0 : (int64_t)readlane(index, i0 + i) * a.dout_stride + col + N - limit;
                    if (ballot(over > 0)) shift_down<T, N>(x[i], over > 0 ? (int)over : 0);
                }
                T t[N];
                __builtin_memcpy(t, &x[i], sizeof(t));
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += (float)t[j];
                if ((ends >> (i0 + i)) & 1u) {
                    if (opened) {
                        store_floats<float, N>(a.partial + chunk * 2 * a.partial_stride + c, N, acc);
                    } else if (live) {
                        O o[N];
                        if constexpr (ADD) __builtin_memcpy(o, &was[i], sizeof(o));
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            float y = acc[j] * a.scale;
                            if constexpr (ADD) y += (float)o[j];
                            o[j] = (O)y;
                        }
                        O* p = grad + (int64_t)readlane(key, i0 + i) * a.grad_stride + c;
                        if (WHOLE || valid >= N) {
                            u32x4 u;
                            __builtin_memcpy(&u, o, sizeof(u));
                            if constexpr (ADD)
                                __builtin_nontemporal_store(u, reinterpret_cast<Vec*>(p));
                            else
                                *reinterpret_cast<Vec*>(p) = u;
                        } else {
#pragma unroll
                            for (int j = 0; j < N; ++j)
                                if (j < valid) p[j] = o[j];
                        }
                    }
                    opened = false;
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
                }
            }
        }
    }
    if (!((ends >> (count - 1)) & 1u)) {  // the last run goes on
        store_floats<float, N>(a.partial + (chunk * 2 + (opened ? 0 : 1)) * a.partial_stride + c, N, acc);
        if (!opened && first_slab && lane == 0) a.crossing[1 + atomicAdd(a.crossing, 1u)] = (uint32_t)chunk;
    }
}

template <typename T, typename O, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_sum_kernel(const T* __restrict__ dout, O* __restrict__ grad,
                                                                 GradArgs a, int64_t slabs, int64_t units,
                                                                 ClearArgs clear)
{
    if constexpr (!ADD) {
        if (blockIdx.x >= (uint32_t)clear.skip) return clear_other_rows<kThreads>(clear, a.keys, a.n);
    }
    constexpr int N = GradCols<T, O>::value;
    static_assert(N == Vec16<O>::kN, "one access per row of the gradient");
    const int64_t unit = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit >= units) return;
    const int64_t chunk = unit / slabs, slab = unit % slabs, c = (slab * kWave + lane_id()) * N;
    if (a.dim % N == 0 || (slab + 1) * kWave * N <= a.dim)
        sum_chunk_of_slab<T, O, ADD, true>(dout, grad, a, chunk, c, slab == 0);
    else
        sum_chunk_of_slab<T, O, ADD, false>(dout, grad, a, chunk, c, slab == 0);
}

// ---------------------------------------------------------------------------
// Up to kFewMax tokens: one launch, no sorting. A wave has one token's position
// and one slab; every wave holds all ids, two to a lane. The wave of a row's
// first position adds up the row's positions, in order, and the clearing waves
// see which rows have tokens. (Three launches take 14.5 us of the host.)
// ---------------------------------------------------------------------------
constexpr int kFewMax = 2 * kWave;

template <typename T, typename O, bool ADD, bool WHOLE>
__device__ __forceinline__ void sum_positions(const T* __restrict__ dout, O* __restrict__ grad, const GradArgs& a,
                                              uint32_t row, uint64_t low, uint64_t high, int64_t c)
{
    constexpr int N = GradCols<T, O>::value, kAhead = 8;
    const bool live = c < a.dim;
    const int64_t col = live ? c : 0, valid = a.dim - col, limit = (a.n - 1) * a.dout_stride + a.dim;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    int count = __builtin_popcountll(low) + __builtin_popcountll(high);
    for (; count > 0; count -= kAhead) {
        Pack<T, N> x[kAhead];
        int at[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            at[k] = low ? __builtin_ctzll(low) : high ? kWave + __builtin_ctzll(high) : at[k ? k - 1 : 0];
            if (low) low &= low - 1;
            else high &= high - 1;
            const int64_t from = at[k] * a.dout_stride + col;
            if (WHOLE || limit >= N) {
                x[k] = load_window<T, N>(dout, from, WHOLE ? INT64_MAX : limit);
            } else {
                T t[N];
#pragma unroll
                for (int j = 0; j < N; ++j) t[j] = j < valid ? dout[from + j] : (T)0.0f;
                __builtin_memcpy(&x[k], t, sizeof(t));
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (k < count) {  // uniform
                if constexpr (!WHOLE) {
                    const int64_t over = limit < N ? 0 : at[k] * a.dout_stride + col + N - limit;
                    if (ballot(over > 0)) shift_down<T, N>(x[k], over > 0 ? (int)over : 0);
                }
                T t[N];
                __builtin_memcpy(t, &x[k], sizeof(t));
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += (float)t[j];
            }
        }
    }
    if (!live) return;
    O* p = grad + (int64_t)row * a.grad_stride + c;
    float y[N], old[N];
#pragma unroll
    for (int j = 0; j < N; ++j) old[j] = 0.0f;
    if constexpr (ADD) load_floats<O, N>(p, valid, old);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = acc[j] * a.scale + (ADD ? old[j] : 0.0f);
    store_floats<O, N>(p, valid, y);
}

template <typename T, typename O, bool ADD, typename ID>
__global__ __launch_bounds__(kThreads) void embedding_few_kernel(const ID* __restrict__ ids, const T* __restrict__ dout,
                                                                 O* __restrict__ grad, GradArgs a, int64_t slabs,
                                                                 ClearArgs clear)
{
    constexpr int N = GradCols<T, O>::value;
    const int lane = lane_id();
    const uint32_t id0 = lane < a.n ? token_key(ids[lane], a.rows) : (uint32_t)a.rows;
    const uint32_t id1 = lane + kWave < a.n ? token_key(ids[lane + kWave], a.rows) : (uint32_t)a.rows;
    if (!ADD && blockIdx.x >= (uint32_t)clear.skip) {
        const int64_t r0 = clear.first + clear_wave<kThreads>(clear) * clear.per_wave;
        const int64_t r1 = r0 + clear.per_wave < clear.last ? r0 + clear.per_wave : clear.last;
        if (r0 >= r1) return;
        const auto within = [&](uint32_t id) { return (int64_t)id >= r0 && (int64_t)id < r1; };
        if (clear.stride_bytes == clear.row_bytes && !(ballot(within(id0)) | ballot(within(id1))))
            return clear_span(clear.grad + r0 * clear.stride_bytes, (r1 - r0) * clear.row_bytes);
        for (int64_t r = r0; r < r1; ++r)
            if (!(ballot((int64_t)id0 == r) | ballot((int64_t)id1 == r)))
                clear_span(clear.grad + r * clear.stride_bytes, clear.row_bytes);
        return;
    }
    const int64_t unit = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t i = unit / slabs, slab = unit % slabs, c = (slab * kWave + lane) * N;
    if (i >= a.n) return;
    const uint32_t row = i < kWave ? readlane(id0, (int)i) : readlane(id1, (int)i - kWave);
    if (row >= (uint32_t)a.rows) return;
    const uint64_t low = ballot(id0 == row), high = ballot(id1 == row);
    if ((low ? __builtin_ctzll(low) : kWave + __builtin_ctzll(high)) != i) return;  // not the row's first position
    if (a.dim % N == 0 || (slab + 1) * kWave * N <= a.dim)
        sum_positions<T, O, ADD, true>(dout, grad, a, row, low, high, c);
    else
        sum_positions<T, O, ADD, false>(dout, grad, a, row, low, high, c);
}

// The rows whose runs cross chunks: for each chunk in the list and 128 columns
// (two per lane), a wave adds the run's part there and the first parts of the
// chunks that it reaches. kJoinAhead parts are in flight: a frequent token
// fills hundreds of chunks, most runs two. (A workgroup per item, the parts
// split over its waves, took twice as long: most items are short, and it is
// their number that counts.) A row that has all tokens is one such chain, and
// its terms come in one wave per 128 columns: 65,536 tokens of 256 columns take
// 107 us then, 81 with half of them on one row, 49 spread over 50,000 rows;
// 1,000,003 tokens 1,290, 790 and 280.
constexpr int kJoinCols = 2;
constexpr int kJoinAhead = 16;

template <typename O, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(O* __restrict__ grad, GradArgs a, int64_t groups)
{
    const int lane = lane_id();
    const int64_t chunks = (a.n + a.chunk - 1) / a.chunk;
    int64_t u = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (; u < chunks * groups; u += (int64_t)gridDim.x * kWaves) {
        // loads that depend on each other are what this takes its time for: the item comes with the count
        const uint32_t count = a.crossing[0], item = a.crossing[1 + u / groups];
        if (u >= (int64_t)count * groups) return;
        const int64_t chunk = item, c = ((u % groups) * kWave + lane) * kJoinCols;
        const int64_t end = (chunk + 1) * a.chunk;
        // parts 0 (row 1 of this chunk) and 1 .. reached (row 0 of the next ones): rows 2 chunk + 1, + 2, + 4, ...
        const float* p = a.partial + (chunk * 2 + 1) * a.partial_stride + c;  // c < partial_stride
        float acc[kJoinCols], second[kJoinCols];
#pragma unroll
        for (int j = 0; j < kJoinCols; ++j) {
            acc[j] = p[j];
            second[j] = p[a.partial_stride + j];
        }
        const uint32_t begins = key_at(a, end + (int64_t)lane * a.chunk);  // keys that the next chunks begin with
        const uint32_t run = readlane(begins, 0);
        uint64_t other = ~ballot(begins == run);
        int64_t reached = other ? __builtin_ctzll(other) : kWave;  // chunks after this one that begin with the run
        while (!other) {
            other = ~ballot(key_at(a, end + (reached + lane) * a.chunk) == run);
            reached += other ? __builtin_ctzll(other) : kWave;
        }
#pragma unroll
        for (int j = 0; j < kJoinCols; ++j) acc[j] += second[j];
        for (int64_t q0 = 2; q0 <= reached; q0 += kJoinAhead) {
            float x[kJoinAhead][kJoinCols];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int64_t q = q0 + k <= reached ? q0 + k : reached;
#pragma unroll
                for (int j = 0; j < kJoinCols; ++j) x[k][j] = p[(2 * q - 1) * a.partial_stride + j];
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (q0 + k <= reached) {
#pragma unroll
                    for (int j = 0; j < kJoinCols; ++j) acc[j] += x[k][j];
                }
        }
        O* out = grad + (int64_t)run * a.grad_stride + c;
#pragma unroll
        for (int j = 0; j < kJoinCols; ++j) {
            if (c + j < a.dim) {
                float y = acc[j] * a.scale;
                if constexpr (ADD) y += (float)out[j];
                out[j] = (O)y;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes on a row, steps of a row and groups of rows in flight: the whole row or
// four steps of it, and eight steps in all where that leaves enough waves.
struct LookupShape {
    int lanes, steps, rows;
    int64_t blocks;
    LookupShape(ElemKind kind, int64_t n, int64_t dim)
    {
        const int64_t vecs = ceil_div(dim, kind == kF32 ? 4 : 8);
        lanes = 1;
        while (lanes < kWave && lanes < vecs) lanes *= 2;
        steps = vecs <= kWave ? 1 : 4;
        rows = ceil_div(n, kWave / lanes) >= 16384 ? 8 / steps : 1;
        blocks = ceil_div(n, (int64_t)(kWave / lanes) * rows * kWaves);
    }
};

int64_t embedding_blocks(ElemKind kind, int64_t n, int64_t dim) { return LookupShape(kind, n, dim).blocks; }

template <typename T, typename ID>
static hipError_t embedding_typed(ElemKind kind, const void* table, int64_t rows, int64_t dim, int64_t table_stride,
                                  const void* ids, int64_t n, float scale, void* out, int64_t out_stride,
                                  hipStream_t stream)
{
    const LookupShape s(kind, n, dim);
    const auto kernel = s.steps == 1 ? s.rows == 1 ? embedding_kernel<T, ID, 1, 1> : embedding_kernel<T, ID, 1, 8>
                        : s.rows == 1 ? embedding_kernel<T, ID, 4, 1> : embedding_kernel<T, ID, 4, 2>;
    kernel<<<dim3((unsigned)s.blocks), dim3(kThreads), 0, stream>>>((const T*)table, rows, dim, table_stride,
                                                                    (const ID*)ids, n, scale, (T*)out, out_stride,
                                                                    s.lanes);
    return hipGetLastError();
}

hipError_t launch_embedding(ElemKind kind, const void* table, int64_t rows, int64_t dim, int64_t table_stride,
                            const void* ids, bool wide_ids, int64_t n, float scale, void* out, int64_t out_stride,
                            hipStream_t stream)
{
#define DS_LOOKUP(T)                                                                                              \
    return wide_ids ? embedding_typed<T, int64_t>(kind, table, rows, dim, table_stride, ids, n, scale, out,       \
                                                  out_stride, stream)                                             \
                    : embedding_typed<T, int32_t>(kind, table, rows, dim, table_stride, ids, n, scale, out,       \
                                                  out_stride, stream)
    switch (kind) {
    case kF32: DS_LOOKUP(float);
    case kBF16: DS_LOOKUP(bf16);
    case kF16: DS_LOOKUP(fp16);
    default: return hipErrorInvalidValue;
    }
#undef DS_LOOKUP
}

int64_t embedding_most_rows() { return ((int64_t)1 << 27) - 1; }

// Positions per chunk: 64 where that leaves work for every CU, fewer for few
// tokens, so that more waves share the rows; but not above 512 chunks, because
// a frequent token's parts are added up one after another (32,768 tokens of 256
// columns: 58 us with 8 positions to a chunk, 39 with 32, 43 with 64).
static int sum_chunk(int64_t n, int64_t slabs)
{
    int chunk = 64;
    while (chunk > 8 && ceil_div(n, chunk) * slabs < 4096 && ceil_div(n, chunk) <= 512) chunk /= 2;
    return chunk;
}

EmbeddingGradPlan embedding_grad_plan(ElemKind grad_kind, int64_t n, int64_t rows, int64_t dim)
{
    EmbeddingGradPlan p{};
    const int64_t per = grad_kind == kF32 ? 4 : 8;  // columns per lane
    p.slabs = ceil_div(dim, kWave * per);
    p.chunk = sum_chunk(n, p.slabs);
    p.chunks = ceil_div(n, p.chunk);
    p.partial_stride = p.slabs * kWave * per;
    if (n <= kFewMax) return p;
    int bits = 1;
    while (((int64_t)1 << bits) < rows + 1) ++bits;
    if (n > kTileSortMax) {
        p.radix_bits = 8;
        p.digits = (bits + 7) / 8;
        p.table_words = sort_aux_words(true, n, p.radix_bits);
        // A table of more than one tile is scanned without the look-back: a wait there that gave up would leave words
        // of earlier calls among the sorted keys and positions, and the sums take both for addresses. (Three passes,
        // rows of 8: 1,000,003 tokens, one launch per scan, 280 us against 276 with the look-back; 2,000,003, three
        // launches per scan, 463 against 445.)
        const int64_t words = ((int64_t)1 << p.radix_bits) * sort_table_columns(true, n);
        if (words > tile_elems(kU32, false, words)) p.totals_words = ceil_div(words, three_pass_tile_elems(4));
        p.table_words += p.totals_words;
    } else if (n > kRankSortMax) {
        p.digits = (bits + kDigitBits - 1) / kDigitBits;
        p.bits = (bits + p.digits - 1) / p.digits;
        p.items = n > kTileSortMax / 2 ? 4 : 2;
        p.tiles = (int)ceil_div(n, kTileThreads * p.items);
        p.table_words = (int64_t)p.tiles << p.bits;
    }
    p.table_words = ceil_div(p.table_words, 4) * 4;
    // keys and index, twice where passes go back and forth; then the parts of rows, 16-byte aligned
    p.crossing_at = p.table_words + n * (p.digits ? 4 : 2);
    const int64_t words = p.crossing_at + 1 + p.chunks;
    p.partial_at = ceil_div(words, 4) * 16;
    p.bytes = p.partial_at + p.chunks * 2 * p.partial_stride * 4;
    return p;
}

// What each launch of a call clears.
struct Clearing {
    ClearArgs a;
    int64_t rows, share;
    // A sort's launch takes about 5 us, in which this much can be cleared.
    static constexpr int64_t kShareBytes = 24 << 20;
    Clearing(bool add, void* grad, int64_t rows_, int64_t dim, int64_t stride, int esz)
    {
        a = ClearArgs{static_cast<char*>(grad), dim * esz, stride * esz, 0, 0, 0, 1};
        rows = add ? 0 : rows_;
        share = ceil_div(kShareBytes, a.row_bytes);
    }
    // The part of a launch that has `before` workgroups of `threads` of its own: its share, or all that is left;
    // others: but for rows that have tokens. Returns the workgroups in all.
    unsigned next(int64_t before, int threads, bool all = false, bool others = false)
    {
        a.first = a.last;
        a.last = all || rows - a.first < share ? rows : a.first + share;
        a.skip = (int)before;
        // as many rows to a wave as leave 8,192 waves (the lanes of a wave look for one row each)
        const int64_t each = (a.last - a.first) / 8192;
        a.per_wave = (int)(each < 1 ? 1 : each < kWave ? each : kWave);
        int64_t waves = ceil_div(a.last - a.first, a.per_wave);
        if (!others && a.last > a.first && a.stride_bytes == a.row_bytes)
            waves = ceil_div(a.last * a.row_bytes, kPiece) - a.first * a.row_bytes / kPiece;
        return (unsigned)(before + ceil_div(waves, threads / kWave));
    }
};

// All in one launch, for few tokens.
template <typename T, typename O, bool ADD>
static hipError_t embedding_few_typed(const EmbeddingGradPlan& p, const void* ids, bool wide_ids, const void* dout,
                                      void* grad, const GradArgs& a, Clearing& clear, hipStream_t stream)
{
    unsigned blocks = clear.next(ceil_div(a.n * p.slabs, kWaves), kThreads, true, true);
    // spans of some kilobytes, where rows are short: waves that share a cache line are slow
    const int64_t each = ceil_div(4 * kPiece, clear.a.row_bytes);
    if (clear.a.per_wave < each) {
        clear.a.per_wave = (int)(each < 1024 ? each : 1024);
        blocks = (unsigned)(clear.a.skip + ceil_div(ceil_div(clear.a.last - clear.a.first, clear.a.per_wave), kWaves));
    }
    if (wide_ids)
        embedding_few_kernel<T, O, ADD><<<dim3(blocks), dim3(kThreads), 0, stream>>>((const int64_t*)ids, (const T*)dout,
                                                                                     (O*)grad, a, p.slabs, clear.a);
    else
        embedding_few_kernel<T, O, ADD><<<dim3(blocks), dim3(kThreads), 0, stream>>>((const int32_t*)ids, (const T*)dout,
                                                                                     (O*)grad, a, p.slabs, clear.a);
    return hipGetLastError();
}

template <typename T, typename O, bool ADD>
static hipError_t embedding_grad_typed(const EmbeddingGradPlan& p, const void* dout, void* grad, const GradArgs& a,
                                       Clearing& clear, hipStream_t stream)
{
    const int64_t units = p.chunks * p.slabs;
    const unsigned blocks = clear.next(ceil_div(units, kWaves), kThreads, true, true);
    embedding_sum_kernel<T, O, ADD><<<dim3(blocks), dim3(kThreads), 0, stream>>>((const T*)dout, (O*)grad, a, p.slabs,
                                                                                 units, clear.a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t groups = ceil_div(a.dim, kWave * kJoinCols), joins = ceil_div(p.chunks * groups, kWaves);
    embedding_join_kernel<O, ADD><<<dim3((unsigned)(joins < 2048 ? joins : 2048)), dim3(kThreads), 0, stream>>>(
        (O*)grad, a, groups);
    return hipGetLastError();
}

int64_t embedding_grad_blocks(const EmbeddingGradPlan& p, int64_t n, int64_t rows, int64_t row_bytes)
{
    const int64_t sum = ceil_div(p.chunks * p.slabs, kWaves), keys = ceil_div(n, kThreads);
    const int64_t clear = ceil_div(rows * row_bytes, kPiece * kWaves) + ceil_div(rows, kWaves * kWave) + 8192;
    return (sum > keys ? sum : keys) + clear;
}

hipError_t launch_embedding_grad(ElemKind kind, ElemKind grad_kind, const EmbeddingGradPlan& p, const void* dout,
                                 int64_t dout_stride, const void* ids, bool wide_ids, int64_t n, int64_t rows,
                                 int64_t dim, float scale, void* grad, int64_t grad_stride, bool add, char* aux,
                                 hipStream_t stream)
{
    hipError_t e = hipSuccess;
    uint32_t* table = reinterpret_cast<uint32_t*>(aux);
    uint32_t* keys = table + p.table_words;
    uint32_t *index = keys + n, *keys2 = index + n, *index2 = keys2 + n;
    const bool tiled = p.tiles > 0;
    uint32_t* crossing = table + p.crossing_at;
    Clearing clear(add, grad, rows, dim, grad_stride, grad_kind == kF32 ? 4 : 2);
    if (n <= kFewMax) {
        const GradArgs a{nullptr, nullptr, n, rows, dim, dout_stride, grad_stride, 0, scale, nullptr, 0, nullptr};
#define DS_FEW(T, O)                                                                                \
    return add ? embedding_few_typed<T, O, true>(p, ids, wide_ids, dout, grad, a, clear, stream) \
               : embedding_few_typed<T, O, false>(p, ids, wide_ids, dout, grad, a, clear, stream)
        if (kind == kF32 && grad_kind == kF32) DS_FEW(float, float);
        if (kind == kBF16 && grad_kind == kBF16) DS_FEW(bf16, bf16);
        if (kind == kBF16 && grad_kind == kF32) DS_FEW(bf16, float);
        if (kind == kF16 && grad_kind == kF16) DS_FEW(fp16, fp16);
        if (kind == kF16 && grad_kind == kF32) DS_FEW(fp16, float);
#undef DS_FEW
        return hipErrorInvalidValue;
    }
    if (p.radix_bits) {
        const unsigned grid = clear.next(ceil_div(n, kThreads), kThreads);
        if (wide_ids)
            token_keys_kernel<<<dim3(grid), dim3(kThreads), 0, stream>>>((const int64_t*)ids, n, rows, keys, index,
                                                                         crossing, clear.a);
        else
            token_keys_kernel<<<dim3(grid), dim3(kThreads), 0, stream>>>((const int32_t*)ids, n, rows, keys, index,
                                                                         crossing, clear.a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t totals_at = sort_aux_words(true, n, p.radix_bits);
        const DevWs ws{nullptr, nullptr, p.totals_words ? table + totals_at : nullptr};
        for (int d = 0; d < p.digits; ++d) {
            e = launch_radix_pass(keys, index, keys2, index2, n, d * p.radix_bits, p.radix_bits, table, ws, 1, stream);
            if (e != hipSuccess) return e;
            uint32_t* t = keys; keys = keys2; keys2 = t;
            t = index; index = index2; index2 = t;
        }
    } else if (tiled) {
        const TileSort a{(uint32_t)n, rows, p.bits, p.digits, p.items, p.tiles, table};
        for (int d = 0; d < p.digits; ++d) {
            const void* from = d ? nullptr : ids;
            unsigned grid = clear.next(p.tiles, kTileThreads);
            if (wide_ids)
                token_count_kernel<<<dim3(grid), dim3(kTileThreads), 0, stream>>>((const int64_t*)from, a, d, keys,
                                                                                  crossing, clear.a);
            else
                token_count_kernel<<<dim3(grid), dim3(kTileThreads), 0, stream>>>((const int32_t*)from, a, d, keys,
                                                                                  crossing, clear.a);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
            grid = clear.next(p.tiles, kTileThreads);
            const auto kernel = p.items == 2 ? token_pass_kernel<2> : token_pass_kernel<4>;
            kernel<<<dim3(grid), dim3(kTileThreads), 0, stream>>>(keys, d ? index : nullptr, a, d, keys2, index2, clear.a);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
            uint32_t* t = keys; keys = keys2; keys2 = t;
            t = index; index = index2; index2 = t;
        }
    } else {
        // All of it where few rows can have tokens: two launches that clear cost more than some rows cleared in vain
        // (1,003 tokens, 32,000 rows of 1,000: 17.3 us for both against 19.2).
        const unsigned grid = clear.next(ceil_div(n, kRankTokens), kThreads, n <= rows / 8);
        const size_t lds = (size_t)((n + 63) / 64 * 64) * 4;
        if (wide_ids)
            token_rank_sort_kernel<<<dim3(grid), dim3(kThreads), lds, stream>>>((const int64_t*)ids, (uint32_t)n, rows,
                                                                               keys, index, crossing, clear.a);
        else
            token_rank_sort_kernel<<<dim3(grid), dim3(kThreads), lds, stream>>>((const int32_t*)ids, (uint32_t)n, rows,
                                                                               keys, index, crossing, clear.a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const GradArgs a{keys, index, n, rows, dim, dout_stride, grad_stride, p.chunk, scale,
                     reinterpret_cast<float*>(aux + p.partial_at), p.partial_stride, crossing};
#define DS_GRAD(T, O)                                                              \
    return add ? embedding_grad_typed<T, O, true>(p, dout, grad, a, clear, stream) \
               : embedding_grad_typed<T, O, false>(p, dout, grad, a, clear, stream)
    if (kind == kF32 && grad_kind == kF32) DS_GRAD(float, float);
    if (kind == kBF16 && grad_kind == kBF16) DS_GRAD(bf16, bf16);
    if (kind == kBF16 && grad_kind == kF32) DS_GRAD(bf16, float);
    if (kind == kF16 && grad_kind == kF16) DS_GRAD(fp16, fp16);
    if (kind == kF16 && grad_kind == kF32) DS_GRAD(fp16, float);
#undef DS_GRAD
    return hipErrorInvalidValue;
}

}  // namespace ds
