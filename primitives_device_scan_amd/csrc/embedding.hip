// embedding.hip -- token embedding (rows of a table by token id, scaled) and
// the gradient of the table.
//
//   out[i] = scale * table[ids[i]]                 (zero where ids[i] is no row)
//   grad[v] = scale * sum over i with ids[i] = v of dout[i]    (+ grad[v])
//
// The gradient goes by sorted tokens: the positions i are put in order of
// their token (equal tokens in input order), so that each row's terms are
// consecutive, and are then summed in that order: no atomics on the sums, and
// the same bits on every run. Up to kRankSortMax tokens one launch sorts
// (every token's place is the number of tokens that sort before it, counted
// directly); above, two or three passes of the stable counting sort do.
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

// ---------------------------------------------------------------------------
// Lookup. A wave takes whole rows: `lanes` lanes (a power of two) side by side
// on one row, 64 / lanes rows at once, 16 bytes per lane and step.
// ---------------------------------------------------------------------------
template <typename T, typename ID>
__global__ __launch_bounds__(kThreads) void embedding_kernel(const T* __restrict__ table, int64_t rows, int64_t dim,
                                                             int64_t table_stride, const ID* __restrict__ ids,
                                                             int64_t n, float scale, T* __restrict__ out,
                                                             int64_t out_stride, int lanes)
{
    constexpr int N = Vec16<T>::kN;
    const int per_wave = kWave / lanes;
    const int64_t wave = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    const int64_t i = wave * per_wave + lane_id() / lanes;
    if (i >= n) return;
    const int64_t id = (int64_t)ids[i];
    const bool live = id >= 0 && id < rows;
    const T* src = table + (live ? id : 0) * table_stride;
    T* dst = out + i * out_stride;
    for (int64_t c = (int64_t)(lane_id() % lanes) * N; c < dim; c += (int64_t)lanes * N) {
        float x[N];
        if (live) {
            load_floats<T, N>(src + c, dim - c, x);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] *= scale;
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = 0.0f;
        }
        store_floats<T, N>(dst + c, dim - c, x);
    }
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

constexpr int64_t kRankSortMax = 8192;
constexpr int kRankParts = 16;                     // lanes that count for one token
constexpr int kRankTokens = kThreads / kRankParts; // tokens per workgroup

// place(i) = #{j : key_j < key_i} + #{j < i : key_j = key_i}. Every workgroup
// holds all keys in LDS; 16 lanes share one token's count.
template <typename ID>
__global__ __launch_bounds__(kThreads) void token_rank_sort_kernel(const ID* __restrict__ ids, uint32_t n,
                                                                   int64_t rows, uint32_t* __restrict__ keys,
                                                                   uint32_t* __restrict__ places)
{
    extern __shared__ __align__(16) uint32_t s_key[];  // n rounded up to 64 keys
    const uint32_t padded = (n + 63u) & ~63u;
    for (uint32_t j = threadIdx.x; j < padded; j += kThreads) s_key[j] = j < n ? token_key(ids[j], rows) : 0xFFFFFFFFu;
    __syncthreads();
    const uint32_t i = blockIdx.x * kRankTokens + threadIdx.x / kRankParts, part = threadIdx.x % kRankParts;
    const uint32_t key = i < n ? s_key[i] : 0u;
    uint32_t below = 0;
    for (uint32_t j = part * 4; j < padded; j += kRankParts * 4) {
        const u32x4 k = *reinterpret_cast<const u32x4*>(s_key + j);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) below += k[q] < key + (j + q < i ? 1u : 0u) ? 1u : 0u;
    }
    below += dpp<0x111>(below);  // sums over the row of 16 lanes: row_shr 1, 2, 4, 8
    below += dpp<0x112>(below);
    below += dpp<0x114>(below);
    below += dpp<0x118>(below);
    if (part == kRankParts - 1 && i < n) {
        keys[below] = key;
        places[below] = i;
    }
}

// Keys for the counting-sort passes: the key written in base `base` (at most
// 511, the most buckets a pass has), kDigitBits bits to a digit, so that two
// passes order up to 511^2 - 1 = 261,120 rows where 8-bit digits would need
// three. Digits keep the order of the keys.
constexpr int kDigitBits = 9;

template <typename ID>
__global__ __launch_bounds__(kThreads) void token_digits_kernel(const ID* __restrict__ ids, int64_t n, int64_t rows,
                                                                uint32_t base, int digits,
                                                                uint32_t* __restrict__ keys,
                                                                uint32_t* __restrict__ index)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    uint32_t key = token_key(ids[i], rows), packed = 0;
    for (int d = 0; d < digits; ++d) {
        packed |= (key % base) << (d * kDigitBits);
        key /= base;
    }
    keys[i] = packed;
    index[i] = (uint32_t)i;
}

__device__ __forceinline__ uint32_t digits_key(uint32_t packed, uint32_t base, int digits)
{
    uint32_t key = 0;
    for (int d = digits - 1; d >= 0; --d) key = key * base + ((packed >> (d * kDigitBits)) & ((1u << kDigitBits) - 1u));
    return key;
}

// ---------------------------------------------------------------------------
// Sums. The sorted positions are cut into chunks of `chunk` (8 to 64), the
// columns into slabs of one 16-byte access per lane; a wave adds up one chunk
// of one slab, run by run. A run that lies inside its chunk is a whole row of
// the gradient. The part of a run that crosses a chunk's edge goes to
// `partial` (two 32-bit rows per chunk: 0 for a run that began in an earlier
// chunk, 1 for one that begins here and goes on), and embedding_join_kernel
// adds the parts up in order.
// ---------------------------------------------------------------------------
struct GradArgs {
    const uint32_t* keys;   // sorted; packed digits where digits > 0
    const uint32_t* index;  // position of each sorted token in the input
    int64_t n, rows, dim, dout_stride, grad_stride;
    uint32_t base;
    int digits, chunk, add;
    float scale;
    float* partial;  // [chunks][2][dim rounded up to whole slabs]
    int64_t partial_stride;
};

__device__ __forceinline__ uint32_t key_at(const GradArgs& a, int64_t p)
{
    if (p < 0 || p >= a.n) return 0xFFFFFFFFu;
    const uint32_t k = a.keys[p];
    return a.digits ? digits_key(k, a.base, a.digits) : k;
}

template <typename O, int N>
__device__ __forceinline__ void write_row(const GradArgs& a, O* grad, uint32_t key, int64_t c, const float (&acc)[N])
{
    O* p = grad + (int64_t)key * a.grad_stride + c;
    const int64_t valid = a.dim - c;
    float x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = acc[j] * a.scale;
    if (a.add) {
        constexpr int kPer = Vec16<O>::kN;
#pragma unroll
        for (int v = 0; v < N / kPer; ++v) {
            float old[kPer];
            load_floats<O, kPer>(p + v * kPer, valid - v * kPer, old);
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[v * kPer + j] += old[j];
        }
    }
    store_floats<O, N>(p, valid, x);
}

template <int N>
__device__ __forceinline__ void write_partial(const GradArgs& a, int64_t chunk, int which, int64_t c,
                                              const float (&acc)[N])
{
    store_floats<float, N>(a.partial + (chunk * 2 + which) * a.partial_stride + c, N, acc);
}

template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void embedding_sum_kernel(const T* __restrict__ dout, O* __restrict__ grad,
                                                                 GradArgs a, int64_t slabs, int64_t units)
{
    constexpr int N = Vec16<T>::kN;
    constexpr int kAhead = 8;  // rows in flight
    const int64_t unit = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit >= units) return;
    const int64_t chunk = unit / slabs, c = ((unit % slabs) * kWave + lane_id()) * N;
    const int64_t p0 = chunk * a.chunk;
    const int lane = lane_id();
    const uint32_t key = lane < a.chunk ? key_at(a, p0 + lane) : 0xFFFFFFFFu;
    const uint32_t before = key_at(a, p0 - 1), after = key_at(a, p0 + a.chunk);
    const uint32_t index = lane < a.chunk && p0 + lane < a.n ? a.index[p0 + lane] : 0u;
    const int count = __builtin_popcountll(ballot(key < (uint32_t)a.rows));
    if (count == 0) return;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    uint32_t run = readlane(key, 0);
    bool opened = run == before;  // the current run began in an earlier chunk
    const bool live = c < a.dim;
    for (int i0 = 0; i0 < count; i0 += kAhead) {
        float x[kAhead][N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < count && live)
                load_floats<T, N>(dout + (int64_t)readlane(index, i0 + i) * a.dout_stride + c, a.dim - c, x[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i < count) {
                const uint32_t k = readlane(key, i0 + i);
                if (k != run) {
                    if (live) {
                        if (opened)
                            write_partial<N>(a, chunk, 0, c, acc);
                        else
                            write_row<O, N>(a, grad, run, c, acc);
                    }
                    opened = false;
                    run = k;
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += x[i][j];
            }
        }
    }
    if (!live) return;
    if (opened)
        write_partial<N>(a, chunk, 0, c, acc);
    else if (run == after)
        write_partial<N>(a, chunk, 1, c, acc);
    else
        write_row<O, N>(a, grad, run, c, acc);
}

// The rows whose runs cross chunks: the wave of the chunk in which such a run
// begins adds its part and the first parts of the chunks that it reaches.
template <typename O, int N>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(O* __restrict__ grad, GradArgs a, int64_t slabs,
                                                                  int64_t units)
{
    const int64_t unit = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit >= units) return;
    const int64_t chunk = unit / slabs, c = ((unit % slabs) * kWave + lane_id()) * N;
    const int64_t p0 = chunk * a.chunk, end = p0 + a.chunk;
    const uint32_t run = key_at(a, end - 1);
    if (run >= (uint32_t)a.rows || run != key_at(a, end)) return;      // no run goes on from here
    if (run == key_at(a, p0) && run == key_at(a, p0 - 1)) return;      // it began earlier
    if (c >= a.dim) return;
    float acc[N];
    const float* p = a.partial + (chunk * 2 + 1) * a.partial_stride + c;
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = p[j];
    for (int64_t q = chunk + 1; key_at(a, q * a.chunk) == run; ++q) {
        p = a.partial + q * 2 * a.partial_stride + c;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += p[j];
    }
    write_row<O, N>(a, grad, run, c, acc);
}

// Zeros for a whole gradient (rows of `dim` elements, `stride` apart).
template <typename O>
__global__ __launch_bounds__(kThreads) void embedding_clear_kernel(O* __restrict__ grad, int64_t rows, int64_t dim,
                                                                   int64_t stride, int64_t slabs)
{
    constexpr int N = Vec16<O>::kN;
    const int64_t units = rows * slabs, waves = (int64_t)gridDim.x * kWaves;
    for (int64_t u = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave; u < units; u += waves) {
        const int64_t c = ((u % slabs) * kWave + lane_id()) * N;
        const float x[N] = {};
        if (c < dim) store_floats<O, N>(grad + (u / slabs) * stride + c, dim - c, x);
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static int lookup_lanes(ElemKind kind, int64_t dim)
{
    const int64_t vecs = ceil_div(dim, kind == kF32 ? 4 : 8);
    int lanes = 1;
    while (lanes < kWave && lanes < vecs) lanes *= 2;
    return lanes;
}

int64_t embedding_blocks(ElemKind kind, int64_t n, int64_t dim)
{
    return ceil_div(ceil_div(n, kWave / lookup_lanes(kind, dim)), kWaves);
}

template <typename T>
static hipError_t embedding_typed(ElemKind kind, const void* table, int64_t rows, int64_t dim, int64_t table_stride,
                                  const void* ids, bool wide_ids, int64_t n, float scale, void* out,
                                  int64_t out_stride, hipStream_t stream)
{
    const dim3 grid((unsigned)embedding_blocks(kind, n, dim)), block(kThreads);
    const int lanes = lookup_lanes(kind, dim);
    if (wide_ids)
        embedding_kernel<T, int64_t><<<grid, block, 0, stream>>>((const T*)table, rows, dim, table_stride,
                                                                 (const int64_t*)ids, n, scale, (T*)out, out_stride,
                                                                 lanes);
    else
        embedding_kernel<T, int32_t><<<grid, block, 0, stream>>>((const T*)table, rows, dim, table_stride,
                                                                 (const int32_t*)ids, n, scale, (T*)out, out_stride,
                                                                 lanes);
    return hipGetLastError();
}

hipError_t launch_embedding(ElemKind kind, const void* table, int64_t rows, int64_t dim, int64_t table_stride,
                            const void* ids, bool wide_ids, int64_t n, float scale, void* out, int64_t out_stride,
                            hipStream_t stream)
{
    switch (kind) {
    case kF32: return embedding_typed<float>(kind, table, rows, dim, table_stride, ids, wide_ids, n, scale, out, out_stride, stream);
    case kBF16: return embedding_typed<bf16>(kind, table, rows, dim, table_stride, ids, wide_ids, n, scale, out, out_stride, stream);
    case kF16: return embedding_typed<fp16>(kind, table, rows, dim, table_stride, ids, wide_ids, n, scale, out, out_stride, stream);
    default: return hipErrorInvalidValue;
    }
}

int64_t embedding_most_rows()
{
    const int64_t most = sort_max_buckets();  // three digits of kDigitBits bits fit a 32-bit key
    return most * most * most - 1;
}

// Digits of the counting-sort passes: the fewest, and the smallest base that
// still holds the keys 0 .. rows.
static void sort_digits(int64_t rows, uint32_t* base, int* digits)
{
    const int64_t most = sort_max_buckets();
    int d = 1;
    for (int64_t reach = most; reach < rows + 1; reach *= most) ++d;
    int64_t b = 2;
    for (;; ++b) {
        int64_t reach = 1;
        for (int i = 0; i < d; ++i) reach *= b;
        if (reach >= rows + 1) break;
    }
    *base = (uint32_t)b;
    *digits = d;
}

// Positions per chunk: 64 where that leaves work for every CU, fewer for few
// tokens, so that more waves share the rows.
static int sum_chunk(int64_t n, int64_t slabs)
{
    int chunk = 64;
    while (chunk > 8 && ceil_div(n, chunk) * slabs < 4096) chunk /= 2;
    return chunk;
}

EmbeddingGradPlan embedding_grad_plan(ElemKind kind, int64_t n, int64_t rows, int64_t dim)
{
    EmbeddingGradPlan p{};
    const int64_t per = kind == kF32 ? 4 : 8;
    p.slabs = ceil_div(dim, kWave * per);
    p.chunk = sum_chunk(n, p.slabs);
    p.chunks = ceil_div(n, p.chunk);
    p.partial_stride = p.slabs * kWave * per;
    if (n > kRankSortMax) sort_digits(rows, &p.base, &p.digits);
    p.table_words = p.digits ? sort_pass_words(n, p.base) : 0;
    // keys and index, twice where passes go back and forth; then the parts of rows, 16-byte aligned
    const int64_t words = p.table_words + n * (p.digits ? 4 : 2);
    p.partial_at = ceil_div(words, 4) * 16;
    p.bytes = p.partial_at + p.chunks * 2 * p.partial_stride * 4;
    return p;
}

template <typename T, typename O>
static hipError_t embedding_grad_typed(const EmbeddingGradPlan& p, const void* dout, int64_t dout_stride, int64_t n,
                                       int64_t rows, int64_t dim, float scale, void* grad, int64_t grad_stride,
                                       bool add, const uint32_t* keys, const uint32_t* index, char* aux,
                                       hipStream_t stream)
{
    constexpr int N = Vec16<T>::kN;
    const GradArgs a{keys, index, n, rows, dim, dout_stride, grad_stride, p.base, p.digits, p.chunk, add ? 1 : 0,
                     scale, reinterpret_cast<float*>(aux + p.partial_at), p.partial_stride};
    const int64_t units = p.chunks * p.slabs;
    const dim3 grid((unsigned)ceil_div(units, kWaves)), block(kThreads);
    embedding_sum_kernel<T, O><<<grid, block, 0, stream>>>((const T*)dout, (O*)grad, a, p.slabs, units);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    embedding_join_kernel<O, N><<<grid, block, 0, stream>>>((O*)grad, a, p.slabs, units);
    return hipGetLastError();
}

template <typename O>
static hipError_t clear_typed(void* grad, int64_t rows, int64_t dim, int64_t stride, hipStream_t stream)
{
    const int64_t slabs = ceil_div(dim, kWave * Vec16<O>::kN);
    const int64_t blocks = ceil_div(rows * slabs, kWaves);
    embedding_clear_kernel<O><<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, stream>>>(
        (O*)grad, rows, dim, stride, slabs);
    return hipGetLastError();
}

hipError_t launch_embedding_grad(ElemKind kind, ElemKind grad_kind, const EmbeddingGradPlan& p, const void* dout,
                                 int64_t dout_stride, const void* ids, bool wide_ids, int64_t n, int64_t rows,
                                 int64_t dim, float scale, void* grad, int64_t grad_stride, bool add, char* aux,
                                 const DevWs& ws, uint32_t spin_limit, hipStream_t stream)
{
    hipError_t e = hipSuccess;
    if (!add) {
        if (grad_kind == kF32) e = clear_typed<float>(grad, rows, dim, grad_stride, stream);
        else e = clear_typed<bf16>(grad, rows, dim, grad_stride, stream);  // any 16-bit type: zero bits
        if (e != hipSuccess) return e;
    }
    if (n == 0) return hipSuccess;
    uint32_t* table = reinterpret_cast<uint32_t*>(aux);
    uint32_t* keys = table + p.table_words;
    uint32_t* index = keys + n;
    if (!p.digits) {
        const dim3 grid((unsigned)ceil_div(n, kRankTokens)), block(kThreads);
        const size_t lds = (size_t)((n + 63) / 64 * 64) * 4;
        if (wide_ids)
            token_rank_sort_kernel<int64_t><<<grid, block, lds, stream>>>((const int64_t*)ids, (uint32_t)n, rows, keys, index);
        else
            token_rank_sort_kernel<int32_t><<<grid, block, lds, stream>>>((const int32_t*)ids, (uint32_t)n, rows, keys, index);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else {
        const dim3 grid((unsigned)ceil_div(n, kThreads)), block(kThreads);
        if (wide_ids)
            token_digits_kernel<int64_t><<<grid, block, 0, stream>>>((const int64_t*)ids, n, rows, p.base, p.digits, keys, index);
        else
            token_digits_kernel<int32_t><<<grid, block, 0, stream>>>((const int32_t*)ids, n, rows, p.base, p.digits, keys, index);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        uint32_t *keys2 = index + n, *index2 = keys2 + n;
        for (int d = 0; d < p.digits; ++d) {
            e = launch_sort_pass(keys, index, keys2, index2, n, d * kDigitBits, p.base, table, ws, spin_limit, stream);
            if (e != hipSuccess) return e;
            uint32_t* t = keys; keys = keys2; keys2 = t;
            t = index; index = index2; index2 = t;
        }
    }
#define DS_GRAD(T, O) \
    return embedding_grad_typed<T, O>(p, dout, dout_stride, n, rows, dim, scale, grad, grad_stride, add, keys, index, aux, stream)
    if (kind == kF32 && grad_kind == kF32) DS_GRAD(float, float);
    if (kind == kBF16 && grad_kind == kBF16) DS_GRAD(bf16, bf16);
    if (kind == kBF16 && grad_kind == kF32) DS_GRAD(bf16, float);
    if (kind == kF16 && grad_kind == kF16) DS_GRAD(fp16, fp16);
    if (kind == kF16 && grad_kind == kF32) DS_GRAD(fp16, float);
#undef DS_GRAD
    return hipErrorInvalidValue;
}

}  // namespace ds
