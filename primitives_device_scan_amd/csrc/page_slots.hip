// page_slots.hip -- page tables and slot maps of a ragged batch of requests
// whose caches are held in pages: with held_r = ceil(context_r / page) and
// need_r = ceil((context_r + new_r) / page) - held_r,
//
//   offsets = exclusive prefix sum of new, q = exclusive prefix sum of need
//   tables[r, held_r + j] = free[count - 1 - (q_r + j)]                j < need_r
//   slots[offsets_r + i] = tables[r, p / page] * page + p % page       p = context_r + i, i < new_r
//
// The bytes are few (8 a request, 12 a token), so a launch's latency and the
// two prefix sums are the time. One launch does all: every workgroup scans all
// requests itself (from the L2) and serves its share of the tokens and pages.
// Slots of pages that this call takes are worked out from the free list, not
// read back from the tables, so that workgroups need not wait for each other.
#include "launch.hpp"
#include "tile.hpp"

namespace ds {

constexpr int kPageThreads = 1024;
constexpr int kPageWaves = kPageThreads / kWave;

// The last i of [0, n) with first[i] <= v, where first[0] <= v and first does
// not decrease.
__device__ __forceinline__ int last_at_most(const int64_t* first, int n, int64_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPageThreads) void page_slots_kernel(PageSlots a)
{
    __shared__ int64_t s_tokens[kPageThreads + 1], s_pages[kPageThreads + 1];  // first of each request in the chunk
    __shared__ int64_t s_wave[2][kPageWaves];
    __shared__ int32_t s_context[kPageThreads];
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int64_t top = min(max((int64_t)*a.count, (int64_t)0), a.capacity) - 1;
    const int64_t page = a.page;
    const auto free_page = [&](int64_t q) { return q <= top ? a.free_pages[top - q] : -1; };
    int64_t tokens = 0, pages = 0;  // of the requests before the chunk
    for (int64_t base = 0; base < a.requests; base += kPageThreads) {
        const int64_t r = base + threadIdx.x;
        const int here = (int)min((int64_t)kPageThreads, a.requests - base);
        const int64_t context = r < a.requests ? max(a.context[r], 0) : 0;
        const int64_t fresh = r < a.requests ? max(a.fresh[r], 0) : 0;
        const int64_t held = (context + page - 1) / page;
        const int64_t need = (context + fresh + page - 1) / page - held;
        const int64_t tokens_to = wave_inclusive_scan(fresh), pages_to = wave_inclusive_scan(need);
        if (lane == kWave - 1) {
            s_wave[0][wave] = tokens_to;
            s_wave[1][wave] = pages_to;
        }
        __syncthreads();
        int64_t t0 = tokens, p0 = pages;
        for (int w = 0; w < kPageWaves; ++w) {
            if (w < wave) {
                t0 += s_wave[0][w];
                p0 += s_wave[1][w];
            }
            tokens += s_wave[0][w];
            pages += s_wave[1][w];
        }
        s_tokens[threadIdx.x] = t0 + tokens_to - fresh;
        s_pages[threadIdx.x] = p0 + pages_to - need;
        s_context[threadIdx.x] = (int32_t)context;
        if (blockIdx.x == 0 && r < a.requests)
            a.offsets[r] = (int32_t)min(t0 + tokens_to - fresh, (int64_t)INT32_MAX);
        __syncthreads();
        const int64_t first_token = s_tokens[0], first_page = s_pages[0];
        // pages that the chunk's requests take
        for (int64_t q = first_page + blockIdx.x * kPageThreads + threadIdx.x; q < pages;
             q += (int64_t)gridDim.x * kPageThreads) {
            const int i = last_at_most(s_pages, here, q);
            const int64_t col = (s_context[i] + page - 1) / page + q - s_pages[i];
            if (col < a.width) a.tables[(base + i) * a.table_stride + col] = free_page(q);
        }
        // their tokens
        const int64_t end = min(tokens, a.tokens);
        for (int64_t t = first_token + blockIdx.x * kPageThreads + threadIdx.x; t < end;
             t += (int64_t)gridDim.x * kPageThreads) {
            const int i = last_at_most(s_tokens, here, t);
            const int64_t position = s_context[i] + t - s_tokens[i];
            const int64_t col = position / page, own = (s_context[i] + page - 1) / page;
            int64_t id = -1;
            if (col < a.width)
                id = col < own ? a.tables[(base + i) * a.table_stride + col] : free_page(s_pages[i] + col - own);
            a.slots[t] = id < 0 ? -1 : id * page + position % page;
            a.positions[t] = (int32_t)min(position, (int64_t)INT32_MAX);
        }
        __syncthreads();
    }
    for (int64_t t = min(tokens, a.tokens) + blockIdx.x * kPageThreads + threadIdx.x; t < a.tokens;
         t += (int64_t)gridDim.x * kPageThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.offsets[a.requests] = (int32_t)min(tokens, (int64_t)INT32_MAX);
        *a.left = (int32_t)max(top + 1 - pages, (int64_t)INT32_MIN);
    }
}

hipError_t launch_page_slots(const PageSlots& a, hipStream_t stream)
{
    // a workgroup for every 4,096 tokens: each scans all requests again
    int64_t blocks = (a.tokens + 4095) / 4096;
    blocks = blocks < 1 ? 1 : blocks > 256 ? 256 : blocks;
    page_slots_kernel<<<dim3((unsigned)blocks), dim3(kPageThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ds
