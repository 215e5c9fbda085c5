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
// requests itself (from the L2) and serves its share of the tokens and pages (256
// requests of one token each: 5.0 us; 512 of up to 512, 133,000 tokens: 9.8, where
// the bytes take 0.3; a binary search of the requests in LDS for each token and
// page is most of the rest).
// Slots of pages that this call takes are worked out from the free list, not
// read back from the tables, so that workgroups need not wait for each other.
#include "launch.hpp"
#include "tile.hpp"

namespace ds {

constexpr int kPageThreads = 1024;
constexpr int kPageWaves = kPageThreads / kWave;

// A request's tokens and pages before it in its chunk of requests: sums of 1,024
// numbers below 2^31 may need 64 bits.
struct Before {
    int64_t tokens, pages;
};

__global__ __launch_bounds__(kPageThreads) void page_slots_kernel(PageSlots a)
{
    __shared__ Before s_first[kPageThreads], s_wave[kPageWaves];
    __shared__ uint32_t s_context[kPageThreads];
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int64_t top = min(max((int64_t)*a.count, (int64_t)0), a.capacity) - 1;
    const uint32_t page = (uint32_t)a.page;
    const auto free_page = [&](int64_t q) { return q <= top ? a.free_pages[top - q] : -1; };
    const auto pages_of = [&](uint32_t tokens) { return tokens / page + (tokens % page != 0); };
    // the last request i of the chunk's `here` with s_first[i].*what <= v
    const auto owner = [&](int64_t Before::*what, int here, int64_t v) {
        int lo = 0, hi = here;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_first[mid].*what <= v)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    int64_t tokens = 0, pages = 0;  // of the requests before the chunk
    for (int64_t base = 0; base < a.requests; base += kPageThreads) {
        const int64_t r = base + threadIdx.x;
        const int here = (int)min((int64_t)kPageThreads, a.requests - base);
        const uint32_t context = r < a.requests ? (uint32_t)max(a.context[r], 0) : 0u;
        const uint32_t fresh = r < a.requests ? (uint32_t)max(a.fresh[r], 0) : 0u;
        const uint32_t need = pages_of(context + fresh) - pages_of(context);
        const int64_t tokens_to = wave_inclusive_scan((int64_t)fresh), pages_to = wave_inclusive_scan((int64_t)need);
        if (lane == kWave - 1) s_wave[wave] = {tokens_to, pages_to};
        s_context[threadIdx.x] = context;
        __syncthreads();
        const int64_t first_token = tokens, first_page = pages;
        int64_t t0 = tokens_to - fresh, p0 = pages_to - need;
        for (int w = 0; w < kPageWaves; ++w) {
            const Before n = s_wave[w];
            t0 += w < wave ? n.tokens : 0;
            p0 += w < wave ? n.pages : 0;
            tokens += n.tokens;
            pages += n.pages;
        }
        t0 += first_token;
        p0 += first_page;
        s_first[threadIdx.x] = {t0, p0};
        if (blockIdx.x == 0 && r < a.requests) a.offsets[r] = (int32_t)min(t0, (int64_t)INT32_MAX);
        __syncthreads();
        // pages that the chunk's requests take, or where those are more than its tables have entries
        // (lengths of 2^31 would take minutes) the entries that they go to
        const int64_t entries = here * a.width;
        if (pages - first_page <= entries) {
            for (int64_t q = first_page + blockIdx.x * kPageThreads + threadIdx.x; q < pages;
                 q += (int64_t)gridDim.x * kPageThreads) {
                const int i = owner(&Before::pages, here, q);
                const int64_t col = pages_of(s_context[i]) + (q - s_first[i].pages);
                if (col < a.width) a.tables[(base + i) * a.table_stride + col] = free_page(q);
            }
        } else {
            for (int64_t c = (int64_t)blockIdx.x * kPageThreads + threadIdx.x; c < entries;
                 c += (int64_t)gridDim.x * kPageThreads) {
                const int i = (int)(c / a.width);
                const int64_t col = c % a.width, own = pages_of(s_context[i]), q = s_first[i].pages + (col - own);
                if (col >= own && q < (i + 1 < here ? s_first[i + 1].pages : pages))
                    a.tables[(base + i) * a.table_stride + col] = free_page(q);
            }
        }
        // their tokens
        const int64_t end = min(tokens, a.tokens);
        for (int64_t t = first_token + blockIdx.x * kPageThreads + threadIdx.x; t < end;
             t += (int64_t)gridDim.x * kPageThreads) {
            const int i = owner(&Before::tokens, here, t);
            const uint32_t position = s_context[i] + (uint32_t)(t - s_first[i].tokens);
            const uint32_t col = position / page, own = pages_of(s_context[i]);
            int32_t id = -1;
            if (col < a.width)
                id = col < own ? a.tables[(base + i) * a.table_stride + col] : free_page(s_first[i].pages + (col - own));
            a.slots[t] = id < 0 ? -1 : (int64_t)id * page + position % page;
            a.positions[t] = (int32_t)min(position, (uint32_t)INT32_MAX);
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
