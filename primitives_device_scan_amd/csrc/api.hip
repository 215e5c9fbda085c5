// api.hip -- the C ABI of include/devscan.h: argument validation on the host,
// the per-(device, stream) workspace, and dispatch to the kernel launchers.
#include <hip/hip_runtime.h>

#include <stdlib.h>

#include <initializer_list>
#include <map>
#include <mutex>
#include <set>
#include <utility>
#include <vector>

#include "devscan.h"
#include "launch.hpp"
#include "tile.hpp"

// Scratch of ds_scan_noalloc (see below); 256-byte aligned like a HIP allocation.
constexpr size_t kNoAllocScratchBytes = (size_t)4 << 20;
static __device__ __align__(256) char scratch[kNoAllocScratchBytes];

__global__ void noalloc_clear_kernel(uint64_t* p, int64_t words)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x)
        p[i] = 0;
}

namespace {

using ds::Ctrl;
using ds::DevWs;

// An earlier buffer of a workspace that graphs hold.
struct Retired {
    char* p;
    int64_t tiles;  // of a `base`; 0 for an `aux`
};

// Workspace layout: [Ctrl][status: one 128-byte line per tile][totals: 8 B per
// tile]; `aux` is a separate scratch buffer, for the counting-sort tables and
// for what ds_embedding_grad and ds_moe_experts keep between their launches.
struct Workspace {
    char* base = nullptr;
    int64_t tile_cap = 0;
    uint64_t lookback_launches = 0;  // launches that stamped an epoch since the last clear
    bool base_captured = false;   // some graph holds the address of base
    char* aux = nullptr;
    size_t aux_cap = 0;
    bool aux_captured = false;    // some graph holds the address of aux
    std::vector<Retired> retired; // freed by ds_release_workspace
};

std::mutex g_mu;
std::map<std::pair<int, hipStream_t>, Workspace> g_ws;
uint32_t g_spin_limit = 1u << 20;
int g_fail_allocs = -1;  // workspace allocations still to refuse (testing hook); -1: not read from the environment yet

constexpr uint32_t kDefaultSpin = 1u << 20;
// Epochs are 30 bits: clear the status words well before one comes round again.
constexpr uint64_t kEpochClearPeriod = 1ull << 29;
// Largest n: the grid (tiles x 256 work-items) must stay below 2^32 work-items.
constexpr int64_t kMaxTiles = ((int64_t)1 << 32) / ds::kThreads - 1;
constexpr size_t kStatusBytes = (size_t)ds::kStatusWords * sizeof(uint64_t);  // per tile

size_t ws_bytes(int64_t tiles) { return sizeof(Ctrl) + (size_t)tiles * (kStatusBytes + 8); }

DevWs view(const Workspace& w)
{
    DevWs d;
    d.ctrl = reinterpret_cast<Ctrl*>(w.base);
    d.status = reinterpret_cast<uint64_t*>(w.base + sizeof(Ctrl));
    d.totals = w.base + sizeof(Ctrl) + (size_t)w.tile_cap * kStatusBytes;
    return d;
}

// True when `stream` is being captured into a graph: the workspace may then
// be used but not allocated, grown or cleared (those are not kernel launches).
bool capturing(hipStream_t stream)
{
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &cs) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return cs != hipStreamCaptureStatusNone;
}

// Testing hook: DEVSCAN_FAIL_ALLOCS=k in the environment (read once) or
// ds_fail_next_allocations(k) makes the next k workspace allocations report
// DS_ERR_OUT_OF_MEMORY without calling hipMalloc.
bool refuse_allocation()
{
    if (g_fail_allocs < 0) {
        const char* s = getenv("DEVSCAN_FAIL_ALLOCS");
        g_fail_allocs = s ? atoi(s) : 0;
        if (g_fail_allocs < 0) g_fail_allocs = 0;
    }
    if (g_fail_allocs == 0) return false;
    --g_fail_allocs;
    return true;
}

// Returns the workspace of (current device, stream) with room for `tiles`;
// a new allocation is cleared on the stream before any kernel uses it.
int get_workspace(hipStream_t stream, int64_t tiles, Workspace** out)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_HIP;
    Workspace& w = g_ws[{dev, stream}];
    const bool grow = w.tile_cap < tiles;
    const bool clear = w.lookback_launches >= kEpochClearPeriod;
    const bool recording = capturing(stream);
    if ((grow || clear) && recording) return DS_ERR_STREAM_CAPTURING;
    if (grow) {
        int64_t cap = w.tile_cap * 2 > tiles ? w.tile_cap * 2 : tiles;
        if (cap < 1024) cap = 1024;
        if (refuse_allocation()) return DS_ERR_OUT_OF_MEMORY;
        if (w.base && w.base_captured) {
            w.retired.push_back({w.base, w.tile_cap});  // a replay may still use it
        } else if (w.base) {
            // The old buffer may still be in use by work queued on the stream.
            if (hipStreamSynchronize(stream) != hipSuccess) return DS_ERR_HIP;
            (void)hipFree(w.base);
        }
        w.base = nullptr;
        w.tile_cap = 0;
        w.base_captured = false;
        void* p = nullptr;
        if (hipMalloc(&p, ws_bytes(cap)) != hipSuccess) {
            (void)hipGetLastError();
            return DS_ERR_OUT_OF_MEMORY;
        }
        if (hipMemsetAsync(p, 0, ws_bytes(cap), stream) != hipSuccess) {
            (void)hipFree(p);
            return DS_ERR_HIP;
        }
        w.base = static_cast<char*>(p);
        w.tile_cap = cap;
        w.lookback_launches = 0;
    }
    if (w.lookback_launches >= kEpochClearPeriod) {
        if (hipMemsetAsync(w.base + sizeof(Ctrl), 0, (size_t)w.tile_cap * kStatusBytes, stream) != hipSuccess)
            return DS_ERR_HIP;
        w.lookback_launches = 0;
    }
    w.base_captured |= recording;
    *out = &w;
    return DS_OK;
}

// Scratch of at least `bytes` for (current device, stream); its contents are
// undefined (every user writes what it reads).
int get_aux(hipStream_t stream, size_t bytes, char** out)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_HIP;
    Workspace& w = g_ws[{dev, stream}];
    const bool recording = capturing(stream);
    if (w.aux_cap < bytes) {
        if (recording) return DS_ERR_STREAM_CAPTURING;
        size_t cap = w.aux_cap * 2 > bytes ? w.aux_cap * 2 : bytes;
        if (cap < ((size_t)1 << 20)) cap = (size_t)1 << 20;
        if (refuse_allocation()) return DS_ERR_OUT_OF_MEMORY;
        if (w.aux && w.aux_captured) {
            w.retired.push_back({w.aux, 0});  // a replay may still write to it
        } else if (w.aux) {
            if (hipStreamSynchronize(stream) != hipSuccess) return DS_ERR_HIP;
            (void)hipFree(w.aux);
        }
        w.aux = nullptr;
        w.aux_cap = 0;
        w.aux_captured = false;
        void* p = nullptr;
        if (hipMalloc(&p, cap) != hipSuccess) {
            (void)hipGetLastError();
            return DS_ERR_OUT_OF_MEMORY;
        }
        w.aux = static_cast<char*>(p);
        w.aux_cap = cap;
    }
    w.aux_captured |= recording;
    *out = w.aux;
    return DS_OK;
}

// ---------------------------------------------------------------------------
// The allocation-free look-back scan (ds_scan_noalloc): its control block and
// status words live in `scratch`, a fixed array in the library's own device
// memory, one copy per GPU, held until the process ends. Host code never
// passes `scratch` itself to a kernel (in host code the name is a host-side
// stand-in); it takes each device's address once with hipGetSymbolAddress and
// uses that.
// ---------------------------------------------------------------------------
constexpr int64_t kNoAllocMaxTiles = (int64_t)((kNoAllocScratchBytes - sizeof(Ctrl)) / kStatusBytes);

struct NoAllocDev {
    char* ptr = nullptr;           // device address of this GPU's `scratch`
    bool cleared = false;          // the clear kernel has been enqueued once
    uint64_t launches = 0;         // launches since the last clear (epoch wrap guard)
};
std::map<int, NoAllocDev> g_noalloc;  // per device, guarded by g_mu

// Devices on which a gated recurrence or its gradient has had tiles that wait.
std::set<int> g_gated;

bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na && nb && x < y + nb && y < x + na;
}

// The look-back workspace for an exclusive uint32 scan of `words` entries
// (none when it fits one tile).
int scan_workspace_u32(hipStream_t stream, int64_t words, DevWs* dws, Workspace** w)
{
    const int64_t te = ds::tile_elems(ds::kU32, false, words);
    const int64_t tiles = (words + te - 1) / te;
    *dws = DevWs{nullptr, nullptr, nullptr};
    *w = nullptr;
    if (tiles <= 1) return DS_OK;
    const int st = get_workspace(stream, tiles, w);
    if (st == DS_OK) *dws = view(**w);
    return st;
}

bool valid_dtype(int dtype) { return dtype >= DS_INT32 && dtype <= DS_UINT64; }

int elem_bytes(int dtype) { return (dtype == DS_INT64 || dtype == DS_UINT64) ? 8 : 4; }

ds::ElemKind kind_of(int dtype)
{
    switch (dtype) {
    case DS_INT32: return ds::kI32;
    case DS_UINT32: return ds::kU32;
    case DS_FP32: return ds::kF32;
    case DS_INT64: return ds::kI64;
    default: return ds::kU64;
    }
}

// Checks shared by every entry point that reads n elements and writes n.
int check_io(int dtype, const void* in, const void* out, int64_t n, bool allow_same)
{
    if (!valid_dtype(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (n < 0) return DS_ERR_INVALID_VALUE;
    if (n == 0) return DS_OK;
    if (!in || !out) return DS_ERR_INVALID_VALUE;
    const int64_t sz = elem_bytes(dtype);
    const int64_t smallest_tile = ds::lds_tile_elems();  // 4,096: the most tiles any entry point launches
    if ((n + smallest_tile - 1) / smallest_tile > kMaxTiles) return DS_ERR_TOO_LARGE;
    if (((uintptr_t)in % sz) || ((uintptr_t)out % sz)) return DS_ERR_MISALIGNED;
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out, len = (uintptr_t)(n * sz);
    if (a == b) return allow_same ? DS_OK : DS_ERR_OVERLAP;
    if (a < b + len && b < a + len) return DS_ERR_OVERLAP;
    return DS_OK;
}

// seed (look-back only): null, or one element of dtype in device memory added
// to every prefix.
int scan_impl(int dtype, int inclusive, int algo, const void* in, void* out, int64_t n, hipStream_t stream,
              const void* seed = nullptr)
{
    if (inclusive != 0 && inclusive != 1) return DS_ERR_INVALID_VALUE;
    if (algo < DS_ALGO_DEFAULT || algo > DS_ALGO_LOOKBACK_BLOCKED) return DS_ERR_INVALID_VALUE;
    int st = check_io(dtype, in, out, n, true);
    if (st != DS_OK || n == 0) return st;
    if (algo == DS_ALGO_LOOKBACK_BLOCKED) {
        if (elem_bytes(dtype) != 4) return DS_ERR_UNSUPPORTED_DTYPE;
        const int64_t bt = ds::blocked_tile_elems(n);
        const int64_t btiles = (n + bt - 1) / bt;
        std::lock_guard<std::mutex> lock(g_mu);
        DevWs dws{nullptr, nullptr, nullptr};
        Workspace* w = nullptr;
        if (btiles > 1) {
            st = get_workspace(stream, btiles, &w);
            if (st != DS_OK) return st;
            dws = view(*w);
        }
        const hipError_t e =
            ds::launch_lookback_blocked(kind_of(dtype), inclusive != 0, in, out, n, dws, g_spin_limit, stream);
        if (w && e == hipSuccess) ++w->lookback_launches;
        return e == hipSuccess ? DS_OK : DS_ERR_HIP;
    }
    // Choose the kernel first, then size the workspace by that kernel's own
    // tiles: the look-back and three-pass tiles differ in size, and a
    // three-pass call on one tile runs the look-back kernel instead.
    const int64_t tp = ds::three_pass_tile_elems(elem_bytes(dtype));
    const bool three = algo == DS_ALGO_THREE_PASS && n > tp;
    const int64_t te = three ? tp : ds::tile_elems(kind_of(dtype), inclusive != 0, n);
    const int64_t tiles = (n + te - 1) / te;
    std::lock_guard<std::mutex> lock(g_mu);
    DevWs dws{nullptr, nullptr, nullptr};
    Workspace* w = nullptr;
    if (tiles > 1) {
        st = get_workspace(stream, tiles, &w);
        if (st != DS_OK) return st;
        dws = view(*w);
    }
    hipError_t e;
    if (three) {
        e = ds::launch_three_pass_scan(kind_of(dtype), inclusive != 0, in, out, n, dws, stream);
    } else {
        e = ds::launch_lookback_scan(kind_of(dtype), inclusive != 0, in, out, n, dws, g_spin_limit, stream, seed);
        if (w && e == hipSuccess) ++w->lookback_launches;
    }
    return e == hipSuccess ? DS_OK : DS_ERR_HIP;
}

}  // namespace

extern "C" {

int scan_exclusive(int dtype, const void* d_in, void* d_out, int64_t n, hipStream_t stream)
{
    return scan_impl(dtype, 0, DS_ALGO_DEFAULT, d_in, d_out, n, stream);
}

int scan_inclusive(int dtype, const void* d_in, void* d_out, int64_t n, hipStream_t stream)
{
    return scan_impl(dtype, 1, DS_ALGO_DEFAULT, d_in, d_out, n, stream);
}

int ds_scan(int dtype, int inclusive, int algo, const void* d_in, void* d_out, int64_t n, hipStream_t stream)
{
    return scan_impl(dtype, inclusive, algo, d_in, d_out, n, stream);
}

int ds_scan_seeded(int dtype, int inclusive, const void* d_in, void* d_out, int64_t n, const void* d_seed,
                   hipStream_t stream)
{
    if (inclusive != 0 && inclusive != 1) return DS_ERR_INVALID_VALUE;
    const int st = check_io(dtype, d_in, d_out, n, true);  // the input and output first, as for every scan
    if (st != DS_OK || n == 0) return st;
    if (d_seed) {
        const int64_t sz = elem_bytes(dtype);
        if ((uintptr_t)d_seed % sz) return DS_ERR_MISALIGNED;
        if (overlaps(d_seed, (size_t)sz, d_out, (size_t)(n * sz))) return DS_ERR_OVERLAP;
    }
    return scan_impl(dtype, inclusive, DS_ALGO_LOOKBACK, d_in, d_out, n, stream, d_seed);
}

int ds_scan_noalloc(int dtype, int inclusive, const void* d_in, void* d_out, int64_t n, hipStream_t stream)
{
    if (inclusive != 0 && inclusive != 1) return DS_ERR_INVALID_VALUE;
    int st = check_io(dtype, d_in, d_out, n, true);
    if (st != DS_OK || n == 0) return st;
    const int64_t te = ds::tile_elems(kind_of(dtype), inclusive != 0, n);
    const int64_t tiles = (n + te - 1) / te;
    if (tiles > kNoAllocMaxTiles) return DS_ERR_TOO_LARGE;
    std::lock_guard<std::mutex> lock(g_mu);
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_HIP;
    NoAllocDev& d = g_noalloc[dev];
    if (!d.ptr) {
        // Once per device, with that device current: this GPU's copy of the array.
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) {
            (void)hipGetLastError();
            return DS_ERR_HIP;
        }
        d.ptr = static_cast<char*>(p);
    }
    DevWs dws{nullptr, nullptr, nullptr};
    if (tiles > 1) {
        if (!d.cleared || d.launches >= kEpochClearPeriod) {
            // Zero the control block and every status word (a kernel, so that
            // a captured call records no memset node); stream-ordered before
            // the scan below.
            const int64_t words = (int64_t)(kNoAllocScratchBytes / sizeof(uint64_t));
            noalloc_clear_kernel<<<dim3(256), dim3(256), 0, stream>>>(reinterpret_cast<uint64_t*>(d.ptr), words);
            if (hipGetLastError() != hipSuccess) return DS_ERR_HIP;
            d.cleared = true;
            d.launches = 0;
        }
        dws.ctrl = reinterpret_cast<Ctrl*>(d.ptr);
        dws.status = reinterpret_cast<uint64_t*>(d.ptr + sizeof(Ctrl));
    }
    const hipError_t e =
        ds::launch_lookback_scan(kind_of(dtype), inclusive != 0, d_in, d_out, n, dws, g_spin_limit, stream);
    if (e != hipSuccess) return DS_ERR_HIP;
    if (tiles > 1) ++d.launches;
    return DS_OK;
}

int compact_if(int dtype, const void* d_in, void* d_out, int64_t* d_num_selected, int64_t n, int cmp,
               uint64_t operand_bits, hipStream_t stream)
{
    if (!valid_dtype(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (cmp < DS_LT || cmp > DS_NE) return DS_ERR_INVALID_VALUE;
    if (!d_num_selected || n < 0) return DS_ERR_INVALID_VALUE;
    if (((uintptr_t)d_num_selected) % 8) return DS_ERR_MISALIGNED;
    if (n >= ((int64_t)1 << 32)) return DS_ERR_TOO_LARGE;
    int st = check_io(dtype, d_in, d_out, n, true);
    if (st != DS_OK) return st;
    if (n == 0)  // nothing to scan: the count is 0, written by a one-thread kernel (capturable)
        return ds::launch_write_count(d_num_selected, 0, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
    const int64_t ct = ds::compact_tile_elems(elem_bytes(dtype));
    const int64_t tiles = (n + ct - 1) / ct;
    std::lock_guard<std::mutex> lock(g_mu);
    DevWs dws{nullptr, nullptr, nullptr};
    Workspace* w = nullptr;
    if (tiles > 1) {
        st = get_workspace(stream, tiles, &w);
        if (st != DS_OK) return st;
        dws = view(*w);
    }
    const hipError_t e = ds::launch_compact(kind_of(dtype), d_in, d_out, d_num_selected, n, cmp, operand_bits, dws,
                                            g_spin_limit, stream);
    if (w && e == hipSuccess) ++w->lookback_launches;
    return e == hipSuccess ? DS_OK : DS_ERR_HIP;
}

int ds_compact_unordered(int dtype, const void* d_in, void* d_out, int64_t* d_num_selected, int64_t n, int cmp,
                         uint64_t operand_bits, int claim, hipStream_t stream)
{
    if (!valid_dtype(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (cmp < DS_LT || cmp > DS_NE) return DS_ERR_INVALID_VALUE;
    if (claim != DS_CLAIM_PER_WAVE && claim != DS_CLAIM_PER_WORKGROUP) return DS_ERR_INVALID_VALUE;
    if (!d_num_selected || n < 0) return DS_ERR_INVALID_VALUE;
    if (((uintptr_t)d_num_selected) % 8) return DS_ERR_MISALIGNED;
    if (n >= ((int64_t)1 << 32)) return DS_ERR_TOO_LARGE;
    int st = check_io(dtype, d_in, d_out, n, false);  // out is written in any order: never in place
    if (st != DS_OK) return st;
    if (n == 0)  // nothing to scan: the count is 0, written by a one-thread kernel (capturable)
        return ds::launch_write_count(d_num_selected, 0, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
    return ds::launch_compact_unordered(kind_of(dtype), d_in, d_out, d_num_selected, n, cmp, operand_bits,
                                        claim == DS_CLAIM_PER_WORKGROUP, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_copy(const void* d_in, void* d_out, int64_t nbytes, hipStream_t stream)
{
    if (nbytes < 0 || (nbytes % 16)) return DS_ERR_INVALID_VALUE;
    if (nbytes == 0) return DS_OK;
    if (!d_in || !d_out) return DS_ERR_INVALID_VALUE;
    if (((uintptr_t)d_in % 16) || ((uintptr_t)d_out % 16)) return DS_ERR_MISALIGNED;
    const uintptr_t a = (uintptr_t)d_in, b = (uintptr_t)d_out, len = (uintptr_t)nbytes;
    if (a < b + len && b < a + len) return DS_ERR_OVERLAP;
    if (nbytes / ds::tile_bytes() >= kMaxTiles) return DS_ERR_TOO_LARGE;
    return ds::launch_copy(d_in, d_out, nbytes, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
}

int ds_bandwidth_pattern(int mode, int vectors_per_thread, int layout, const void* d_in, void* d_out, int64_t nbytes,
                         hipStream_t stream)
{
    if (mode < 0 || mode > 5 || layout < 0 || layout > 1 || !ds::pattern_vpt_ok(vectors_per_thread))
        return DS_ERR_INVALID_VALUE;
    if (nbytes < 0 || (nbytes % 16)) return DS_ERR_INVALID_VALUE;
    if (nbytes == 0) return DS_OK;
    if (!d_out || (mode != 1 && !d_in)) return DS_ERR_INVALID_VALUE;
    if (((uintptr_t)d_in % 16) || ((uintptr_t)d_out % 16)) return DS_ERR_MISALIGNED;
    if (mode != 1) {
        const uintptr_t a = (uintptr_t)d_in, b = (uintptr_t)d_out, len = (uintptr_t)nbytes;
        if (a < b + len && b < a + len) return DS_ERR_OVERLAP;
    }
    if (nbytes / 4096 + 8 >= kMaxTiles) return DS_ERR_TOO_LARGE;
    return ds::launch_pattern(mode, vectors_per_thread, layout, d_in, d_out, nbytes, stream) == hipSuccess ? DS_OK
                                                                                                        : DS_ERR_HIP;
}

static int check_tile_args(int dtype, int variant, const void* in, void* out, int64_t n)
{
    if (!valid_dtype(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (elem_bytes(dtype) != 4) return DS_ERR_UNSUPPORTED_DTYPE;
    if (variant < DS_TILE_TREE || variant > DS_TILE_HS) return DS_ERR_INVALID_VALUE;
    if (n >= ((int64_t)1 << 32)) return DS_ERR_TOO_LARGE;
    return check_io(dtype, in, out, n, true);
}

int ds_tile_scan(int dtype, int variant, const void* d_in, void* d_out, void* d_tile_sums, int64_t n,
                 hipStream_t stream)
{
    int st = check_tile_args(dtype, variant, d_in, d_out, n);
    if (st != DS_OK || n == 0) return st;
    if (((uintptr_t)d_tile_sums) % 4) return DS_ERR_MISALIGNED;
    return ds::launch_tile_scan(kind_of(dtype), variant, d_in, d_out, d_tile_sums, n, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_tile_pipeline(int dtype, int variant, const void* d_in, void* d_out, int64_t n, hipStream_t stream)
{
    int st = check_tile_args(dtype, variant, d_in, d_out, n);
    if (st != DS_OK || n == 0) return st;
    const int64_t tiles = (n + ds::lds_tile_elems() - 1) / ds::lds_tile_elems();
    std::lock_guard<std::mutex> lock(g_mu);
    Workspace* w = nullptr;
    st = get_workspace(stream, tiles, &w);
    if (st != DS_OK) return st;
    return ds::launch_tile_pipeline(kind_of(dtype), variant, d_in, d_out, n, view(*w), stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

// Whether a wait on this look-back workspace has given up (sets *gave_up if so).
static int take_timeout(char* base, int64_t tiles, bool* gave_up)
{
    Ctrl* c = reinterpret_cast<Ctrl*>(base);
    uint32_t flag = 0;
    if (hipMemcpy(&flag, &c->timeout, sizeof(flag), hipMemcpyDeviceToHost) != hipSuccess) return DS_ERR_HIP;
    if (!flag) return DS_OK;
    // A wait that gave up may have let the last tile advance the epoch
    // before slower tiles read it, so their status words can carry the
    // next launch's epoch. The stream is idle: clear every status word
    // (and the flag) so the next launch starts from a clean array.
    if (hipMemset(base + sizeof(Ctrl), 0, (size_t)tiles * kStatusBytes) != hipSuccess) return DS_ERR_HIP;
    const uint32_t zero = 0;
    if (hipMemcpy(&c->timeout, &zero, sizeof(zero), hipMemcpyHostToDevice) != hipSuccess) return DS_ERR_HIP;
    *gave_up = true;
    return DS_OK;
}

int ds_query_timeout(hipStream_t stream, int* timed_out)
{
    if (!timed_out) return DS_ERR_INVALID_VALUE;
    *timed_out = 0;
    if (hipStreamSynchronize(stream) != hipSuccess) return DS_ERR_HIP;
    std::lock_guard<std::mutex> lock(g_mu);
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_HIP;
    int from_scratch = 0;
    auto na = g_noalloc.find(dev);
    if (na != g_noalloc.end() && na->second.ptr && na->second.cleared) {
        // ds_scan_noalloc's flag: the same rule, on the device's scratch array
        Ctrl* c = reinterpret_cast<Ctrl*>(na->second.ptr);
        uint32_t flag = 0;
        if (hipMemcpy(&flag, &c->timeout, sizeof(flag), hipMemcpyDeviceToHost) != hipSuccess) return DS_ERR_HIP;
        if (flag) {
            na->second.cleared = false;  // the next ds_scan_noalloc clears every word first
            from_scratch = 1;
        }
    }
    bool gave_up = false;
    if (g_gated.count(dev) && (ds::take_gated_scan_give_up(&gave_up) != hipSuccess ||
                               ds::take_gated_scan_grad_give_up(&gave_up) != hipSuccess))
        return DS_ERR_HIP;
    auto it = g_ws.find({dev, stream});
    if (it != g_ws.end()) {
        Workspace& w = it->second;
        if (w.base) {
            const int st = take_timeout(w.base, w.tile_cap, &gave_up);
            if (st != DS_OK) return st;
            if (gave_up) w.lookback_launches = 0;
        }
        for (const Retired& r : w.retired) {  // graphs may still run on these
            const int st = r.tiles ? take_timeout(r.p, r.tiles, &gave_up) : DS_OK;
            if (st != DS_OK) return st;
        }
    }
    *timed_out = (gave_up || from_scratch) ? 1 : 0;
    return DS_OK;
}

int ds_fail_next_allocations(int count)
{
    if (count < 0) return DS_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lock(g_mu);
    g_fail_allocs = count;
    return DS_OK;
}

int ds_set_spin_limit(uint32_t polls)
{
    std::lock_guard<std::mutex> lock(g_mu);
    g_spin_limit = polls ? polls : kDefaultSpin;
    return DS_OK;
}

const char* ds_status_string(int status)
{
    switch (status) {
    case DS_OK: return "DS_OK";
    case DS_ERR_INVALID_VALUE: return "DS_ERR_INVALID_VALUE: bad argument (n < 0, null pointer, bad enum)";
    case DS_ERR_UNSUPPORTED_DTYPE: return "DS_ERR_UNSUPPORTED_DTYPE";
    case DS_ERR_OVERLAP: return "DS_ERR_OVERLAP: input and output partially overlap";
    case DS_ERR_OUT_OF_MEMORY: return "DS_ERR_OUT_OF_MEMORY: workspace allocation failed";
    case DS_ERR_HIP: return "DS_ERR_HIP: a HIP call or kernel launch failed";
    case DS_ERR_MISALIGNED: return "DS_ERR_MISALIGNED: pointer not aligned to the element size";
    case DS_ERR_TOO_LARGE: return "DS_ERR_TOO_LARGE: n beyond the entry point's limit";
    case DS_ERR_STREAM_CAPTURING:
        return "DS_ERR_STREAM_CAPTURING: the workspace would have to be allocated, grown or cleared while the "
               "stream is being captured (make one call on the stream before capturing)";
    default: return "unknown ds_status";
    }
}

int ds_radix_pass(const uint32_t* d_keys_in, uint32_t* d_keys_out, const uint32_t* d_vals_in, uint32_t* d_vals_out,
                  int64_t n, int shift, int bits, hipStream_t stream)
{
    if (n < 0 || bits < 1 || bits > 8 || shift < 0 || shift > 31 || shift + bits > 32) return DS_ERR_INVALID_VALUE;
    if ((d_vals_in == nullptr) != (d_vals_out == nullptr)) return DS_ERR_INVALID_VALUE;
    if (n == 0) return DS_OK;
    if (n >= ((int64_t)1 << 32)) return DS_ERR_TOO_LARGE;
    if (!d_keys_in || !d_keys_out) return DS_ERR_INVALID_VALUE;
    const void* ptrs[4] = {d_keys_in, d_keys_out, d_vals_in, d_vals_out};
    for (const void* p : ptrs)
        if ((uintptr_t)p % 4) return DS_ERR_MISALIGNED;
    const size_t bytes = (size_t)n * 4;
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j) {
            if (i == 0 && j == 2) continue;  // the two inputs may share memory: both are only read
            if (ptrs[i] && ptrs[j] && overlaps(ptrs[i], bytes, ptrs[j], bytes)) return DS_ERR_OVERLAP;
        }
    const int64_t words = ((int64_t)1 << bits) * ds::sort_table_columns(d_vals_in != nullptr, n);
    std::lock_guard<std::mutex> lock(g_mu);
    char* aux = nullptr;
    int st = get_aux(stream, (size_t)ds::sort_aux_words(d_vals_in != nullptr, n, bits) * 4, &aux);
    if (st != DS_OK) return st;
    DevWs dws;
    Workspace* w = nullptr;
    st = scan_workspace_u32(stream, words, &dws, &w);
    if (st != DS_OK) return st;
    const hipError_t e = ds::launch_radix_pass(d_keys_in, d_vals_in, d_keys_out, d_vals_out, n, shift, bits,
                                               reinterpret_cast<uint32_t*>(aux), dws, g_spin_limit, stream);
    if (w && e == hipSuccess) ++w->lookback_launches;
    return e == hipSuccess ? DS_OK : DS_ERR_HIP;
}

int ds_moe_align(const int32_t* d_topk_ids, int64_t n, int num_experts, int block, int32_t* d_counts,
                 int32_t* d_offsets, int32_t* d_sorted_ids, int64_t capacity, hipStream_t stream)
{
    if (n < 0 || block < 1 || num_experts < 1 || num_experts > ds::sort_max_buckets()) return DS_ERR_INVALID_VALUE;
    if (!d_counts || !d_offsets || !d_sorted_ids || (n > 0 && !d_topk_ids)) return DS_ERR_INVALID_VALUE;
    const int64_t worst = n + (int64_t)num_experts * (block - 1);
    if (worst >= ((int64_t)1 << 31)) return DS_ERR_TOO_LARGE;
    if (capacity < worst) return DS_ERR_INVALID_VALUE;
    const void* ptrs[4] = {d_topk_ids, d_counts, d_offsets, d_sorted_ids};
    const size_t sizes[4] = {(size_t)n * 4, (size_t)num_experts * 4, (size_t)(num_experts + 1) * 4,
                             (size_t)capacity * 4};
    for (int i = 0; i < 4; ++i) {
        if ((uintptr_t)ptrs[i] % 4) return DS_ERR_MISALIGNED;
        for (int j = i + 1; j < 4; ++j)
            if (ptrs[i] && ptrs[j] && overlaps(ptrs[i], sizes[i], ptrs[j], sizes[j])) return DS_ERR_OVERLAP;
    }
    const int64_t tiles = (n + ds::moe_tile_elems() - 1) / ds::moe_tile_elems();
    const int64_t words = (int64_t)num_experts * tiles;
    std::lock_guard<std::mutex> lock(g_mu);
    char* aux = nullptr;
    int st = get_aux(stream, (size_t)(2 * words + 1) * 4, &aux);
    if (st != DS_OK) return st;
    DevWs dws;
    Workspace* w = nullptr;
    st = scan_workspace_u32(stream, words, &dws, &w);
    if (st != DS_OK) return st;
    uint32_t* hist = reinterpret_cast<uint32_t*>(aux);
    uint32_t* slots = hist + words;
    const ds::MoeOut out{d_counts, d_offsets, d_sorted_ids, block, capacity};
    const hipError_t e = ds::launch_moe_align(d_topk_ids, n, num_experts, out, hist, slots, dws, g_spin_limit,
                                              stream);
    if (w && e == hipSuccess && n > 0) ++w->lookback_launches;
    return e == hipSuccess ? DS_OK : DS_ERR_HIP;
}

// Language-model operators. Their matrices are rows of contiguous elements,
// `stride` elements apart.
static int float_bytes(int dtype) { return dtype == DS_FP32 ? 4 : dtype == DS_BF16 || dtype == DS_FP16 ? 2 : 0; }

static ds::ElemKind float_kind(int dtype)
{
    return dtype == DS_FP32 ? ds::kF32 : dtype == DS_BF16 ? ds::kBF16 : ds::kF16;
}

// Bytes from the first to the last element of a matrix; -1 past what a pointer can address.
static int64_t span_bytes(int64_t rows, int64_t cols, int64_t stride, int esz)
{
    if (rows <= 0 || cols <= 0) return 0;
    const __int128 b = ((__int128)(rows - 1) * stride + cols) * esz;
    return b > ((__int128)1 << 56) ? -1 : (int64_t)b;
}

struct Buf {
    const void* p;
    int64_t bytes;  // 0: not used
    int align;
    bool written;
};

// Every buffer in use is there, aligned, and no written one overlaps another.
static int check_buffers(const Buf* b, int count)
{
    for (int i = 0; i < count; ++i) {
        if (b[i].bytes < 0) return DS_ERR_TOO_LARGE;
        if (b[i].bytes && !b[i].p) return DS_ERR_INVALID_VALUE;
    }
    for (int i = 0; i < count; ++i)
        if (b[i].bytes && (uintptr_t)b[i].p % b[i].align) return DS_ERR_MISALIGNED;
    for (int i = 0; i < count; ++i)
        for (int j = i + 1; j < count; ++j)
            if ((b[i].written || b[j].written) && overlaps(b[i].p, (size_t)b[i].bytes, b[j].p, (size_t)b[j].bytes))
                return DS_ERR_OVERLAP;
    return DS_OK;
}

int ds_embedding(int dtype, const void* d_table, int64_t rows, int64_t dim, int64_t table_stride, const void* d_ids,
                 int id_bytes, int64_t n, float scale, void* d_out, int64_t out_stride, hipStream_t stream)
{
    const int esz = float_bytes(dtype);
    if (!esz) return DS_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || dim < 0 || n < 0 || table_stride < dim || out_stride < dim || (id_bytes != 4 && id_bytes != 8))
        return DS_ERR_INVALID_VALUE;
    if (n == 0 || dim == 0) return DS_OK;
    if (n >= ((int64_t)1 << 40) || dim >= ((int64_t)1 << 40)) return DS_ERR_TOO_LARGE;
    const Buf bufs[3] = {{d_table, span_bytes(rows, dim, table_stride, esz), esz, false},
                         {d_ids, n * id_bytes, id_bytes, false},
                         {d_out, span_bytes(n, dim, out_stride, esz), esz, true}};
    const int st = check_buffers(bufs, 3);
    if (st != DS_OK) return st;
    if (ds::embedding_blocks(float_kind(dtype), n, dim) > kMaxTiles) return DS_ERR_TOO_LARGE;
    return ds::launch_embedding(float_kind(dtype), d_table, rows, dim, table_stride, d_ids, id_bytes == 8, n, scale,
                                d_out, out_stride, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

// The scratch of a call: the caller's, checked against the call's buffers too, or the stream's own.
static int check_scratch(const void* scratch, int64_t have, int64_t need, const Buf* bufs, int count)
{
    if (have < 0 || (scratch && have < need)) return DS_ERR_INVALID_VALUE;
    if ((uintptr_t)scratch % 256) return DS_ERR_MISALIGNED;
    for (int i = 0; scratch && i < count; ++i)
        if (overlaps(scratch, (size_t)need, bufs[i].p, (size_t)bufs[i].bytes)) return DS_ERR_OVERLAP;
    return DS_OK;
}

int ds_embedding_grad(int dtype, const void* d_dout, int64_t dout_stride, const void* d_ids, int id_bytes, int64_t n,
                      float scale, int grad_dtype, void* d_grad, int64_t rows, int64_t dim, int64_t grad_stride,
                      int accumulate, hipStream_t stream)
{
    return ds_embedding_grad_scratch(dtype, d_dout, dout_stride, d_ids, id_bytes, n, scale, grad_dtype, d_grad, rows,
                                     dim, grad_stride, accumulate, nullptr, 0, stream);
}

int64_t ds_embedding_grad_scratch_bytes(int grad_dtype, int64_t n, int64_t rows, int64_t dim)
{
    if (!float_bytes(grad_dtype) || rows < 1 || dim < 1 || n < 1) return 0;
    if (n >= ((int64_t)1 << 31) || dim >= ((int64_t)1 << 31) || rows > ds::embedding_most_rows()) return 0;
    return ds::embedding_grad_plan(float_kind(grad_dtype), n, rows, dim).bytes;
}

int ds_embedding_grad_scratch(int dtype, const void* d_dout, int64_t dout_stride, const void* d_ids, int id_bytes,
                              int64_t n, float scale, int grad_dtype, void* d_grad, int64_t rows, int64_t dim,
                              int64_t grad_stride, int accumulate, void* d_scratch, int64_t scratch_bytes,
                              hipStream_t stream)
{
    const int esz = float_bytes(dtype), gsz = float_bytes(grad_dtype);
    if (!esz || !gsz || (grad_dtype != dtype && grad_dtype != DS_FP32)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || dim < 0 || n < 0 || dout_stride < dim || grad_stride < dim || (id_bytes != 4 && id_bytes != 8) ||
        (accumulate != 0 && accumulate != 1))
        return DS_ERR_INVALID_VALUE;
    if (rows == 0 || dim == 0 || (n == 0 && accumulate)) return DS_OK;
    if (n >= ((int64_t)1 << 31) || dim >= ((int64_t)1 << 31) || rows > ds::embedding_most_rows())
        return DS_ERR_TOO_LARGE;
    const Buf bufs[3] = {{d_dout, span_bytes(n, dim, dout_stride, esz), esz, false},
                         {d_ids, n * id_bytes, id_bytes, false},
                         {d_grad, span_bytes(rows, dim, grad_stride, gsz), gsz, true}};
    int st = check_buffers(bufs, 3);
    if (st != DS_OK) return st;
    const ds::EmbeddingGradPlan plan = ds::embedding_grad_plan(float_kind(grad_dtype), n, rows, dim);
    if (ds::embedding_grad_blocks(plan, n, rows, dim * gsz) > kMaxTiles / 2) return DS_ERR_TOO_LARGE;
    st = check_scratch(d_scratch, scratch_bytes, plan.bytes, bufs, 3);
    if (st != DS_OK) return st;
    std::lock_guard<std::mutex> lock(g_mu);
    char* aux = static_cast<char*>(d_scratch);
    if (plan.bytes && !aux) {
        st = get_aux(stream, (size_t)plan.bytes, &aux);
        if (st != DS_OK) return st;
    }
    return ds::launch_embedding_grad(float_kind(dtype), float_kind(grad_dtype), plan, d_dout, dout_stride, d_ids,
                                     id_bytes == 8, n, rows, dim, scale, d_grad, grad_stride, accumulate != 0, aux,
                                     stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

static int check_route(int dtype, int64_t tokens, int num_experts, int64_t stride, int top_k, int score,
                       int renormalize)
{
    if (!float_bytes(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (tokens < 0 || num_experts < 1 || num_experts > ds::route_max_experts() || stride < num_experts || top_k < 1 ||
        top_k > num_experts || top_k > DS_ROUTE_MAX_TOP_K || score < DS_SCORE_SOFTMAX || score > DS_SCORE_SIGMOID ||
        (renormalize != 0 && renormalize != 1))
        return DS_ERR_INVALID_VALUE;
    return ds::route_blocks(tokens) > kMaxTiles ? DS_ERR_TOO_LARGE : DS_OK;
}

int ds_moe_route(int dtype, const void* d_logits, int64_t tokens, int num_experts, int64_t stride,
                 const float* d_bias, int top_k, int score, int renormalize, float scale, float* d_weights,
                 int32_t* d_ids, hipStream_t stream)
{
    int st = check_route(dtype, tokens, num_experts, stride, top_k, score, renormalize);
    if (st != DS_OK || tokens == 0) return st;
    const int esz = float_bytes(dtype);
    const Buf bufs[4] = {{d_logits, span_bytes(tokens, num_experts, stride, esz), esz, false},
                         {d_bias, d_bias ? (int64_t)num_experts * 4 : 0, 4, false},
                         {d_weights, tokens * top_k * 4, 4, true},
                         {d_ids, tokens * top_k * 4, 4, true}};
    st = check_buffers(bufs, 4);
    if (st != DS_OK) return st;
    const ds::RouteArgs a{tokens, stride, num_experts, top_k, score == DS_SCORE_SIGMOID, renormalize != 0, scale};
    return ds::launch_moe_route(float_kind(dtype), a, d_logits, d_bias, d_weights, d_ids, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_moe_route_grad(int dtype, const void* d_logits, int64_t tokens, int num_experts, int64_t stride,
                      const int32_t* d_ids, const float* d_dweights, int top_k, int score, int renormalize,
                      float scale, void* d_dlogits, int64_t dlogits_stride, hipStream_t stream)
{
    return ds_moe_route_grad_biased(dtype, d_logits, tokens, num_experts, stride, nullptr, d_ids, d_dweights, top_k,
                                    score, renormalize, scale, d_dlogits, dlogits_stride, stream);
}

int ds_moe_route_grad_biased(int dtype, const void* d_logits, int64_t tokens, int num_experts, int64_t stride,
                             const float* d_bias, const int32_t* d_ids, const float* d_dweights, int top_k, int score,
                             int renormalize, float scale, void* d_dlogits, int64_t dlogits_stride, hipStream_t stream)
{
    int st = check_route(dtype, tokens, num_experts, stride, top_k, score, renormalize);
    if (st == DS_OK && dlogits_stride < num_experts) st = DS_ERR_INVALID_VALUE;
    if (st != DS_OK || tokens == 0) return st;
    const int esz = float_bytes(dtype);
    const Buf bufs[5] = {{d_logits, span_bytes(tokens, num_experts, stride, esz), esz, false},
                         {d_bias, d_bias ? (int64_t)num_experts * 4 : 0, 4, false},
                         {d_ids, tokens * top_k * 4, 4, false},
                         {d_dweights, tokens * top_k * 4, 4, false},
                         {d_dlogits, span_bytes(tokens, num_experts, dlogits_stride, esz), esz, true}};
    st = check_buffers(bufs, 5);
    if (st != DS_OK) return st;
    const ds::RouteArgs a{tokens, stride, num_experts, top_k, score == DS_SCORE_SIGMOID, renormalize != 0, scale};
    return ds::launch_moe_route_grad(float_kind(dtype), a, d_logits, d_bias, d_ids, d_dweights, d_dlogits,
                                     dlogits_stride, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_moe_experts(int dtype, const void* d_x, int64_t tokens, int64_t dim, int64_t x_stride, int weight_dtype,
                   const void* d_w_in, const float* d_w_in_scale, const void* d_w_out, const float* d_w_out_scale,
                   int num_experts, int64_t hidden, const int32_t* d_ids, const float* d_weights, int top_k,
                   void* d_y, int64_t y_stride, hipStream_t stream)
{
    return ds_moe_experts_scratch(dtype, d_x, tokens, dim, x_stride, weight_dtype, d_w_in, d_w_in_scale, d_w_out,
                                  d_w_out_scale, num_experts, hidden, d_ids, d_weights, top_k, d_y, y_stride, nullptr,
                                  0, stream);
}

int64_t ds_moe_experts_scratch_bytes(int weight_dtype, int64_t tokens, int64_t dim, int num_experts, int64_t hidden,
                                     int top_k)
{
    if (tokens < 1 || dim < 1 || hidden < 1 || num_experts < 1 || num_experts > ds::experts_max_experts() ||
        top_k < 1 || dim > DS_EXPERTS_MAX_WIDTH || hidden > DS_EXPERTS_MAX_WIDTH ||
        tokens > ds::experts_max_assignments() || tokens * top_k > ds::experts_max_assignments())
        return 0;
    // weights at any address: whichever launch that leads to
    return ds::experts_most_aux_bytes(weight_dtype == DS_FP8_E4M3, tokens, (int)dim, num_experts, (int)hidden, top_k);
}

int ds_moe_experts_scratch(int dtype, const void* d_x, int64_t tokens, int64_t dim, int64_t x_stride, int weight_dtype,
                           const void* d_w_in, const float* d_w_in_scale, const void* d_w_out,
                           const float* d_w_out_scale, int num_experts, int64_t hidden, const int32_t* d_ids,
                           const float* d_weights, int top_k, void* d_y, int64_t y_stride, void* d_scratch,
                           int64_t scratch_bytes, hipStream_t stream)
{
    if (dtype != DS_BF16 && dtype != DS_FP16) return DS_ERR_UNSUPPORTED_DTYPE;
    const bool eight = weight_dtype == DS_FP8_E4M3;
    if (weight_dtype != dtype && !eight) return DS_ERR_UNSUPPORTED_DTYPE;
    if (tokens < 0 || dim < 1 || hidden < 1 || num_experts < 1 || num_experts > ds::experts_max_experts() ||
        top_k < 1 || x_stride < dim || y_stride < dim)
        return DS_ERR_INVALID_VALUE;
    if (tokens == 0) return DS_OK;
    if (dim > DS_EXPERTS_MAX_WIDTH || hidden > DS_EXPERTS_MAX_WIDTH || tokens > ds::experts_max_assignments() ||
        tokens * top_k > ds::experts_max_assignments())
        return DS_ERR_TOO_LARGE;
    const int64_t n = tokens * top_k, E = num_experts, wsz = eight ? 1 : 2;
    const auto blocks = [](int64_t v) { return (v + 127) / 128; };
    const Buf bufs[8] = {
        {d_x, span_bytes(tokens, dim, x_stride, 2), 2, false},
        {d_w_in, E * 2 * hidden * dim * wsz, (int)wsz, false},
        {d_w_out, E * hidden * dim * wsz, (int)wsz, false},
        {d_w_in_scale, eight ? E * blocks(2 * hidden) * blocks(dim) * 4 : 0, 4, false},
        {d_w_out_scale, eight ? E * blocks(dim) * blocks(hidden) * 4 : 0, 4, false},
        {d_ids, n * 4, 4, false},
        {d_weights, n * 4, 4, false},
        {d_y, span_bytes(tokens, dim, y_stride, 2), 2, true}};
    int st = check_buffers(bufs, 8);
    if (st != DS_OK) return st;
    const ds::ExpertsCall call{tokens, (int)dim, (int)hidden, num_experts, top_k, d_x, x_stride, d_w_in, d_w_out,
                               d_w_in_scale, d_w_out_scale, d_ids, d_weights, d_y, y_stride};
    if (ds::experts_workgroups(eight, call) > kMaxTiles) return DS_ERR_TOO_LARGE;
    const int64_t need = ds::experts_aux_bytes(eight, call);
    st = check_scratch(d_scratch, scratch_bytes, need, bufs, 8);
    if (st != DS_OK) return st;
    std::lock_guard<std::mutex> lock(g_mu);
    char* aux = static_cast<char*>(d_scratch);
    if (!aux) st = get_aux(stream, (size_t)need, &aux);
    if (st != DS_OK) return st;
    return ds::launch_moe_experts(float_kind(dtype), eight, call, aux, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
}

// Operators on ragged batches.
static constexpr int64_t kMost31 = ((int64_t)1 << 31) - 1;

static int check_gated(int dtype, int64_t tokens, int64_t dim, const int32_t* offsets, int64_t sequences, int form,
                       int mix)
{
    if (!float_bytes(dtype)) return DS_ERR_UNSUPPORTED_DTYPE;
    if (tokens < 0 || dim < 0 || sequences < 0 || form < DS_GATE_DECAY || form > DS_GATE_SIGMOID ||
        (mix != 0 && mix != 1) || (!offsets && sequences != 1))
        return DS_ERR_INVALID_VALUE;
    return tokens > kMost31 || sequences > kMost31 ? DS_ERR_TOO_LARGE : DS_OK;
}

// Distances between rows that the recurrence's 32-bit offsets within a tile can take.
static int check_gated_strides(std::initializer_list<int64_t> strides, int64_t dim)
{
    for (const int64_t s : strides)
        if (s < dim) return DS_ERR_INVALID_VALUE;
    for (const int64_t s : strides)
        if (s > DS_GATED_MAX_STRIDE) return DS_ERR_TOO_LARGE;
    return DS_OK;
}

static int64_t gated_scratch(const ds::GatedPlan& plan) { return (plan.words * 8 + 15) / 16 * 16; }

int64_t ds_gated_scan_scratch_bytes(int dtype, int grad, int64_t tokens, int64_t dim)
{
    if (!float_bytes(dtype) || tokens < 1 || dim < 1 || tokens > kMost31 || dim > DS_GATED_MAX_STRIDE) return 0;
    // of either kind of input
    const int64_t plain = gated_scratch(ds::gated_plan(float_kind(dtype), grad != 0, false, tokens, dim));
    const int64_t mixed = gated_scratch(ds::gated_plan(float_kind(dtype), grad != 0, true, tokens, dim));
    return plain > mixed ? plain : mixed;
}

// The words of a scan or its gradient, in the call's scratch.
static int gated_words(const ds::GatedPlan& plan, int64_t need, void* d_scratch, int64_t scratch_bytes,
                       const Buf* bufs, int count, hipStream_t stream, uint64_t** words)
{
    if (plan.tiles * plan.cblocks > kMaxTiles) return DS_ERR_TOO_LARGE;
    int st = check_scratch(d_scratch, scratch_bytes, need, bufs, count);
    if (st != DS_OK) return st;
    char* aux = static_cast<char*>(d_scratch);
    if (need && !aux) st = get_aux(stream, (size_t)need, &aux);
    *words = reinterpret_cast<uint64_t*>(aux);
    if (plan.tiles > 1 && st == DS_OK) {
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_HIP;
        g_gated.insert(dev);  // ds_query_timeout asks there
    }
    return st;
}

int ds_gated_scan(int dtype, const void* d_gate, int64_t gate_stride, const void* d_x, int64_t x_stride,
                  int64_t tokens, int64_t dim, const int32_t* d_offsets, int64_t sequences, int form, int mix,
                  const float* d_initial, void* d_h, int64_t h_stride, float* d_final, void* d_scratch,
                  int64_t scratch_bytes, hipStream_t stream)
{
    int st = check_gated(dtype, tokens, dim, d_offsets, sequences, form, mix);
    if (st == DS_OK) st = check_gated_strides({gate_stride, x_stride, h_stride}, dim);
    if (st != DS_OK || dim == 0 || sequences == 0) return st;
    const int esz = float_bytes(dtype);
    const int64_t states = span_bytes(sequences, dim, dim, 4);
    const Buf bufs[6] = {{d_gate, span_bytes(tokens, dim, gate_stride, esz), esz, false},
                         {d_x, span_bytes(tokens, dim, x_stride, esz), esz, false},
                         {d_offsets, d_offsets ? (sequences + 1) * 4 : 0, 4, false},
                         {d_initial, d_initial ? states : 0, 4, false},
                         {d_h, span_bytes(tokens, dim, h_stride, esz), esz, true},
                         {d_final, d_final ? states : 0, 4, true}};
    st = check_buffers(bufs, 6);
    if (st != DS_OK) return st;
    const ds::GatedScan a{d_gate, d_x, d_h, gate_stride, x_stride, h_stride, tokens, dim, d_offsets, sequences, form,
                          mix != 0, d_initial, d_final};
    const ds::GatedPlan plan = ds::gated_plan(float_kind(dtype), false, mix != 0, tokens, dim);
    std::lock_guard<std::mutex> lock(g_mu);
    uint64_t* words = nullptr;
    st = gated_words(plan, ds_gated_scan_scratch_bytes(dtype, 0, tokens, dim), d_scratch, scratch_bytes, bufs, 6, stream,
                     &words);
    if (st != DS_OK) return st;
    return ds::launch_gated_scan(float_kind(dtype), a, plan, words, g_spin_limit, stream) == hipSuccess ? DS_OK
                                                                                                        : DS_ERR_HIP;
}

int ds_gated_scan_grad(int dtype, const void* d_gate, int64_t gate_stride, const void* d_h, int64_t h_stride,
                       const void* d_dh, int64_t dh_stride, const void* d_x, int64_t x_stride, int64_t tokens,
                       int64_t dim, const int32_t* d_offsets, int64_t sequences, int form, int mix,
                       const float* d_initial, const float* d_dfinal, void* d_dgate, int64_t dgate_stride,
                       void* d_dx, int64_t dx_stride, float* d_dinitial, void* d_scratch, int64_t scratch_bytes,
                       hipStream_t stream)
{
    int st = check_gated(dtype, tokens, dim, d_offsets, sequences, form, mix);
    if (st == DS_OK)
        st = check_gated_strides({gate_stride, h_stride, dh_stride, mix ? x_stride : dim, dgate_stride, dx_stride}, dim);
    if (st != DS_OK || dim == 0 || sequences == 0) return st;
    const int esz = float_bytes(dtype);
    const int64_t states = span_bytes(sequences, dim, dim, 4);
    const Buf bufs[10] = {{d_gate, span_bytes(tokens, dim, gate_stride, esz), esz, false},
                          {d_h, span_bytes(tokens, dim, h_stride, esz), esz, false},
                          {d_dh, span_bytes(tokens, dim, dh_stride, esz), esz, false},
                          {d_x, mix ? span_bytes(tokens, dim, x_stride, esz) : 0, esz, false},
                          {d_offsets, d_offsets ? (sequences + 1) * 4 : 0, 4, false},
                          {d_initial, d_initial ? states : 0, 4, false},
                          {d_dfinal, d_dfinal ? states : 0, 4, false},
                          {d_dgate, span_bytes(tokens, dim, dgate_stride, esz), esz, true},
                          {d_dx, span_bytes(tokens, dim, dx_stride, esz), esz, true},
                          {d_dinitial, d_dinitial ? states : 0, 4, true}};
    st = check_buffers(bufs, 10);
    if (st != DS_OK) return st;
    const ds::GatedScanGrad a{{d_gate, d_x, const_cast<void*>(d_h), gate_stride, x_stride, h_stride, tokens, dim,
                               d_offsets, sequences, form, mix != 0, d_initial, nullptr},
                              d_dh, d_dgate, d_dx, dh_stride, dgate_stride, dx_stride, d_dfinal, d_dinitial};
    const ds::GatedPlan plan = ds::gated_plan(float_kind(dtype), true, mix != 0, tokens, dim);
    std::lock_guard<std::mutex> lock(g_mu);
    uint64_t* words = nullptr;
    st = gated_words(plan, ds_gated_scan_scratch_bytes(dtype, 1, tokens, dim), d_scratch, scratch_bytes, bufs, 10, stream,
                     &words);
    if (st != DS_OK) return st;
    return ds::launch_gated_scan_grad(float_kind(dtype), a, plan, words, g_spin_limit, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_gated_step(int dtype, const void* d_gate, int64_t gate_stride, const void* d_x, int64_t x_stride, int64_t rows,
                  int64_t dim, const int32_t* d_slots, float* d_state, int64_t pool, int64_t state_stride, int form,
                  int mix, void* d_h, int64_t h_stride, hipStream_t stream)
{
    const int esz = float_bytes(dtype);
    if (!esz) return DS_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || dim < 0 || pool < 0 || form < DS_GATE_DECAY || form > DS_GATE_SIGMOID || (mix != 0 && mix != 1) ||
        gate_stride < dim || x_stride < dim || h_stride < dim || state_stride < dim || (!d_slots && pool < rows))
        return DS_ERR_INVALID_VALUE;
    if (rows == 0 || dim == 0) return DS_OK;
    if (rows > (d_slots ? DS_GATED_MAX_SLOTS : kMost31) || dim > kMost31 || pool > kMost31) return DS_ERR_TOO_LARGE;
    const Buf bufs[5] = {{d_gate, span_bytes(rows, dim, gate_stride, esz), esz, false},
                         {d_x, span_bytes(rows, dim, x_stride, esz), esz, false},
                         {d_slots, d_slots ? rows * 4 : 0, 4, false},
                         {d_state, span_bytes(pool, dim, state_stride, 4), 4, true},
                         {d_h, span_bytes(rows, dim, h_stride, esz), esz, true}};
    const int st = check_buffers(bufs, 5);
    if (st != DS_OK) return st;
    const ds::GatedStep a{d_gate, d_x, d_h, gate_stride, x_stride, h_stride, rows, dim, d_slots, d_state, pool,
                          state_stride, form, mix != 0};
    if (ds::gated_step_blocks(float_kind(dtype), a) > kMaxTiles) return DS_ERR_TOO_LARGE;
    return ds::launch_gated_step(float_kind(dtype), a, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
}

// What the product and the gradient of its matrices have in common.
static int check_grouped(int dtype, int64_t x_rows, int num_experts, int64_t rows, int64_t cols, int64_t m,
                         const int32_t* index, int top_k)
{
    if (dtype != DS_BF16 && dtype != DS_FP16) return DS_ERR_UNSUPPORTED_DTYPE;
    if (x_rows < 0 || m < 0 || rows < 0 || cols < 0 || num_experts < 0 || num_experts > ds::grouped_most_experts() ||
        (index ? top_k < 1 : x_rows < m))
        return DS_ERR_INVALID_VALUE;
    return m > DS_GROUPED_MAX_ROWS || x_rows > kMost31 || rows > DS_EXPERTS_MAX_WIDTH || cols > DS_EXPERTS_MAX_WIDTH
               ? DS_ERR_TOO_LARGE
               : DS_OK;
}

// Division by top_k without one: with 2^shift >= top_k, magic = floor(2^32 (2^shift - top_k) / top_k) + 1.
static void set_divisor(ds::Grouped& a)
{
    const uint64_t d = a.index ? (uint64_t)a.top_k : 1;
    while (((uint64_t)1 << a.shift) < d) ++a.shift;
    a.magic = (uint32_t)(((((uint64_t)1 << a.shift) - d) << 32) / d + 1);
    const uint64_t all = (uint64_t)a.x_rows * d;
    a.entries = (uint32_t)(all < ((uint64_t)1 << 31) ? all : (uint64_t)1 << 31);
}

int ds_grouped_matmul(int dtype, const void* d_x, int64_t x_rows, int64_t x_stride, const void* d_w, int num_experts,
                      int64_t rows, int64_t cols, int transposed, const int32_t* d_offsets, int64_t m,
                      const int32_t* d_index, int top_k, void* d_y, int64_t y_stride, hipStream_t stream)
{
    int st = check_grouped(dtype, x_rows, num_experts, rows, cols, m, d_index, top_k);
    if (st != DS_OK) return st;
    if (transposed != 0 && transposed != 1) return DS_ERR_INVALID_VALUE;
    const int64_t depth = transposed ? rows : cols, out = transposed ? cols : rows;
    if (x_stride < depth || y_stride < out) return DS_ERR_INVALID_VALUE;
    if (num_experts == 0 || m == 0 || out == 0) return DS_OK;
    const Buf bufs[5] = {{d_x, span_bytes(x_rows, depth, x_stride, 2), 2, false},
                         {d_w, span_bytes(num_experts * rows, cols, cols, 2), 2, false},
                         {d_offsets, ((int64_t)num_experts + 1) * 4, 4, false},
                         {d_index, d_index ? m * 4 : 0, 4, false},
                         {d_y, span_bytes(m, out, y_stride, 2), 2, true}};
    st = check_buffers(bufs, 5);
    if (st != DS_OK) return st;
    ds::Grouped a{d_x, d_w, d_y, nullptr, x_rows, x_stride, y_stride, m, d_offsets, d_index, num_experts, top_k, rows,
                  cols, x_rows ? depth : 0, transposed != 0, false, 0, 0, 0};
    set_divisor(a);
    if (ds::grouped_tiles(a, false) > kMost31) return DS_ERR_TOO_LARGE;
    return ds::launch_grouped_matmul(float_kind(dtype), a, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
}

int ds_grouped_matmul_grad(int dtype, const void* d_dy, int64_t m, int64_t dy_stride, const void* d_x, int64_t x_rows,
                           int64_t x_stride, const int32_t* d_offsets, int num_experts, const int32_t* d_index,
                           int top_k, int64_t rows, int64_t cols, int grad_dtype, void* d_dw, int accumulate,
                           hipStream_t stream)
{
    int st = check_grouped(dtype, x_rows, num_experts, rows, cols, m, d_index, top_k);
    if (st != DS_OK) return st;
    if (grad_dtype != dtype && grad_dtype != DS_FP32) return DS_ERR_UNSUPPORTED_DTYPE;
    if (dy_stride < rows || x_stride < cols || (accumulate != 0 && accumulate != 1)) return DS_ERR_INVALID_VALUE;
    if (num_experts == 0 || rows == 0 || cols == 0 || (m == 0 && accumulate)) return DS_OK;
    const int gsz = float_bytes(grad_dtype);
    const Buf bufs[5] = {{d_dy, span_bytes(m, rows, dy_stride, 2), 2, false},
                         {d_x, span_bytes(x_rows, cols, x_stride, 2), 2, false},
                         {d_offsets, ((int64_t)num_experts + 1) * 4, 4, false},
                         {d_index, d_index ? m * 4 : 0, 4, false},
                         {d_dw, span_bytes(num_experts * rows, cols, cols, gsz), gsz, true}};
    st = check_buffers(bufs, 5);
    if (st != DS_OK) return st;
    // without rows of x every sum is empty, as with groups without rows
    ds::Grouped a{d_x, nullptr, const_cast<void*>(d_dy), d_dw, x_rows, x_stride, dy_stride, x_rows ? m : 0, d_offsets,
                  d_index, num_experts, top_k, rows, cols, 0, false, accumulate != 0, 0, 0, 0};
    set_divisor(a);
    if (ds::grouped_tiles(a, true) > kMost31) return DS_ERR_TOO_LARGE;
    return ds::launch_grouped_matmul_grad(float_kind(dtype), float_kind(grad_dtype), a, stream) == hipSuccess
               ? DS_OK
               : DS_ERR_HIP;
}

int ds_page_slots(const int32_t* d_context, const int32_t* d_new, int64_t requests, int32_t* d_tables, int64_t width,
                  int64_t table_stride, const int32_t* d_free, int64_t capacity, const int32_t* d_count, int page,
                  int32_t* d_offsets, int64_t* d_slots, int32_t* d_positions, int64_t tokens, int32_t* d_left,
                  hipStream_t stream)
{
    if (requests < 0 || width < 0 || table_stride < width || capacity < 0 || page < 1 || tokens < 0)
        return DS_ERR_INVALID_VALUE;
    if (requests > kMost31 || width > kMost31 || capacity > kMost31 || tokens > kMost31) return DS_ERR_TOO_LARGE;
    const Buf bufs[9] = {{d_context, requests * 4, 4, false},
                         {d_new, requests * 4, 4, false},
                         {d_tables, span_bytes(requests, width, table_stride, 4), 4, true},
                         {d_free, capacity * 4, 4, false},
                         {d_count, 4, 4, false},
                         {d_offsets, (requests + 1) * 4, 4, true},
                         {d_slots, tokens * 8, 8, true},
                         {d_positions, tokens * 4, 4, true},
                         {d_left, 4, 4, true}};
    const int st = check_buffers(bufs, 9);
    if (st != DS_OK) return st;
    const ds::PageSlots a{d_context, d_new, requests, d_tables, width, table_stride, d_free, capacity, d_count, page,
                          d_offsets, d_slots, d_positions, tokens, d_left};
    return ds::launch_page_slots(a, stream) == hipSuccess ? DS_OK : DS_ERR_HIP;
}

void ds_release_workspace(void)
{
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ws.empty()) (void)hipDeviceSynchronize();
    for (auto& kv : g_ws) {
        if (kv.second.base) (void)hipFree(kv.second.base);
        if (kv.second.aux) (void)hipFree(kv.second.aux);
        for (const Retired& r : kv.second.retired) (void)hipFree(r.p);
    }
    g_ws.clear();
}

int64_t ds_tile_elems(int dtype, int entry)
{
    if (!valid_dtype(dtype)) return -1;
    const int b = elem_bytes(dtype);
    switch (entry) {
    case DS_TILE_OF_SCAN_EXCLUSIVE: return ds::tile_elems(kind_of(dtype), false, INT64_MAX / 16);
    case DS_TILE_OF_SCAN_INCLUSIVE: return ds::tile_elems(kind_of(dtype), true, INT64_MAX / 16);
    case DS_TILE_OF_THREE_PASS: return ds::three_pass_tile_elems(b);
    case DS_TILE_OF_COMPACT: return ds::compact_tile_elems(b);
    case DS_TILE_OF_LDS_TILE_SCAN: return b == 4 ? ds::lds_tile_elems() : -1;
    case DS_TILE_OF_COUNTING_SORT: return b == 4 ? ds::sort_tile_elems(false) : -1;
    case DS_TILE_OF_COUNTING_SORT_VALUES: return b == 4 ? ds::sort_tile_elems(true) : -1;
    case DS_TILE_OF_MOE_ALIGN: return b == 4 ? ds::moe_tile_elems() : -1;
    default: return -1;
    }
}

int64_t ds_scan_tile_elems(int dtype, int inclusive, int64_t n)
{
    if (!valid_dtype(dtype) || (inclusive != 0 && inclusive != 1) || n < 0) return -1;
    return ds::tile_elems(kind_of(dtype), inclusive != 0, n);
}

int ds_version(void) { return 2; }

}  // extern "C"
