// gated_scan.hip -- a gated linear recurrence over packed sequences, channel
// by channel, its gradient, and its step for single tokens:
//
//   a_t = g_t, exp(g_t) or sigmoid(g_t)          b_t = x_t, or (1 - a_t) x_t
//   h_t = a_t h_{t-1} + b_t                      h before a sequence: its initial state, or 0
//
// It is a scan: steps (a, b) followed by (a', b') are the step (a a', a' b + b').
#include "float_types.hpp"
#include "gate.hpp"
#include "launch.hpp"

namespace ds {

// Sequence s's tokens [first, end), inside [0, tokens) whatever the offsets say.
__device__ __forceinline__ void sequence_range(const GatedScan& a, int64_t s, int64_t& first, int64_t& end)
{
    first = a.offsets ? min(max((int64_t)a.offsets[s], (int64_t)0), a.tokens) : 0;
    end = a.offsets ? min(max((int64_t)a.offsets[s + 1], first), a.tokens) : a.tokens;
}

template <typename T, GateForm FORM, bool MIX>
__global__ __launch_bounds__(kThreads) void gated_scan_kernel(GatedScan a)
{
    const int64_t cblocks = (a.dim + kThreads - 1) / kThreads;
    const int64_t s = blockIdx.x / cblocks, c = blockIdx.x % cblocks * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    int64_t first, end;
    sequence_range(a, s, first, end);
    float h = a.initial ? a.initial[s * a.dim + c] : 0.0f;
    for (int64_t t = first; t < end; ++t) {
        const float v = gate_of<FORM>((float)static_cast<const T*>(a.gate)[t * a.gate_stride + c]);
        const float x = (float)static_cast<const T*>(a.x)[t * a.x_stride + c];
        h = step_of<FORM>(v, h, MIX ? rest_of<FORM>(v) * x : x);
        static_cast<T*>(a.h)[t * a.h_stride + c] = (T)h;
    }
    if (a.final) a.final[s * a.dim + c] = h;
}

template <typename T, GateForm FORM, bool MIX>
__global__ __launch_bounds__(kThreads) void gated_scan_grad_kernel(GatedScanGrad a)
{
    const int64_t cblocks = (a.s.dim + kThreads - 1) / kThreads;
    const int64_t s = blockIdx.x / cblocks, c = blockIdx.x % cblocks * kThreads + threadIdx.x;
    if (c >= a.s.dim) return;
    int64_t first, end;
    sequence_range(a.s, s, first, end);
    float total = a.dfinal ? a.dfinal[s * a.s.dim + c] : 0.0f;  // what reaches h_t from later steps
    for (int64_t t = end - 1; t >= first; --t) {
        const float v = gate_of<FORM>((float)static_cast<const T*>(a.s.gate)[t * a.s.gate_stride + c]);
        float before = 0.0f;
        if (t > first)
            before = (float)static_cast<const T*>(a.s.h)[(t - 1) * a.s.h_stride + c];
        else if (a.s.initial)
            before = a.s.initial[s * a.s.dim + c];
        total += (float)static_cast<const T*>(a.dh)[t * a.dh_stride + c];
        float dx = total;
        if (MIX) {
            dx *= rest_of<FORM>(v);
            before -= (float)static_cast<const T*>(a.s.x)[t * a.s.x_stride + c];
        }
        static_cast<T*>(a.dx)[t * a.dx_stride + c] = (T)dx;
        static_cast<T*>(a.dgate)[t * a.dgate_stride + c] = (T)(total * before * slope_of<FORM>(v));
        total = step_of<FORM>(v, total, 0.0f);
    }
    if (a.dinitial) a.dinitial[s * a.s.dim + c] = total;
}

// A workgroup takes one row's columns. Rows whose slot an earlier row names are
// that slot's next tokens: the first such row's workgroups do them, in order.
template <typename T, GateForm FORM, bool MIX>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedStep a)
{
    const int64_t cblocks = (a.dim + kThreads - 1) / kThreads;
    int64_t i = blockIdx.x / cblocks;
    const int64_t c = blockIdx.x % cblocks * kThreads + threadIdx.x;
    const int64_t slot = a.slots ? a.slots[i] : i;
    const bool used = slot >= 0 && slot < a.pool;
    if (!used) {
        if (c < a.dim) static_cast<T*>(a.h)[i * a.h_stride + c] = (T)0.0f;
        return;
    }
    if (a.slots) {
        int earlier = 0;
        for (int64_t j = threadIdx.x; j < i; j += kThreads) earlier |= a.slots[j] == slot;
        if (__syncthreads_or(earlier)) return;
    }
    float* const state = a.state + slot * a.state_stride + c;
    float h = c < a.dim ? *state : 0.0f;
    for (;;) {
        if (c < a.dim) {
            const float v = gate_of<FORM>((float)static_cast<const T*>(a.gate)[i * a.gate_stride + c]);
            const float x = (float)static_cast<const T*>(a.x)[i * a.x_stride + c];
            h = step_of<FORM>(v, h, MIX ? rest_of<FORM>(v) * x : x);
            static_cast<T*>(a.h)[i * a.h_stride + c] = (T)h;
        }
        if (!a.slots) break;
        // the next row of this slot
        __shared__ int s_next;
        if (threadIdx.x == 0) s_next = INT32_MAX;
        __syncthreads();
        for (int64_t j = i + 1 + threadIdx.x; j < a.rows; j += kThreads)
            if (a.slots[j] == slot) {
                atomicMin(&s_next, (int)j);
                break;
            }
        __syncthreads();
        const int next = s_next;
        __syncthreads();
        if (next == INT32_MAX) break;
        i = next;
    }
    if (c < a.dim) *state = h;
}

int64_t gated_scan_blocks(const GatedScan& a) { return (a.dim + kThreads - 1) / kThreads * a.sequences; }
int64_t gated_step_blocks(const GatedStep& a) { return (a.dim + kThreads - 1) / kThreads * a.rows; }

template <typename F> static void with_form(int form, bool mix, F&& f)
{
    const auto go = [&](auto fm) {
        if (mix)
            f(fm, std::true_type{});
        else
            f(fm, std::false_type{});
    };
    if (form == kDecay)
        go(std::integral_constant<GateForm, kDecay>{});
    else if (form == kLog)
        go(std::integral_constant<GateForm, kLog>{});
    else
        go(std::integral_constant<GateForm, kSigmoid>{});
}

template <typename F> static hipError_t with_type(ElemKind kind, int form, bool mix, F&& f)
{
    with_form(form, mix, [&](auto fm, auto mx) {
        if (kind == kF32)
            f(float{}, fm, mx);
        else if (kind == kBF16)
            f(bf16{}, fm, mx);
        else
            f(fp16{}, fm, mx);
    });
    return hipGetLastError();
}

hipError_t launch_gated_scan(ElemKind kind, const GatedScan& a, hipStream_t stream)
{
    return with_type(kind, a.form, a.mix, [&](auto t, auto fm, auto mx) {
        gated_scan_kernel<decltype(t), decltype(fm)::value, decltype(mx)::value>
            <<<dim3((unsigned)gated_scan_blocks(a)), dim3(kThreads), 0, stream>>>(a);
    });
}

hipError_t launch_gated_scan_grad(ElemKind kind, const GatedScanGrad& a, hipStream_t stream)
{
    return with_type(kind, a.s.form, a.s.mix, [&](auto t, auto fm, auto mx) {
        gated_scan_grad_kernel<decltype(t), decltype(fm)::value, decltype(mx)::value>
            <<<dim3((unsigned)gated_scan_blocks(a.s)), dim3(kThreads), 0, stream>>>(a);
    });
}

hipError_t launch_gated_step(ElemKind kind, const GatedStep& a, hipStream_t stream)
{
    return with_type(kind, a.form, a.mix, [&](auto t, auto fm, auto mx) {
        gated_step_kernel<decltype(t), decltype(fm)::value, decltype(mx)::value>
            <<<dim3((unsigned)gated_step_blocks(a)), dim3(kThreads), 0, stream>>>(a);
    });
}

}  // namespace ds
