// gated_scan_grad.hip -- the gradient of the gated recurrence (gated_scan.hip):
//
//   G_t = dh_t + a_{t+1} G_{t+1}                  at a sequence's last row: dh_t + dfinal
//   dx_t = G_t, or (1 - a_t) G_t with mix         dgate_t = G_t (h_{t-1}, or h_{t-1} - x_t) da/dg
//
// and dinitial = a G of the first row. h_{t-1} is the scan's output.
#include "gated.hpp"

namespace ds {

// The gradient runs from the last row to the first. What passes from row t to
// row t - 1 is S = a_t G_t, with G_t = dh_t + S of row t + 1 (or dfinal), so the
// scan's pairs need no row but their own.
template <typename T, int V, GateForm FORM, bool MIX, int TQ>
__global__ __launch_bounds__(kThreads, 2) void gated_scan_grad_kernel(GatedScanGrad a, GatedWords w)
{
    constexpr int kRows = kSub * TQ, kSpan = kLanes * V;
    __shared__ float s_a[kSub][kSpan], s_b[kSub][kSpan];
    __shared__ int s_new[kSub], s_seq[kRows + 2];
    const Place<V> p(a.s.dim);
    const int part = (int)threadIdx.x / kLanes, at = (int)threadIdx.x % kLanes * V;  // parts from the last row on
    const int64_t tiles = gridDim.x / p.cblocks, row0 = (tiles - 1 - p.tile) * kRows;
    const int top = (kSub - 1 - part) * TQ;  // the part's first row in the tile
    const int64_t mine = row0 + top;
    if (a.s.tokens > 0) {
        const int64_t left = a.s.tokens - mine;  // rows of this part that there are, or more
        const Rows<const T> gate(static_cast<const T*>(a.s.gate), a.s.gate_stride, row0, top, p.channel);
        const Rows<const T> grad(static_cast<const T*>(a.dh), a.dh_stride, row0, top, p.channel);
        const Rows<const T> state(static_cast<const T*>(a.s.h), a.s.h_stride, row0, top, p.channel);
        const Rows<const T> in(static_cast<const T*>(a.s.x), a.s.x_stride, row0, top, p.channel);
        Cells<T, V> g[TQ] = {}, dh[TQ] = {}, x[TQ] = {}, before[TQ] = {};
        if (row0 > 0 && row0 + kRows <= a.s.tokens) {
#pragma unroll
            for (int k = TQ - 1; k >= 0; --k) {
                g[k].load(gate.at(k), gate.bytes);
                dh[k].load(grad.at(k), grad.bytes);
            }
#pragma unroll
            for (int k = TQ - 1; k >= 0; --k) {
                before[k].load(state.at(k - 1), state.bytes);
                if constexpr (MIX) x[k].load(in.at(k), in.bytes);
            }
        } else {
#pragma unroll
            for (int k = TQ - 1; k >= 0; --k)
                if (k < left) {
                    g[k].load(gate.at(k), gate.bytes);
                    dh[k].load(grad.at(k), grad.bytes);
                    if (mine + k > 0) before[k].load(state.at(k - 1), state.bytes);
                    if constexpr (MIX) x[k].load(in.at(k), in.bytes);
                }
        }
        const bool inside = find_sequences<kRows>(a.s, row0, s_seq);
        uint32_t first = 0, last = 0, none = 0;
        if (!inside)
            for (int k = 0; k < TQ; ++k) {
                const int s = s_seq[top + k + 1];
                none |= (uint32_t)(s < 0) << k;
                first |= (uint32_t)(s >= 0 && s != s_seq[top + k]) << k;
                last |= (uint32_t)(s >= 0 && s != s_seq[top + k + 2]) << k;
            }
        const auto states = [&](const float* from, int k, float (&h)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = 0.0f;
            if (from) load_states(from + (int64_t)s_seq[top + k + 1] * a.s.dim + p.channel, h);
        };
        float v[TQ][V], pa[V], s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            pa[i] = 1.0f;
            s[i] = 0.0f;
        }
#pragma unroll
        for (int k = TQ - 1; k >= 0; --k) {
            if (last >> k & 1) states(a.dfinal, k, s);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] = gate_of<T, FORM>(g[k][i]);
                s[i] = keep_of<FORM>(v[k][i], s[i] + dh[k][i]);
                pa[i] = keep_of<FORM>(v[k][i], pa[i]);
            }
            pin(v[k]);
            dh[k].pin();
        }
        store_states(&s_a[part][at], pa);
        store_states(&s_b[part][at], s);
        if (at == 0) s_new[part] = last != 0;
        __syncthreads();
        join_parts<kSpan>(s_a, s_b, s_new, p.tile, tiles, p.cblock, p.cblocks,
                          s_seq[kRows] >= 0 && s_seq[kRows + 1] == s_seq[kRows], w);
        __syncthreads();
        load_states(&s_a[part][at], s);
        const Rows<T> to_gate(static_cast<T*>(a.dgate), a.dgate_stride, row0, top, p.channel);
        const Rows<T> to_x(static_cast<T*>(a.dx), a.dx_stride, row0, top, p.channel);
#pragma unroll
        for (int k = TQ - 1; k >= 0; --k) {
            if (last >> k & 1) states(a.dfinal, k, s);
            float prior[V];
            if (first >> k & 1)
                states(a.s.initial, k, prior);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) prior[i] = before[k][i];
            float dg[V], dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float total = s[i] + dh[k][i];
                const float from = MIX ? prior[i] - x[k][i] : prior[i];
                dg[i] = total * from * slope_of<FORM>(v[k][i]);
                dx[i] = MIX ? total * rest_of<FORM>(v[k][i]) : total;
                s[i] = keep_of<FORM>(v[k][i], total);
            }
            if (p.live && !(none >> k & 1)) {
                Cells<T, V> out;
                out.set(dg);
                out.store(to_gate.at(k), to_gate.bytes);
                out.set(dx);
                out.store(to_x.at(k), to_x.bytes);
            }
            if (p.live && (first >> k & 1) && a.dinitial)
                store_states(a.dinitial + (int64_t)s_seq[top + k + 1] * a.s.dim + p.channel, s);
        }
    }
    pass_empty(a.s, p, a.dfinal, a.dinitial);
}

hipError_t launch_gated_scan_grad(ElemKind kind, const GatedScanGrad& a, const GatedPlan& plan, uint64_t* scratch,
                                  uint32_t spin_limit, hipStream_t stream)
{
    const GatedWords w = clear_words(plan, scratch, spin_limit, stream);
    const dim3 grid((unsigned)(plan.tiles * plan.cblocks)), block(kThreads);
    return with_type(kind, a.s.form, a.s.mix, [&](auto t, auto fm, auto mx) {
        using T = decltype(t);
        if (vector_of(kind, a.s.dim) == 1)
            gated_scan_grad_kernel<T, 1, decltype(fm)::value, decltype(mx)::value, kGradRows<T>><<<grid, block, 0, stream>>>(a, w);
        else
            gated_scan_grad_kernel<T, Vec16<T>::kN, decltype(fm)::value, decltype(mx)::value, kGradRows<T>>
                <<<grid, block, 0, stream>>>(a, w);
    });
}

}  // namespace ds
