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
// scan's pairs need no row but their own. h_{t-1} and x are loaded into the gates'
// registers once the tile's pairs are made, and arrive while it waits.
template <typename T, int V, GateForm FORM, bool MIX, int TQ>
__global__ __launch_bounds__(kThreads, (kGradPerCu<T, MIX>)) void gated_scan_grad_kernel(GatedScanGrad a, GatedWords w)
{
    constexpr int kRows = kSub * TQ, kSpan = kLanes * V;
    __shared__ float s_a[kSub][kSpan], s_b[kSub][kSpan];
    __shared__ int s_new[kSub], s_seq[kRows + 2];
    const Place<V> p(a.s.dim);
    const int part = (int)threadIdx.x / kLanes, at = (int)threadIdx.x % kLanes * V;  // parts from the last row on
    const int64_t tiles = gridDim.x / p.cblocks, tile = tiles - 1 - p.tile, row0 = tile * kRows;
    const int top = (kSub - 1 - part) * TQ;  // the part's first row in the tile
    const int64_t mine = row0 + top;
    if (a.s.tokens > 0) {
        const Rows<const T> gate(static_cast<const T*>(a.s.gate), a.s.gate_stride, row0, top, p.channel);
        const Rows<const T> grad(static_cast<const T*>(a.dh), a.dh_stride, row0, top, p.channel);
        const Rows<const T> state(static_cast<const T*>(a.s.h), a.s.h_stride, row0, top, p.channel);
        const Rows<const T> in(static_cast<const T*>(a.s.x), a.s.x_stride, row0, top, p.channel);
        const Rows<T> to_gate(static_cast<T*>(a.dgate), a.dgate_stride, row0, top, p.channel);
        const Rows<T> to_x(static_cast<T*>(a.dx), a.dx_stride, row0, top, p.channel);
        const TileInfo info = info_of(a.s, w, tiles, tile, kRows);
        Product<FORM> all[V];
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 0.0f;
        const auto publish = [&](bool anew, Enter enter, const float* given) {
            float pa[V];
#pragma unroll
            for (int i = 0; i < V; ++i) pa[i] = all[i].value();
            store_states(&s_a[part][at], pa);
            store_states(&s_b[part][at], s);
            if (at == 0) s_new[part] = anew;
            __syncthreads();
            join_parts<V, FORM>(s_a, s_b, s_new, p, tiles, a.s.dim, enter, given, w);
            __syncthreads();
            load_states(&s_a[part][at], s);
        };
        // row k's outputs, from v, what reaches it, the state before it and x
        const auto finish = [&](int k, bool there, const float (&v)[V], const float (&total)[V], const float (&prior)[V],
                                const Cells<T, V>& x) {
            float dg[V], dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dg[i] = total[i] * (MIX ? prior[i] - x[i] : prior[i]) * slope_of<FORM>(v[i]);
                dx[i] = MIX ? total[i] * rest_of<FORM>(v[i]) : total[i];
            }
            if (!there) return;
            Cells<T, V> out;
            out.set(dg);
            out.store(to_gate.at(k), to_gate.bytes);
            out.set(dx);
            out.store(to_x.at(k), to_x.bytes);
        };
        const auto states_of = [&](const float* from, int sequence, float (&h)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = 0.0f;
            if (from) load_states(from + (int64_t)sequence * a.s.dim + p.channel, h);
        };
        if (info.sequence >= 0) {
            const bool whole = row0 > 0 && row0 + kRows <= a.s.tokens;
            Cells<T, V> g[TQ], dh[TQ], x[TQ], before[TQ];
            if (whole) {
#pragma unroll
                for (int k = TQ - 1; k >= 0; --k) {
                    g[k].load(gate.at(k), gate.bytes);
                    dh[k].load(grad.at(k), grad.bytes);
                }
            } else {  // rows past the end pass on what reaches them
#pragma unroll
                for (int k = TQ - 1; k >= 0; --k) {
                    g[k].fill(open_gate<T, FORM>());
                    dh[k].fill((T)0.0f);
                    if (mine + k < a.s.tokens) {
                        g[k].load(gate.at(k), gate.bytes);
                        dh[k].load(grad.at(k), grad.bytes);
                    }
                }
            }
            float v[TQ][V];
#pragma unroll
            for (int k = TQ - 1; k >= 0; --k) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[k][i] = gate_of<T, FORM>(g[k][i]);
                    s[i] = keep_of<FORM>(v[k][i], s[i] + dh[k][i]);
                    all[i].step(v[k][i]);
                }
                pin(v[k]);
                dh[k].pin();
            }
            if (whole) {  // in the gates' registers, while the tile waits
#pragma unroll
                for (int k = TQ - 1; k >= 0; --k) {
                    before[k].load(state.at(k - 1), state.bytes);
                    if constexpr (MIX) x[k].load(in.at(k), in.bytes);
                }
            } else {
#pragma unroll
                for (int k = TQ - 1; k >= 0; --k) {
                    x[k].fill((T)0.0f);
                    before[k].fill((T)0.0f);
                    if (mine + k < a.s.tokens) {
                        if (mine + k > 0) before[k].load(state.at(k - 1), state.bytes);
                        if constexpr (MIX) x[k].load(in.at(k), in.bytes);
                    }
                }
            }
            publish(false, info.ends & 2 ? kGiven : kBefore,
                    a.dfinal ? a.dfinal + (int64_t)info.sequence * a.s.dim : nullptr);
            const bool starts = (info.ends & 1) && part == kSub - 1;  // row 0 of this part is the sequence's first
#pragma unroll
            for (int k = TQ - 1; k >= 0; --k) {
                float prior[V], total[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    prior[i] = before[k][i];
                    total[i] = s[i] + dh[k][i];
                }
                if (k == 0 && starts) states_of(a.s.initial, info.sequence, prior);
                finish(k, p.live && (whole || mine + k < a.s.tokens), v[k], total, prior, x[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = keep_of<FORM>(v[k][i], total[i]);
            }
            if (starts && p.live && a.dinitial) store_states(a.dinitial + (int64_t)info.sequence * a.s.dim + p.channel, s);
        } else {
            find_sequences<kRows>(a.s, row0, s_seq);
            // f(row of the part, of the tile, its sequence, gate, dh, x, state before) from the last row on
            const auto rows = [&](auto second, auto&& f) {
#pragma unroll 1
                for (int k0 = TQ - 2; k0 >= 0; k0 -= 2) {
                    Cells<T, V> g[2], dh[2], x[2], before[2];
#pragma unroll
                    for (int j = 1; j >= 0; --j)
                        if (mine + k0 + j < a.s.tokens) {
                            g[j].load(gate.at(k0 + j), gate.bytes);
                            dh[j].load(grad.at(k0 + j), grad.bytes);
                            if constexpr (decltype(second)::value) {
                                if (mine + k0 + j > 0) before[j].load(state.at(k0 + j - 1), state.bytes);
                                if constexpr (MIX) x[j].load(in.at(k0 + j), in.bytes);
                            }
                        }
#pragma unroll
                    for (int j = 1; j >= 0; --j) {
                        const int row = top + k0 + j, sequence = s_seq[row + 1];
                        if (sequence < 0) continue;
                        if (s_seq[row + 2] != sequence) states_of(a.dfinal, sequence, s);  // the last of its sequence
                        f(k0 + j, row, sequence, g[j], dh[j], x[j], before[j]);
                    }
                }
            };
            using C = Cells<T, V>;
            bool anew = false;
            rows(std::false_type{}, [&](int, int row, int sequence, const C& g, const C& dh, const C&, const C&) {
                anew |= s_seq[row + 2] != sequence;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = gate_of<T, FORM>(g[i]);
                    s[i] = keep_of<FORM>(v, s[i] + dh[i]);
                    all[i].step(v);
                }
            });
            publish(anew, s_seq[kRows] >= 0 && s_seq[kRows + 1] == s_seq[kRows] ? kBefore : kNone, nullptr);
            rows(std::true_type{}, [&](int k, int row, int sequence, const C& g, const C& dh, const C& x, const C& before) {
                const bool starts = s_seq[row] != sequence;
                float v[V], total[V], prior[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[i] = gate_of<T, FORM>(g[i]);
                    total[i] = s[i] + dh[i];
                    prior[i] = before[i];
                }
                if (starts) states_of(a.s.initial, sequence, prior);
                finish(k, p.live, v, total, prior, x);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = keep_of<FORM>(v[i], total[i]);
                if (starts && p.live && a.dinitial) store_states(a.dinitial + (int64_t)sequence * a.s.dim + p.channel, s);
            });
        }
    }
    pass_empty(a.s, p, a.dfinal, a.dinitial);
}

hipError_t take_gated_scan_grad_give_up(bool* flag) { return take_give_up(flag); }

hipError_t launch_gated_scan_grad(ElemKind kind, const GatedScanGrad& a, const GatedPlan& plan, uint64_t* scratch,
                                  uint32_t spin_limit, hipStream_t stream)
{
    const GatedWords w = begin_words(a.s, plan, scratch, spin_limit, stream);
    const dim3 grid((unsigned)(plan.tiles * plan.cblocks)), block(kThreads);
    return with_type(kind, a.s.form, a.s.mix, [&](auto t, auto fm, auto mx) {
        using T = decltype(t);
        with_vector<T>(plan.vector, [&](auto v) {
            constexpr bool kMix = decltype(mx)::value;
            gated_scan_grad_kernel<T, decltype(v)::value, decltype(fm)::value, kMix, kGradRows<T, kMix>>
                <<<grid, block, 0, stream>>>(a, w);
        });
    });
}

}  // namespace ds
