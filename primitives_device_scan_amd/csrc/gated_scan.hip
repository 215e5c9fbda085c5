// gated_scan.hip -- a gated linear recurrence over packed sequences, channel
// by channel, its gradient, and its step for single tokens:
//
//   a_t = g_t, exp(g_t) or sigmoid(g_t)          b_t = x_t, or (1 - a_t) x_t
//   h_t = a_t h_{t-1} + b_t                      h before a sequence: its initial state, or 0
//
// The scan itself (see gated.hpp for how it is cut up) and the step for single
// tokens; the gradient is in gated_scan_grad.hip.
#include "gated.hpp"

namespace ds {

template <typename T, int V, GateForm FORM, bool MIX, int TQ>
__global__ __launch_bounds__(kThreads, 3) void gated_scan_kernel(GatedScan a, GatedWords w)
{
    constexpr int kRows = kSub * TQ, kSpan = kLanes * V;
    __shared__ float s_a[kSub][kSpan], s_b[kSub][kSpan];
    __shared__ int s_new[kSub], s_seq[kRows + 2];
    const Place<V> p(a.dim);
    const int part = (int)threadIdx.x / kLanes, at = (int)threadIdx.x % kLanes * V;
    const int64_t tiles = gridDim.x / p.cblocks, row0 = p.tile * kRows, mine = row0 + part * TQ;
    if (a.tokens > 0) {
        const Rows<const T> gate(static_cast<const T*>(a.gate), a.gate_stride, row0, part * TQ, p.channel);
        const Rows<const T> in(static_cast<const T*>(a.x), a.x_stride, row0, part * TQ, p.channel);
        const Rows<T> to(static_cast<T*>(a.h), a.h_stride, row0, part * TQ, p.channel);
        const TileInfo info = info_of(a, w, tiles, p.tile, kRows);
        Product<FORM> all[V];
        float h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = 0.0f;
        const auto publish = [&](bool anew, Enter enter, const float* given) {
            float pa[V];
#pragma unroll
            for (int i = 0; i < V; ++i) pa[i] = all[i].value();
            store_states(&s_a[part][at], pa);
            store_states(&s_b[part][at], h);
            if (at == 0) s_new[part] = anew;
            __syncthreads();
            join_parts<V, FORM>(s_a, s_b, s_new, p, tiles, a.dim, enter, given, w);
            __syncthreads();
            load_states(&s_a[part][at], h);
        };
        if (info.sequence >= 0) {
            const int64_t states = (int64_t)info.sequence * a.dim;
            const bool whole = row0 + kRows <= a.tokens;
            Cells<T, V> g[TQ], x[TQ];
            if (whole) {
#pragma unroll
                for (int k = 0; k < TQ; ++k) {
                    g[k].load(gate.at(k), gate.bytes);
                    x[k].load(in.at(k), in.bytes);
                }
            } else {  // rows past the end leave the state as it is
#pragma unroll
                for (int k = 0; k < TQ; ++k) {
                    g[k].fill(open_gate<T, FORM>());
                    x[k].fill((T)0.0f);
                    if (mine + k < a.tokens) {
                        g[k].load(gate.at(k), gate.bytes);
                        x[k].load(in.at(k), in.bytes);
                    }
                }
            }
            float v[TQ][V];
#pragma unroll
            for (int k = 0; k < TQ; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[k][i] = gate_of<T, FORM>(g[k][i]);
                    h[i] = step_of<FORM, MIX>(v[k][i], h[i], x[k][i]);
                    all[i].step(v[k][i]);
                }
                pin(v[k]);
                x[k].pin();
            }
            publish(false, info.ends & 1 ? kGiven : kBefore, a.initial ? a.initial + states : nullptr);
#pragma unroll
            for (int k = 0; k < TQ; ++k) {
                Cells<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i) h[i] = step_of<FORM, MIX>(v[k][i], h[i], x[k][i]);
                out.set(h);
                if (p.live && (whole || mine + k < a.tokens)) out.store(to.at(k), to.bytes);
            }
            if ((info.ends & 2) && part == kSub - 1 && p.live && a.final) store_states(a.final + states + p.channel, h);
        } else {
            find_sequences<kRows>(a, row0, s_seq);
            // f(row of the part, its sequence, gate, x) for the part's rows that belong to one
            const auto rows = [&](auto&& f) {
#pragma unroll 1
                for (int k0 = 0; k0 < TQ; k0 += 4) {
                    Cells<T, V> g[4], x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (mine + k0 + j < a.tokens) {
                            g[j].load(gate.at(k0 + j), gate.bytes);
                            x[j].load(in.at(k0 + j), in.bytes);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = part * TQ + k0 + j, s = s_seq[row + 1];
                        if (s < 0) continue;
                        if (s_seq[row] != s) {  // the first of its sequence
#pragma unroll
                            for (int i = 0; i < V; ++i) h[i] = 0.0f;
                            if (a.initial) load_states(a.initial + (int64_t)s * a.dim + p.channel, h);
                        }
                        f(k0 + j, row, s, g[j], x[j]);
                    }
                }
            };
            static_assert(TQ % 4 == 0, "four rows at a time");
            bool anew = false;
            rows([&](int, int row, int s, const Cells<T, V>& g, const Cells<T, V>& x) {
                anew |= s_seq[row] != s;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = gate_of<T, FORM>(g[i]);
                    h[i] = step_of<FORM, MIX>(v, h[i], x[i]);
                    all[i].step(v);
                }
            });
            publish(anew, s_seq[1] >= 0 && s_seq[0] == s_seq[1] ? kBefore : kNone, nullptr);
            rows([&](int k, int row, int s, const Cells<T, V>& g, const Cells<T, V>& x) {
                Cells<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i) h[i] = step_of<FORM, MIX>(gate_of<T, FORM>(g[i]), h[i], x[i]);
                out.set(h);
                if (!p.live) return;
                out.store(to.at(k), to.bytes);
                if (s_seq[row + 2] != s && a.final) store_states(a.final + (int64_t)s * a.dim + p.channel, h);
            });
        }
    }
    pass_empty(a, p, a.initial, a.final);
}

__global__ __launch_bounds__(kThreads) void gated_begin_kernel(GatedScan a, u32x4* words, int64_t count, TileInfo* infos,
                                                               int64_t tiles, int rows)
{
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x, all = (int64_t)gridDim.x * kThreads;
    for (int64_t i = at; i < count; i += all) words[i] = u32x4{0, 0, 0, 0};
    for (int64_t i = at; i < tiles; i += all) infos[i] = tile_info(a, i * rows, rows);
}

// A workgroup takes one row's columns, V to a thread. Rows whose slot an earlier
// row names are that slot's next tokens: the first such row's workgroups do them,
// in order. All slots are looked through for that while the row's data is loaded:
// n slots by each of n rows, which shows from some thousands of rows on (of 2,048
// channels in bf16 with slots and without them: 1,024 rows 10.2 and 9.4 us, 4,096
// 29 and 19, 16,384 199 and 82, 65,536 1,790 and 322). A step moves 3 elements and a
// state in and out for 8 operations: memory's time, a launch's for few rows (1,024 x
// 4,096 bf16 in a pool of 4,096: 13.6 us, 4.3 TB/s; 64 x 2,048: 3.1). 16 bytes to a
// thread; with a channel to a thread 26 us.
template <typename T, int V, GateForm FORM, bool MIX>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedStep a)
{
    const int64_t wide = (int64_t)blockDim.x * V, cblocks = (a.dim + wide - 1) / wide;
    int64_t i = blockIdx.x / cblocks;
    const int64_t c = blockIdx.x % cblocks * wide + (int64_t)threadIdx.x * V;
    const int here = (int)min((int64_t)V, a.dim - c);  // this thread's columns, or none
    const auto each = [&](auto&& whole, auto&& one) {
        if (here == V)
            whole();
        else
            for (int k = 0; k < here; ++k) one(k);
    };
    const int64_t slot = a.slots ? a.slots[i] : i;
    if (slot < 0 || slot >= a.pool) {
        T* const h = static_cast<T*>(a.h) + i * a.h_stride + c;
        Cells<T, V> zero;
        zero.fill((T)0.0f);
        each([&] { zero.store(h, 0); }, [&](int k) { h[k] = (T)0.0f; });
        return;
    }
    float* const state = a.state + slot * a.state_stride + c;
    const T* const gate = static_cast<const T*>(a.gate) + c;
    const T* const in = static_cast<const T*>(a.x) + c;
    Cells<T, V> g, x;
    float h[V];
    g.fill((T)0.0f);
    x.fill((T)0.0f);
    const auto load = [&] {
        each(
            [&] {
                g.load(gate + i * a.gate_stride, 0);
                x.load(in + i * a.x_stride, 0);
            },
            [&](int k) {
                g.put(k, gate[i * a.gate_stride + k]);
                x.put(k, in[i * a.x_stride + k]);
            });
    };
    load();
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = 0.0f;
    each([&] { load_states(state, h); },
         [&](int k) {
#pragma unroll
             for (int j = 0; j < V; ++j)
                 if (j == k) h[j] = state[k];
         });
    __shared__ int s_first, s_next;  // the first row of this slot; the next one after i
    int next = INT32_MAX;
    if (a.slots) {
        if (threadIdx.x == 0) s_first = s_next = INT32_MAX;
        __syncthreads();
        for (int64_t j = threadIdx.x; j < a.rows; j += blockDim.x)
            if (a.slots[j] == slot && j != i) atomicMin(j < i ? &s_first : &s_next, (int)j);
        __syncthreads();
        if (s_first != INT32_MAX) return;  // an earlier row's workgroups do this one
        next = s_next;
    }
    // From the row behind `from` on, as far as there is none: all rows of a slot in one walk.
    const auto find_next = [&](int64_t from) {
        __syncthreads();  // all have read s_next
        if (threadIdx.x == 0) s_next = INT32_MAX;
        __syncthreads();
        for (int64_t j = from + 1 + threadIdx.x; j - (int)threadIdx.x < a.rows; j += blockDim.x) {
            const bool hit = j < a.rows && a.slots[j] == slot;
            if (hit) atomicMin(&s_next, (int)j);
            if (__syncthreads_or(hit)) break;
        }
        return s_next;
    };
    for (;;) {
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = step_of<FORM, MIX>(gate_of<T, FORM>(g[k]), h[k], x[k]);
        T* const to = static_cast<T*>(a.h) + i * a.h_stride + c;
        Cells<T, V> out;
        out.set(h);
        each([&] { out.store(to, 0); }, [&](int k) { to[k] = (T)out[k]; });
        if (next == INT32_MAX) break;
        i = next;
        load();
        next = find_next(i);
    }
    each([&] { store_states(state, h); },
         [&](int k) {
#pragma unroll
             for (int j = 0; j < V; ++j)
                 if (j == k) state[k] = h[j];
         });
}

GatedPlan gated_plan(ElemKind kind, bool grad, bool mix, int64_t tokens, int64_t dim)
{
    return gated_plan_of(kind, grad, mix, tokens, dim);
}

// Threads to a workgroup of a step: those that a row needs, in whole waves.
static int step_threads(const GatedStep& a, int v)
{
    const int64_t need = (a.dim + v - 1) / v;
    return need >= kThreads ? kThreads : (int)((need + kWave - 1) / kWave * kWave);
}

int64_t gated_step_blocks(ElemKind kind, const GatedStep& a)
{
    const int v = vector_of(kind, a.dim);
    const int64_t wide = (int64_t)step_threads(a, v) * v;
    return (a.dim + wide - 1) / wide * a.rows;
}

hipError_t take_gated_scan_give_up(bool* flag) { return take_give_up(flag); }

GatedWords begin_words(const GatedScan& a, const GatedPlan& plan, uint64_t* scratch, uint32_t spin_limit,
                       hipStream_t stream)
{
    uint64_t* const entries = scratch + plan.pair_words;
    uint64_t* const infos = entries + plan.entry_words;
    if (plan.words) {
        const int64_t vecs = (plan.pair_words + plan.entry_words) / 2;  // both even
        const int64_t most = vecs > plan.tiles ? vecs : plan.tiles, blocks = (most + kThreads - 1) / kThreads;
        gated_begin_kernel<<<dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(kThreads), 0, stream>>>(
            a, reinterpret_cast<u32x4*>(scratch), vecs, reinterpret_cast<TileInfo*>(infos), plan.tiles, (int)plan.rows);
    }
    return GatedWords{scratch, entries, infos, spin_limit};
}

hipError_t launch_gated_scan(ElemKind kind, const GatedScan& a, const GatedPlan& plan, uint64_t* scratch,
                             uint32_t spin_limit, hipStream_t stream)
{
    const GatedWords w = begin_words(a, plan, scratch, spin_limit, stream);
    const dim3 grid((unsigned)(plan.tiles * plan.cblocks)), block(kThreads);
    return with_type(kind, a.form, a.mix, [&](auto t, auto fm, auto mx) {
        using T = decltype(t);
        with_vector<T>(plan.vector, [&](auto v) {
            gated_scan_kernel<T, decltype(v)::value, decltype(fm)::value, decltype(mx)::value, kScanRows<T>>
                <<<grid, block, 0, stream>>>(a, w);
        });
    });
}

hipError_t launch_gated_step(ElemKind kind, const GatedStep& a, hipStream_t stream)
{
    const int v = vector_of(kind, a.dim);
    const dim3 grid((unsigned)gated_step_blocks(kind, a)), block(step_threads(a, v));
    return with_type(kind, a.form, a.mix, [&](auto t, auto fm, auto mx) {
        using T = decltype(t);
        if (v == 1)
            gated_step_kernel<T, 1, decltype(fm)::value, decltype(mx)::value><<<grid, block, 0, stream>>>(a);
        else
            gated_step_kernel<T, Vec16<T>::kN, decltype(fm)::value, decltype(mx)::value><<<grid, block, 0, stream>>>(a);
    });
}

}  // namespace ds
