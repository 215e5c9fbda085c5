// moe_experts.hip -- the experts of a mixture-of-experts layer for a few
// tokens: for every token t and choice j with expert e = ids[t, j],
//
//   h = silu(G_e x_t) * (U_e x_t)          G_e, U_e: the first and the last F rows of w_in[e]
//   y_t = sum over j of weights[t, j] * (w_out[e] h)
//
// With a few tokens the weights are what has to be read (3 D F values per
// expert that any token chose, once), so the kernels are built to stream them:
// 16 rows to a tile are the A operand of the matrix instructions, the expert's
// tokens, 16 to a block, are the B operand, read from the cache.
//
// The launches: a plan of which workgroups serve which tokens (above 64
// assignments), gate/up products and activation into `h` (one row per
// assignment), down products into `part` (one 32-bit row per assignment) and
// the weighted sum over each token's choices, in order of the choices, so that
// the result is the same on every run. (Matrix-vector kernels for one token, with
// the sum in the down products' launch, took as long: 12 + 11 us against 12 + 7
// + 4 for top-8 of 128, 2,048 x 768. A launch's 3 us and the bytes are the time.)
//
// The matrix instructions take h in x's 16-bit type. Rounding it there would
// add as much error as the output's own rounding (1.4 times in all), so h is
// kept as its rounded value and the rounded rest, and a token has two columns
// in the down products. That costs nothing for an expert of up to eight tokens
// (blocks are 16 columns wide, and the weights' bytes bound these products); an
// expert of more takes the rounded values alone. A relative error of 0.0016
// becomes one of 0.0021-0.0024 in bf16 (whose own rounding is 0.0016), and a
// token's last bits go by how many tokens its expert has. Both halves for every
// token were measured: 256 tokens, top-8 of 256, 2,048 x 768: 400 -> 415 us; 64,
// top-6 of 64, 2,048 x 1,408 in e4m3: 107 -> 125; 512, top-2 of 8, 4,096 x 2,048:
// 253 -> 286; 300, top-2 of 20, 1,000 x 777: 61 -> 77.
// Measured: 256 tokens, top-8 of 256, 2,048 x 768 in bf16: gate/up 246-252 us
// (1.50 GB at 6.0-6.1 TB/s; 1.56 GB are fetched, as crowded experts' weights are
// read again), down 135-138 (0.75 GB at 5.4-5.6), plan and sum 5 each. 64
// tokens, top-6 of 64, 2,048 x 1,408 in e4m3: 58-65 us (344 MB at 5.3-5.9 TB/s)
// and 35-36 (172 MB at 4.7-4.9).
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

#include <type_traits>

namespace ds {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Operands of one matrix instruction (16 x 16 outputs, 32 deep): 8 values per lane.
template <typename X> struct Frag;
template <> struct Frag<bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x4 mma(type a, type b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Frag<fp16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x4 mma(type a, type b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Eight e4m3 values as X (exact: both 16-bit types hold every one of them).
template <typename X>
__device__ __forceinline__ typename Frag<X>::type widen8(uint32_t lo, uint32_t hi)
{
    union {
        typename Frag<X>::type v;
        uint32_t u[4];
    } r;
    if constexpr (sizeof(X) == 2 && __is_same(X, bf16)) {
        r.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
        r.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
        r.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
        r.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    } else {
        r.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
        r.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
        r.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
        r.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    }
    return r.v;
}

// ---------------------------------------------------------------------------
// One wave multiplies RT row tiles of 16 rows by TT blocks of 16 tokens. It
// takes the weights in stages of 8 KiB: 16 * RT rows by kSegs segments of 16
// bytes (RT 4: 128 bytes of each of 64 rows; RT 2: 256 bytes of each of 32).
//
// In both operands lane l holds row (A) or token (B) l % 16. With s = 4 j +
// l / 16 the segment that lane l reads at its j-th read of a stage, the lane's
// values are those at depths s * kSegVals .. + kSegVals - 1 of the stage, one
// fragment of 8 (16-bit weights) or two (8-bit). Both operands use this order,
// so the products pair up.
// ---------------------------------------------------------------------------
constexpr int kStageBytes = 8192;
constexpr int kRing = 2;  // stages of a wave in LDS
constexpr int kDmaOps = kStageBytes / (kWave * kVecBytes);

template <typename W, int RT> struct Stage {
    static constexpr int kRows = 16 * RT;
    static constexpr int kSegs = kStageBytes / (kRows * kVecBytes);  // per row: 8 or 16
    static constexpr int kSegVals = kVecBytes / (int)sizeof(W);
    static constexpr int kDepth = kSegs * kSegVals;
    static constexpr int kReads = kSegs / 4;        // per tile and lane
    static constexpr int kFrags = kSegVals / 8;     // per read
};

template <typename W, int RT> struct ARegs {
    u32x4 v[RT][Stage<W, RT>::kReads];
};
template <typename W, int RT, int TT> struct BRegs {
    u32x4 v[TT][Stage<W, RT>::kReads][Stage<W, RT>::kFrags];
};

template <typename X, typename W>
__device__ __forceinline__ typename Frag<X>::type a_fragment(const u32x4& v, int f)
{
    if constexpr (sizeof(W) == 1)
        return widen8<X>(v[f * 2], v[f * 2 + 1]);
    else
        return __builtin_bit_cast(typename Frag<X>::type, v);
}

// This lane's values of the token blocks; `valid`: segments of the stage that
// lie below the end of the depth (the others are 0).
template <typename X, typename W, int RT, int TT>
__device__ __forceinline__ void load_b(const X* const (&tok)[TT], int64_t depth0, int lane, BRegs<W, RT, TT>& b)
{
    using S = Stage<W, RT>;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < S::kReads; ++j)
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f)
                b.v[t][j][f] = *reinterpret_cast<const typename Vec16<X>::type*>(
                    tok[t] + depth0 + (4 * j + lane / 16) * S::kSegVals + f * 8);
}

// The same at the end of the depth, for depths of whole segments: the first
// `segs` segments of the stage are there, the others are 0.
template <typename X, typename W, int RT, int TT>
__device__ __forceinline__ void load_b_segs(const X* const (&tok)[TT], int64_t depth0, int segs, int lane,
                                            BRegs<W, RT, TT>& b)
{
    using S = Stage<W, RT>;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < S::kReads; ++j) {
            const int s = 4 * j + lane / 16;
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f) {
                const u32x4 v = *reinterpret_cast<const typename Vec16<X>::type*>(
                    tok[t] + depth0 + (s < segs ? s : 0) * S::kSegVals + f * 8);
                b.v[t][j][f] = s < segs ? v : u32x4{0u, 0u, 0u, 0u};
            }
        }
}

// The same for any depth.
template <typename X, typename W, int RT, int TT>
__device__ __forceinline__ void load_b_end(const X* const (&tok)[TT], int64_t depth0, int64_t depth, int lane,
                                           BRegs<W, RT, TT>& b)
{
    using S = Stage<W, RT>;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < S::kReads; ++j)
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f)
                b.v[t][j][f] = load_end<X>(tok[t], depth0 + (4 * j + lane / 16) * S::kSegVals + f * 8, depth);
}

// Scales of a wave's tiles for 8-bit weights, by block of 128 of the depth.
// Tiles that begin at multiples of 16 rows lie inside one block of 128 rows
// and have one factor (UNIFORM); else each of a lane's four rows has its own.
template <int RT, bool UNIFORM> struct Scales {
    const float* base;                  // of the expert
    int64_t row[RT][UNIFORM ? 1 : 4];   // of the depth's first block
};
template <typename W, int RT, bool UNIFORM> struct ScaleRegs {
    static constexpr int kBlocks = sizeof(W) == 1 ? Stage<W, RT>::kReads / 2 : 0;  // blocks of 128 in a stage
    float v[kBlocks ? kBlocks : 1][RT][UNIFORM ? 1 : 4];
};

// The factors of the stage whose first block of 128 is blk0. last_blk: the
// depth's last block (the last stage may lack its second).
template <typename W, int RT, bool UNIFORM>
__device__ __forceinline__ void load_scales(const Scales<RT, UNIFORM>& sc, int blk0, int last_blk,
                                            ScaleRegs<W, RT, UNIFORM>& s)
{
#pragma unroll
    for (int k = 0; k < ScaleRegs<W, RT, UNIFORM>::kBlocks; ++k) {
        const int blk = blk0 + k < last_blk ? blk0 + k : last_blk;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < (UNIFORM ? 1 : 4); ++i) s.v[k][r][i] = sc.base[sc.row[r][i] + blk];
    }
}

// acc += the products of one stage.
template <typename X, typename W, int RT, int TT, bool UNIFORM>
__device__ __forceinline__ void multiply(const ARegs<W, RT>& a, const BRegs<W, RT, TT>& b,
                                         const ScaleRegs<W, RT, UNIFORM>& sc, f32x4 (&acc)[RT][TT])
{
    using S = Stage<W, RT>;
    constexpr int kPerBlock = sizeof(W) == 1 ? 2 : S::kReads;  // reads per block of 128 (8-bit)
#pragma unroll
    for (int j0 = 0; j0 < S::kReads; j0 += kPerBlock) {
        f32x4 sum[RT][TT];
        if constexpr (sizeof(W) == 1) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) sum[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int j = j0; j < j0 + kPerBlock; ++j)
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const typename Frag<X>::type af = a_fragment<X, W>(a.v[r][j], f);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const typename Frag<X>::type bf = __builtin_bit_cast(typename Frag<X>::type, b.v[t][j][f]);
                        if constexpr (sizeof(W) == 1)
                            sum[r][t] = Frag<X>::mma(af, bf, sum[r][t]);
                        else
                            acc[r][t] = Frag<X>::mma(af, bf, acc[r][t]);
                    }
                }
        if constexpr (sizeof(W) == 1) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                f32x4 s;
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = sc.v[j0 / kPerBlock][r][UNIFORM ? 0 : i];
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[r][t] += s * sum[r][t];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Weights through LDS, for rows that start on 16-byte boundaries. Each wave
// owns a ring of two stages, filled by loads that write LDS directly: no
// registers are held by data in flight (16 KiB a wave, 128 KiB a CU), and the
// lanes of a load take whole 128-byte lines, eight lanes to a line, which the
// operand layout (16 rows side by side) does not give. Non-temporal: a weight
// is read once. Row r keeps its segments in the order c ^ (r % 8), so that
// eight rows' equal segments, which are read together, lie in different banks.
//
// Waves begin at different stages of their rows (`turn`) and wrap round: rows
// that are 2^k bytes apart would otherwise all be read at the same offset, in
// the same memory channels. Streaming 1.6 GB of 4 KiB rows on MI355X: 5.0 TB/s
// from a common start, 6.25 with the turn, 6.9 with whole lines and
// non-temporal loads (register loads in operand order stay at 5.9-6.25).
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ void wait_dma(int newer_ops_8)
{
    if (newer_ops_8)
        asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Reads this lane's segments of a stage. The reads and the wait for them are
// one block, so the compiler, which does not know when the stage was filled,
// neither adds waits of its own for the ring nor moves a use before the data.
template <typename W>
__device__ __forceinline__ void read_stage(uint32_t at, ARegs<W, 4>& a)
{
    const uint32_t at1 = at ^ 64u;  // segment s + 4 of the same row
    asm volatile(
        "ds_read_b128 %0, %8\n\t"
        "ds_read_b128 %1, %9\n\t"
        "ds_read_b128 %2, %8 offset:2048\n\t"
        "ds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %8 offset:4096\n\t"
        "ds_read_b128 %5, %9 offset:4096\n\t"
        "ds_read_b128 %6, %8 offset:6144\n\t"
        "ds_read_b128 %7, %9 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a.v[0][0]), "=&v"(a.v[0][1]), "=&v"(a.v[1][0]), "=&v"(a.v[1][1]), "=&v"(a.v[2][0]),
          "=&v"(a.v[2][1]), "=&v"(a.v[3][0]), "=&v"(a.v[3][1])
        : "v"(at), "v"(at1)
        : "memory");
}
template <typename W>
__device__ __forceinline__ void read_stage(uint32_t at, ARegs<W, 2>& a)
{
    const uint32_t at1 = at ^ 64u;
    asm volatile(
        "ds_read_b128 %0, %8\n\t"
        "ds_read_b128 %1, %9\n\t"
        "ds_read_b128 %2, %8 offset:128\n\t"
        "ds_read_b128 %3, %9 offset:128\n\t"
        "ds_read_b128 %4, %8 offset:4096\n\t"
        "ds_read_b128 %5, %9 offset:4096\n\t"
        "ds_read_b128 %6, %8 offset:4224\n\t"
        "ds_read_b128 %7, %9 offset:4224\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a.v[0][0]), "=&v"(a.v[0][1]), "=&v"(a.v[0][2]), "=&v"(a.v[0][3]), "=&v"(a.v[1][0]),
          "=&v"(a.v[1][1]), "=&v"(a.v[1][2]), "=&v"(a.v[1][3])
        : "v"(at), "v"(at1)
        : "memory");
}

template <typename X, typename W, int RT, int TT>
struct LdsProduct {
    using S = Stage<W, RT>;
    const char* src[kDmaOps];  // this lane's 16 bytes of each load, at the start of the depth
    const X* const (&tok)[TT];
    const Scales<RT, true>& sc;
    lds_char* ring;
    uint32_t read_at;
    int lane, last_blk;
    int seg[kDmaOps];  // segment of its row that this lane loads (each load: 64 / kSegs rows)

    __device__ __forceinline__ LdsProduct(const W* const (&tile)[RT], const int (&last)[RT], int64_t depth,
                                          const X* const (&tok_)[TT], const Scales<RT, true>& sc_, lds_char* ring_, int lane_)
        : tok(tok_), sc(sc_), ring(ring_), lane(lane_), last_blk((int)((depth - 1) / 128))
    {
        const int c = lane % S::kSegs;
#pragma unroll
        for (int i = 0; i < kDmaOps; ++i) {
            const int row = i * (kWave / S::kSegs) + lane / S::kSegs;  // of the stage's kRows
            const int r = row % 16 < last[i * (kWave / S::kSegs) / 16] ? row % 16 : last[i * (kWave / S::kSegs) / 16];
            seg[i] = c ^ (row % 8);
            src[i] = reinterpret_cast<const char*>(tile[i * (kWave / S::kSegs) / 16] + r * depth) + seg[i] * kVecBytes;
        }
        const int r = lane % 16, s = lane / 16;
        read_at = (uint32_t)(uintptr_t)ring + (uint32_t)(r * S::kSegs + (s ^ (r % 8))) * kVecBytes;
    }

    // Factors and token values come a stage ahead too: a wait for them where
    // they are used made the 8-bit products a fifth slower.
    __device__ __forceinline__ void issue(int slot, int stage, BRegs<W, RT, TT>& b, ScaleRegs<W, RT, true>& s)
    {
        load_scales<W, RT, true>(sc, stage * (S::kDepth / 64) / 2, last_blk, s);
        load_b<X, W, RT, TT>(tok, (int64_t)stage * S::kDepth, lane, b);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kDmaOps; ++i)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) uint32_t*)(src[i] + (int64_t)stage * (S::kSegs * kVecBytes)),
                (__attribute__((address_space(3))) uint32_t*)(ring + slot * kStageBytes + i * (kWave * kVecBytes)), 16,
                0, 2);
        __builtin_amdgcn_sched_barrier(0);
    }

    // At the end of the depth only `segs` segments of a row are there: the lanes of the others load the first.
    __device__ __forceinline__ void issue_tail(int stage, int segs, BRegs<W, RT, TT>& b, ScaleRegs<W, RT, true>& s)
    {
        load_scales<W, RT, true>(sc, stage * (S::kDepth / 64) / 2, last_blk, s);
        load_b_segs<X, W, RT, TT>(tok, (int64_t)stage * S::kDepth, segs, lane, b);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kDmaOps; ++i) {
            const char* p = src[i] + (int64_t)stage * (S::kSegs * kVecBytes);
            if (seg[i] >= segs) p -= seg[i] * kVecBytes;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) uint32_t*)p,
                (__attribute__((address_space(3))) uint32_t*)(ring + i * (kWave * kVecBytes)), 16, 0, 2);
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    // newer: whether one more stage has been issued after this one. At most
    // the loads of that stage may be outstanding; loads of token values are
    // older than it, or make the wait stricter than it has to be.
    __device__ __forceinline__ void use(int slot, int newer, const BRegs<W, RT, TT>& b,
                                        const ScaleRegs<W, RT, true>& s, f32x4 (&acc)[RT][TT], int segs = S::kSegs)
    {
        ARegs<W, RT> a;
        wait_dma(newer);
        read_stage<W>(read_at + (uint32_t)slot * kStageBytes, a);
        __builtin_amdgcn_sched_barrier(0);
        if (segs < S::kSegs) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < S::kReads; ++j)
                    if (4 * j + lane / 16 >= segs) a.v[r][j] = u32x4{0u, 0u, 0u, 0u};
        }
        multiply<X, W, RT, TT>(a, b, s, acc);
    }

    // Stages [s0, s1) whole, and `segs` segments of stage s1 (0: none).
    __device__ __forceinline__ void run(int s0, int s1, int segs, uint32_t turn, f32x4 (&acc)[RT][TT])
    {
        BRegs<W, RT, TT> b0, b1;
        ScaleRegs<W, RT, true> c0, c1;
        const int count = s1 - s0;
        if (count > 0) {
            int at = s0 + (int)(turn % (uint32_t)count);
            const auto next = [&](int s) { return s + 1 < s1 ? s + 1 : s0; };
            issue(0, at, b0, c0);
            int j = 0;
            for (; j + 2 < count; j += 2) {
                const int a1 = next(at), a2 = next(a1);
                issue(1, a1, b1, c1);
                use(0, 1, b0, c0, acc);
                issue(0, a2, b0, c0);
                use(1, 1, b1, c1, acc);
                at = a2;
            }
            if (j + 1 < count) {
                const int a1 = next(at);
                issue(1, a1, b1, c1);
                use(0, 1, b0, c0, acc);
                use(1, 0, b1, c1, acc);
            } else {
                use(0, 0, b0, c0, acc);
            }
        }
        if (segs > 0) {
            issue_tail(s1, segs, b0, c0);
            use(0, 0, b0, c0, acc, segs);
        }
    }
};

// Weights straight into registers, for rows at any alignment, one stage at a
// time (a stage ahead in a second set of registers was no faster).
template <typename X, typename W, int RT, int TT>
__device__ __forceinline__ void direct_product(const W* const (&tile)[RT], const int (&last)[RT], int64_t depth,
                                               const X* const (&tok)[TT], const Scales<RT, false>& sc, int64_t k0,
                                               int64_t k1, int lane, f32x4 (&acc)[RT][TT])
{
    using S = Stage<W, RT>;
    const W* row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) row[r] = tile[r] + (lane % 16 < last[r] ? lane % 16 : last[r]) * depth;
    for (int64_t k = k0; k < k1; k += S::kDepth) {
        ARegs<W, RT> a;
        BRegs<W, RT, TT> b;
        ScaleRegs<W, RT, false> s;
        const bool whole = k + S::kDepth <= depth;
        load_scales<W, RT, false>(sc, (int)(k / 128), (int)((depth - 1) / 128), s);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < S::kReads; ++j) {
                const int64_t at = k + (4 * j + lane / 16) * S::kSegVals;
                a.v[r][j] = whole ? *reinterpret_cast<const typename Vec16<W>::type*>(row[r] + at)
                                  : load_end<W>(row[r], at, depth);
            }
        if (whole)
            load_b<X, W, RT, TT>(tok, k, lane, b);
        else
            load_b_end<X, W, RT, TT>(tok, k, depth, lane, b);
        multiply<X, W, RT, TT>(a, b, s, acc);
    }
}

// ---------------------------------------------------------------------------
// Which tokens a workgroup serves. Up to 64 assignments, workgroup slot s looks
// for itself: it serves the expert that assignment s names, unless an earlier
// one names it too. Above, expert_plan_kernel groups the assignments into
// blocks of one expert and at most `chunk` assignments, and slot s is block s.
// ---------------------------------------------------------------------------
constexpr int kFindMax = kWave;
constexpr int kPlanThreads = 1024;
constexpr int kMaxAssignments = 8192;
constexpr int kMaxExperts = 8192;

// plan[s]: expert of block s (-1: none), plan[blocks + s]: its assignments (and
// kLone where the expert has no other block); list[s * chunk ..]: their indices,
// in any order: no result depends on it. Blocks of experts with more than
// kCrowded assignments come first: they take longest, and are not to be the
// last ones running (512 tokens, top-8 of 256: 489 -> 475 us; top-6 of 64, 2,048 x
// 1,408: 346 -> 325). One workgroup.
constexpr int kLone = 1 << 16;
constexpr uint32_t kCrowded = 16;

__global__ __launch_bounds__(kPlanThreads) void expert_plan_kernel(const int32_t* __restrict__ ids, int n, int experts,
                                                                   int chunk, int blocks, int32_t* __restrict__ plan,
                                                                   uint16_t* __restrict__ list)
{
    constexpr int kPer = kMaxAssignments / kPlanThreads, kEach = kMaxExperts / kPlanThreads;
    __shared__ uint32_t s_count[kMaxExperts];  // assignments, then the first block
    __shared__ uint32_t s_wave[kPlanThreads / kWave];
    int e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = threadIdx.x + j * kPlanThreads;
        e[j] = i < n ? ids[i] : -1;
        if (e[j] >= experts) e[j] = -1;
    }
    for (int i = threadIdx.x; i < experts; i += kPlanThreads) s_count[i] = 0;
    __syncthreads();
    uint32_t rank[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (e[j] >= 0) rank[j] = atomicAdd(&s_count[e[j]], 1u);
    __syncthreads();
    // thread t holds experts t * each .. + each - 1
    const int each = (experts + kPlanThreads - 1) / kPlanThreads;
    uint32_t c[kEach], own = 0;  // own: blocks, those of crowded experts in the high half
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int x = threadIdx.x * each + j;
        c[j] = j < each && x < experts ? s_count[x] : 0u;
        own += ((c[j] + chunk - 1) / chunk) << (c[j] > kCrowded ? 16 : 0);
    }
    const uint32_t incl = wave_inclusive_scan(own);
    if (lane_id() == kWave - 1) s_wave[threadIdx.x / kWave] = incl;
    __syncthreads();
    uint32_t first = incl - own, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
        if (w < (int)(threadIdx.x / kWave)) first += s_wave[w];
        total += s_wave[w];
    }
    uint32_t crowded = first >> 16, other = (total >> 16) + (first & 0xFFFFu);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int x = threadIdx.x * each + j;
        uint32_t& at = c[j] > kCrowded ? crowded : other;
        if (j < each && x < experts) s_count[x] = at;
        for (uint32_t left = c[j]; left > 0; ++at) {
            const uint32_t here = left < (uint32_t)chunk ? left : (uint32_t)chunk;
            plan[at] = x;
            plan[blocks + at] = (int32_t)here | (here == c[j] ? kLone : 0);
            left -= here;
        }
    }
    for (int b = (int)((total >> 16) + (total & 0xFFFFu)) + threadIdx.x; b < blocks; b += kPlanThreads) plan[b] = -1;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (e[j] >= 0) list[s_count[e[j]] * chunk + rank[j]] = (uint16_t)(threadIdx.x + j * kPlanThreads);
}

struct Found {
    int expert, count;  // count 0: nothing to do
    bool all;           // these are all the assignments of the expert
};

// Every wave finds the same and writes the same list.
__device__ __forceinline__ Found find_assignments(const int32_t* __restrict__ ids, int n, int experts, int slot,
                                                  uint16_t* s_list)
{
    const int lane = lane_id();
    const int32_t mine = lane < n ? ids[lane] : -1;
    const int32_t e = readlane(mine, slot);
    if (e < 0 || e >= experts) return Found{-1, 0, false};
    const uint64_t same = ballot(mine == e);
    if (__builtin_ctzll(same) < slot) return Found{-1, 0, false};
    if (mine == e)
        s_list[__builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u))] =
            (uint16_t)lane;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return Found{e, __builtin_popcountll(same), true};
}

struct ExpertArgs {
    const int32_t* ids;
    const void *x, *w, *scale;  // scale: [experts][ceil(rows / 128)][ceil(depth / 128)], or null
    void* out;
    int64_t x_stride, out_stride;  // elements between rows of x and of out
    const int32_t* plan;           // null: the workgroups look for themselves
    const uint16_t* list;
    int n, top_k, experts, blocks, slices, chunk;
    int rows, depth;   // of one expert's matrix; gate/up: rows = F (of 2 F), depth = D; down: rows = D, depth = F
};

// The sums of neighbouring columns, in both of them.
__device__ __forceinline__ f32x4 add_halves(f32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += dpp<0xB1>((float)v[i]);
    return v;
}

// A 32-bit h as its value in X and the rest in X (0 where the value is not
// finite). h is pinned to a register: its product would otherwise be rounded
// straight to 16 bits in some places and to 32 first in others, as the compiler
// sees fit, and a token's bits would depend on its column.
template <typename X>
__device__ __forceinline__ void split_h(float h, X& high, X& low)
{
    asm("" : "+v"(h));
    high = (X)h;
    const float rest = h - (float)high;
    low = (X)(rest - rest == 0.0f ? rest : 0.0f);
}

// A wave's tiles from row0 of the output's rows on. GATED: half of the tiles are
// gate rows, the others the up rows that go with them; otherwise the tiles are
// neighbouring rows.
template <typename W, int RT, bool GATED, bool UNIFORM> struct Tiles {
    static constexpr int kHalf = GATED ? RT / 2 : RT;  // tiles of neighbouring rows
    const W* tile[RT];
    int last[RT];  // row of each tile that stands for the rows past the end
    Scales<RT, UNIFORM> sc;

    __device__ __forceinline__ Tiles(const ExpertArgs& a, int expert, int row0, int lane)
    {
        const int64_t all_rows = GATED ? 2 * (int64_t)a.rows : a.rows;
        const W* w = (const W*)a.w + (int64_t)expert * all_rows * a.depth;
        const int grid_cols = (a.depth + 127) / 128, grid_rows = (int)((all_rows + 127) / 128);
        sc.base = (const float*)a.scale + (int64_t)expert * grid_rows * grid_cols;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int64_t begin = GATED ? (int64_t)(r / kHalf) * a.rows : 0;
            int64_t from = row0 + 16 * (r % kHalf);
            if (from > a.rows - 1) from = a.rows - 1;  // a whole tile past the end
            last[r] = (int)(a.rows - 1 - from < 15 ? a.rows - 1 - from : 15);
            tile[r] = w + (begin + from) * a.depth;
            if constexpr (sizeof(W) == 1) {
#pragma unroll
                for (int i = 0; i < (UNIFORM ? 1 : 4); ++i) {
                    int64_t o = begin + from;
                    if (!UNIFORM) o += lane / 16 * 4 + i < last[r] ? lane / 16 * 4 + i : last[r];
                    sc.row[r][i] = o / 128 * grid_cols;
                }
            }
        }
    }
};

// A wave's columns: assignments list[first ..], and its lane's row of x for
// each block of 16 (GATED: the token's; otherwise the assignment's h). SPLIT:
// columns 2 c and 2 c + 1 are the halves of token c. Columns past the end
// repeat the last assignment, and have assign -1, as the second halves have.
template <typename X, int TT, bool GATED, bool SPLIT>
__device__ __forceinline__ void find_columns(const ExpertArgs& a, const uint16_t* list, int first, int count, int lane,
                                             int (&assign)[TT], const X* (&tok)[TT])
{
#pragma unroll
    for (int b = 0; b < TT; ++b) {
        const int col = b * 16 + lane % 16, at = first + (SPLIT ? col / 2 : col);
        assign[b] = list[at < count ? at : count - 1];
        tok[b] = (const X*)a.x + (int64_t)(GATED ? assign[b] / a.top_k : assign[b]) * a.x_stride;
        if (SPLIT) tok[b] += col % 2 * (a.x_stride / 2);
        if (at >= count || (SPLIT && col % 2)) assign[b] = -1;
    }
}

// GATED: silu(gate) * up, rows of its high halves, then its low ones;
// otherwise the 32-bit sums. Lane l holds output rows (l / 16) * 4 .. + 3 of
// each tile for token l % 16 of each block.
template <typename X, int RT, int TT, bool GATED, bool SPLIT>
__device__ __forceinline__ void write_results(const ExpertArgs& a, const int (&assign)[TT], int row0, int lane,
                                              f32x4 (&acc)[RT][TT])
{
    constexpr int kHalf = GATED ? RT / 2 : RT;
    if (row0 >= a.rows) return;
    if constexpr (SPLIT) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int b = 0; b < TT; ++b) acc[r][b] = add_halves(acc[r][b]);
    }
    const int r0 = row0 + lane / 16 * 4;
#pragma unroll
    for (int b = 0; b < TT; ++b) {
        if (assign[b] < 0) continue;
        if constexpr (GATED) {
            X* out = (X*)a.out + (int64_t)assign[b] * a.out_stride;
#pragma unroll
            for (int t = 0; t < kHalf; ++t) {
                X h[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float g = acc[t][b][i], u = acc[kHalf + t][b][i];
                    split_h<X>(g / (1.0f + expf(-g)) * u, h[0][i], h[1][i]);
                }
                const int64_t o = r0 + 16 * t, half = a.out_stride / 2;  // o: a multiple of 4; a half is whole vectors
                if (o < half) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint64_t v;
                        __builtin_memcpy(&v, h[p], sizeof(v));
                        *reinterpret_cast<uint64_t*>(out + p * half + o) = v;
                    }
                }
            }
        } else {
            float* out = (float*)a.out + (int64_t)assign[b] * a.out_stride;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int o = r0 + 16 * r;
                if (o < a.out_stride) *reinterpret_cast<f32x4*>(out + o) = acc[r][b];
            }
        }
    }
}

// Where the products of a tile set begin in the depth (taken modulo its
// stages): not all in the same memory channels, and the same for every token of
// the expert, whichever workgroup it falls to.
__device__ __forceinline__ uint32_t first_stage(const ExpertArgs& a, int expert, int group)
{
    return ((uint32_t)expert * (uint32_t)(a.slices * kWaves) + (uint32_t)group) * 5u;
}

template <int RT, int TT>
__device__ __forceinline__ void clear_sums(f32x4 (&acc)[RT][TT])
{
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < TT; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// The products of a wave. PARTS waves share the tiles, each with a part of the
// depth (PARTS 1: every wave has its own tiles).
template <typename X, typename W, int RT, int TT, bool GATED, bool SPLIT, int PARTS, bool LDS>
__device__ __forceinline__ void expert_block(const ExpertArgs& a, int expert, const uint16_t* list, int first,
                                             int count, int slice, char* s_mem)
{
    using S = Stage<W, RT>;
    const int lane = lane_id(), wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int part = PARTS > 1 ? wave : 0, group = PARTS > 1 ? slice : slice * kWaves + wave;
    const int row0 = group * (16 * (GATED ? RT / 2 : RT));
    f32x4 acc[RT][TT];
    clear_sums(acc);
    int assign[TT];
    const X* tok[TT];
    find_columns<X, TT, GATED, SPLIT>(a, list, first, count, lane, assign, tok);
    // the part of the depth, in whole stages
    const int stages = (a.depth + S::kDepth - 1) / S::kDepth, each = (stages + PARTS - 1) / PARTS;
    const int s0 = part * each, s1 = s0 + each < stages ? s0 + each : stages;
    if (row0 < a.rows && s0 < s1) {
        const Tiles<W, RT, GATED, LDS> t(a, expert, row0, lane);
        if constexpr (LDS) {
            const int segs = a.depth / S::kSegVals - s0 * S::kSegs;  // of the rest of the row
            const int whole = s1 < stages ? s1 : a.depth / S::kDepth;
            const uint32_t turn = first_stage(a, expert, group);
            LdsProduct<X, W, RT, TT> p(t.tile, t.last, a.depth, tok, t.sc,
                                       (lds_char*)(s_mem + wave * (kRing * kStageBytes)), lane);
            p.run(s0, whole, s1 < stages ? 0 : segs - (whole - s0) * S::kSegs, turn, acc);
        } else {
            const int64_t k1 = (int64_t)s1 * S::kDepth;
            direct_product<X, W, RT, TT>(t.tile, t.last, a.depth, tok, t.sc, (int64_t)s0 * S::kDepth,
                                         k1 < a.depth ? k1 : a.depth, lane, acc);
        }
    }
    if constexpr (PARTS > 1) {
        f32x4* s_part = reinterpret_cast<f32x4*>(s_mem);  // over the rings: every wave is past them
        __syncthreads();
        if (wave > 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int b = 0; b < TT; ++b) s_part[((wave - 1) * RT * TT + r * TT + b) * kWave + lane] = acc[r][b];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int p = 0; p < PARTS - 1; ++p)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int b = 0; b < TT; ++b) acc[r][b] += s_part[(p * RT * TT + r * TT + b) * kWave + lane];
        }
        __syncthreads();
        if (wave > 0) return;
    }
    write_results<X, RT, TT, GATED, SPLIT>(a, assign, row0, lane, acc);
}

// ---------------------------------------------------------------------------
// Many tokens of one expert: the waves of a workgroup share four tiles and
// split the tokens, 16 * TT to a wave. The stages of the weights are shared: a
// wave loads one tile of each, three stages make the ring, and a barrier per
// stage says that all tiles of it are there and that the stage that is to be
// overwritten is done with. 512 tokens, top-2 of 8, 4,096 x 2,048 in bf16: 178
// us where the experts have equal shares, 247-253 where the r-th has 1 / r of the
// first's (225 for half the tokens with 64 to a workgroup, 154 with this); the
// tokens' values, which every workgroup reads from the L2, bound it.
// ---------------------------------------------------------------------------
constexpr int kWideRing = 3;
constexpr int kWideOps = kDmaOps / kWaves;  // loads of a wave per stage

template <typename X, typename W, int TT>
struct WideProduct {
    using S = Stage<W, 4>;
    static_assert(kWideOps == 2 && S::kSegs == 8, "a wave loads one tile, eight rows at a time");
    const char* src[kWideOps];
    int seg[kWideOps];
    const X* const (&tok)[TT];
    const Scales<4, true>& sc;
    lds_char *ring, *mine;
    uint32_t read_at;
    int lane, last_blk;

    __device__ __forceinline__ WideProduct(const W* tile, int last, int64_t depth, const X* const (&tok_)[TT],
                                           const Scales<4, true>& sc_, lds_char* ring_, int lane_, int wave)
        : tok(tok_), sc(sc_), ring(ring_), mine(ring_ + wave * (kWideOps * kWave * kVecBytes)), lane(lane_),
          last_blk((int)((depth - 1) / 128))
    {
#pragma unroll
        for (int i = 0; i < kWideOps; ++i) {
            const int row = i * 8 + lane / 8, r = row < last ? row : last;
            seg[i] = lane % 8 ^ row % 8;
            src[i] = reinterpret_cast<const char*>(tile + r * depth) + seg[i] * kVecBytes;
        }
        const int r = lane % 16, s = lane / 16;
        read_at = (uint32_t)(uintptr_t)ring + (uint32_t)(r * S::kSegs + (s ^ (r % 8))) * kVecBytes;
    }

    __device__ __forceinline__ void load(int slot, int stage, int segs)
    {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kWideOps; ++i) {
            const char* p = src[i] + (int64_t)stage * (S::kSegs * kVecBytes);
            if (seg[i] >= segs) p -= seg[i] * kVecBytes;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) uint32_t*)p,
                (__attribute__((address_space(3))) uint32_t*)(mine + slot * kStageBytes + i * (kWave * kVecBytes)), 16,
                0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __forceinline__ void load_x(int stage, int segs, BRegs<W, 4, TT>& b, ScaleRegs<W, 4, true>& s)
    {
        load_scales<W, 4, true>(sc, stage * (S::kDepth / 64) / 2, last_blk, s);
        if (segs == S::kSegs)
            load_b<X, W, 4, TT>(tok, (int64_t)stage * S::kDepth, lane, b);
        else
            load_b_segs<X, W, 4, TT>(tok, (int64_t)stage * S::kDepth, segs, lane, b);
    }

    // Of this wave's loads, those of the stage after this one may be outstanding (newer).
    __device__ __forceinline__ void arrive(bool newer)
    {
        __builtin_amdgcn_sched_barrier(0);
        if (newer)
            asm volatile("s_waitcnt vmcnt(2)" ::: "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __forceinline__ void use(int slot, const BRegs<W, 4, TT>& b, const ScaleRegs<W, 4, true>& s,
                                        f32x4 (&acc)[4][TT], int segs)
    {
        ARegs<W, 4> a;
        read_stage<W>(read_at + (uint32_t)slot * kStageBytes, a);
        if (segs < S::kSegs) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < S::kReads; ++j)
                    if (4 * j + lane / 16 >= segs) a.v[r][j] = u32x4{0u, 0u, 0u, 0u};
        }
        multiply<X, W, 4, TT>(a, b, s, acc);
    }

    // The whole depth, `segs_all` segments. Every wave of the workgroup runs
    // this with the same stages. (All from the start: tokens' values, read again
    // by every workgroup, bound this, and are shared in the cache that way.)
    __device__ __forceinline__ void run(int segs_all, f32x4 (&acc)[4][TT])
    {
        const int stages = (segs_all + S::kSegs - 1) / S::kSegs;
        const auto segs = [&](int s) { return s + 1 < stages ? S::kSegs : segs_all - s * S::kSegs; };
        BRegs<W, 4, TT> b[2];
        ScaleRegs<W, 4, true> c[2];
        load(0, 0, segs(0));
        load_x(0, segs(0), b[0], c[0]);
        if (stages > 1) load(1, 1, segs(1));
        int slot = 0;
        // two stages at a time, so that the register sets are known to the compiler
        const auto step = [&](int s, int which) {
            arrive(s + 1 < stages);
            if (s + 1 < stages) load_x(s + 1, segs(s + 1), b[which ^ 1], c[which ^ 1]);
            if (s + 2 < stages) load(slot >= 1 ? slot - 1 : kWideRing - 1, s + 2, segs(s + 2));
            use(slot, b[which], c[which], acc, segs(s));
            slot = slot + 1 < kWideRing ? slot + 1 : 0;
        };
        int s = 0;
        for (; s + 1 < stages; s += 2) {
            step(s, 0);
            step(s + 1, 1);
        }
        if (s < stages) step(s, 0);
        __builtin_amdgcn_s_barrier();  // the ring is free for the next tiles
        asm volatile("" ::: "memory");
    }
};

template <typename X, typename W, int TT, bool GATED, bool SPLIT>
__device__ __forceinline__ void expert_wide(const ExpertArgs& a, int expert, const uint16_t* list, int first, int count,
                                            int group, char* s_mem)
{
    const int lane = lane_id(), wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row0 = group * (16 * (GATED ? 2 : 4));
    if (row0 >= a.rows) return;  // for the whole workgroup
    f32x4 acc[4][TT];
    clear_sums(acc);
    int assign[TT];
    const X* tok[TT];
    find_columns<X, TT, GATED, SPLIT>(a, list, first + wave * (SPLIT ? 8 : 16) * TT, count, lane, assign, tok);
    const Tiles<W, 4, GATED, true> t(a, expert, row0, lane);
    const W* tile = wave == 0 ? t.tile[0] : wave == 1 ? t.tile[1] : wave == 2 ? t.tile[2] : t.tile[3];
    const int last = wave == 0 ? t.last[0] : wave == 1 ? t.last[1] : wave == 2 ? t.last[2] : t.last[3];
    WideProduct<X, W, TT> p(tile, last, a.depth, tok, t.sc, (lds_char*)s_mem, lane, wave);
    p.run(a.depth / Stage<W, 4>::kSegVals, acc);
    write_results<X, 4, TT, GATED, SPLIT>(a, assign, row0, lane, acc);
}

// Blocks of 16 tokens that a wave holds at once, as registers allow (256 at two
// waves per SIMD): 8-bit weights have a second set of sums (one per block of
// 128 of the depth) and twice the depth to a stage, RT 2 twice the depth too.
template <typename W, int RT = 4> struct MostBlocks {
    static constexpr int value = (sizeof(W) == 1 ? 2 : 4) * RT / 4;
};

// How a workgroup takes a block of tokens: every wave with tiles of its own
// over the whole depth (kStream); all waves on one tile set, each with a part of
// the depth (kParts) or of the tokens (kWide).
enum ExpertMode { kStream, kParts, kWide };

constexpr int kSplitTokens = 8;  // of an expert, at most, for h in two halves: a block of 16 columns

template <typename X, typename W, bool GATED, ExpertMode MODE, bool LDS>
__global__ __launch_bounds__(kThreads, 2) void expert_kernel(ExpertArgs a)
{
    constexpr int RT = MODE == kParts ? 2 : 4, PARTS = MODE == kParts ? kWaves : 1;
    constexpr int kMost = MostBlocks<W, RT>::value;
    constexpr int kPart = (PARTS - 1) * RT * kMost * kWave * 16;
    constexpr int kRings = MODE == kWide ? kWideRing * kStageBytes : LDS ? kWaves * kRing * kStageBytes : 0;
    __shared__ __align__(1024) char s_mem[kRings > kPart ? kRings : kPart > 0 ? kPart : 16];
    __shared__ uint16_t s_list[kFindMax];
    const int slot = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
    Found f;
    const uint16_t* list;
    if (a.plan) {
        const int e = a.plan[slot];
        if (e < 0) return;
        const int count = a.plan[a.blocks + slot];
        f = Found{e, count & (kLone - 1), (count & kLone) != 0};
        list = a.list + (int64_t)slot * a.chunk;
    } else {
        f = find_assignments(a.ids, a.n, a.experts, slot, s_list);
        if (f.count == 0) return;
        list = s_list;
    }
    // halves of h for all tokens of an expert or for none, whatever their order in the list
    const bool split = !GATED && f.all && f.count <= kSplitTokens;
    if constexpr (MODE == kWide) {
        if constexpr (!GATED) {
            if (split) return expert_wide<X, W, 1, GATED, true>(a, f.expert, list, 0, f.count, slice, s_mem);
        }
        for (int first = 0; first < f.count; first += 64 * kMost) {
            const int left = f.count - first;
            if (left > 32 * kMost)
                expert_wide<X, W, kMost, GATED, false>(a, f.expert, list, first, f.count, slice, s_mem);
            else if (kMost > 2 && left > 64)
                expert_wide<X, W, kMost / 2, GATED, false>(a, f.expert, list, first, f.count, slice, s_mem);
            else
                expert_wide<X, W, 1, GATED, false>(a, f.expert, list, first, f.count, slice, s_mem);
        }
    } else {
        int first = 0;
        const auto pass = [&](auto blocks, auto split) {
            expert_block<X, W, RT, decltype(blocks)::value, GATED, decltype(split)::value, PARTS, LDS>(
                a, f.expert, list, first, f.count, slice, s_mem);
        };
        constexpr int kMiddle = kMost > 2 ? kMost / 2 : 1;
        constexpr std::integral_constant<int, kMost> most{};
        constexpr std::integral_constant<int, kMiddle> middle{};
        if constexpr (!GATED) {
            if (split) return pass(std::integral_constant<int, 1>{}, std::true_type{});
        }
        for (; f.count - first > (kMost > 1 ? 8 * kMost : 0); first += 16 * kMost) pass(most, std::false_type{});
        if constexpr (kMost > 1) {
            const int left = f.count - first;
            if (kMost > 2 && left > 16) pass(middle, std::false_type{});
            else if (left > 0) pass(std::integral_constant<int, 1>{}, std::false_type{});
        }
    }
}

// y_t = sum over j of weights[t, j] * part[t, j], choices outside the experts
// left out. A thread sums four columns; rows of `part` are whole vectors.
template <typename X>
__global__ __launch_bounds__(kThreads) void expert_sum_kernel(const float* __restrict__ part, int64_t part_stride,
                                                              const int32_t* __restrict__ ids,
                                                              const float* __restrict__ weights, int tokens, int top_k,
                                                              int experts, int dim, X* __restrict__ y,
                                                              int64_t y_stride)
{
    const int quads = (dim + 3) / 4;
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int t = (int)(at / quads), d = (int)(at % quads) * 4;
    if (t >= tokens) return;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        f32x4 p[8];
        float w[8];
        bool live[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t i = (int64_t)t * top_k + (j0 + j < top_k ? j0 + j : top_k - 1);
            const int e = ids[i];
            live[j] = j0 + j < top_k && e >= 0 && e < experts;
            w[j] = weights[i];
            p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (live[j]) p[j] = *reinterpret_cast<const f32x4*>(part + i * part_stride + d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (live[j]) sum += w[j] * p[j];
    }
    X* out = y + t * y_stride + d;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < dim) out[i] = (X)sum[i];
}

int64_t experts_max_assignments() { return kMaxAssignments; }
int experts_max_experts() { return kMaxExperts; }

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Scratch: rows of h (two halves of 16-byte multiples), rows of parts, the plan and its list.
struct ExpertsScratch {
    int64_t h_stride, part_stride, blocks, part_at, plan_at, list_at, bytes;
    ExpertsScratch(int64_t n, int experts, int dim, int hidden, int chunk)
    {
        h_stride = 2 * (ceil_div(hidden, 8) * 8);
        part_stride = ceil_div(dim, 4) * 4;
        blocks = (experts < n ? experts : n) + n / chunk;
        part_at = ceil_div(n * h_stride * 2, 256) * 256;
        plan_at = part_at + n * part_stride * 4;
        list_at = plan_at + blocks * 2 * 4;
        bytes = list_at + blocks * chunk * 2;
    }
};

// How a call is launched.
struct ExpertsPlan {
    bool wide;        // the waves of a workgroup split an expert's tokens
    int chunk;        // assignments per block of the plan
    int64_t blocks;   // of tokens
    struct Launch {
        ExpertMode mode;
        bool lds;     // weights through LDS: every row of every expert starts on a 16-byte boundary
        int64_t slices;
    } in, out;

    ExpertsPlan(bool eight_bit, const ExpertsCall& c)
    {
        const int64_t n = c.tokens * c.top_k;
        const int wbytes = eight_bit ? 1 : 2, most = eight_bit ? MostBlocks<fp8>::value : MostBlocks<bf16>::value;
        in.lds = whole_vectors(c.w_in, c.dim, wbytes) && (!eight_bit || c.hidden % 16 == 0);
        out.lds = whole_vectors(c.w_out, c.hidden, wbytes);
        wide = in.lds && out.lds && n >= kWideTokens * c.experts;
        chunk = block_size(wide, most);
        blocks = n > kFindMax ? ExpertsScratch(n, c.experts, c.dim, c.hidden, chunk).blocks : n;
        const int64_t used = n < c.experts ? n : c.experts;  // experts at most; without a plan, other blocks are idle
        choose(in, true, c.hidden, used, eight_bit);
        choose(out, false, c.dim, used, eight_bit);
    }

    static int block_size(bool wide, int most) { return (wide ? 64 : 16) * most; }

private:
    // Assignments to an expert on average. In 16 bits: 48 (512 tokens, top-6 of 64, 2,048 x 1,408) 327 us wide and 455
    // not; 24 (256 of these) 287 and 297; 16 (512 tokens, top-8 of 256, 2,048 x 768) 567 and 473; 32 (1,024 of these)
    // 641 and 586, but 32 of few experts (128 tokens, top-2 of 8, 4,096 x 2,048) 120 and 127. In 8 bits the two meet at
    // 64 for many experts (308 and 304; 48: 268 and 250), at 16 for few (66 and 67; 32: 87 and 116). 32 is between.
    static constexpr int64_t kWideTokens = 32;

    static bool whole_vectors(const void* w, int depth, int wbytes)
    {
        return (uintptr_t)w % kVecBytes == 0 && (int64_t)depth * wbytes % kVecBytes == 0;
    }
    void choose(Launch& l, bool gated, int rows, int64_t used, bool eight)
    {
        // A wave streams four tiles of its own where that gives every CU work enough; with few experts the waves of a
        // workgroup share two tiles. 128 tokens, top-8 of 128, 2,048 x 768 (768 and 1,024 workgroups): in 16 bits 230
        // us from 512 workgroups on, 222 from 1,024; in 8 bits, where two tiles hold fewer tokens, 140 and 152.
        l.slices = ceil_div(rows, (gated ? 32 : 64) * kWaves);
        l.mode = wide ? kWide : l.lds && used * l.slices >= (eight ? 512 : 1024) ? kStream : kParts;
        if (l.mode == kWide) l.slices = ceil_div(rows, gated ? 32 : 64);
        if (l.mode == kParts) l.slices = ceil_div(rows, gated ? 16 : 32);
    }
};

int64_t experts_aux_bytes(bool eight_bit, const ExpertsCall& c)
{
    const ExpertsPlan p(eight_bit, c);
    return ExpertsScratch(c.tokens * c.top_k, c.experts, c.dim, c.hidden, p.chunk).bytes;
}

// For any alignment of the weights.
int64_t experts_most_aux_bytes(bool eight_bit, int64_t tokens, int dim, int experts, int hidden, int top_k)
{
    const int most = eight_bit ? MostBlocks<fp8>::value : MostBlocks<bf16>::value;
    const ExpertsScratch narrow(tokens * top_k, experts, dim, hidden, ExpertsPlan::block_size(false, most));
    const ExpertsScratch wide(tokens * top_k, experts, dim, hidden, ExpertsPlan::block_size(true, most));
    return narrow.bytes > wide.bytes ? narrow.bytes : wide.bytes;
}

int64_t experts_workgroups(bool eight_bit, const ExpertsCall& c)
{
    const ExpertsPlan p(eight_bit, c);
    return p.blocks * (p.in.slices > p.out.slices ? p.in.slices : p.out.slices);
}

template <typename X, typename W, bool GATED>
static hipError_t launch_expert_kernel(ExpertArgs a, const ExpertsPlan::Launch& l, hipStream_t stream)
{
    a.slices = (int)l.slices;
    const dim3 grid((unsigned)(a.blocks * l.slices)), block(kThreads);
    if (l.mode == kStream)
        expert_kernel<X, W, GATED, kStream, true><<<grid, block, 0, stream>>>(a);
    else if (l.mode == kWide)
        expert_kernel<X, W, GATED, kWide, true><<<grid, block, 0, stream>>>(a);
    else if (l.lds)
        expert_kernel<X, W, GATED, kParts, true><<<grid, block, 0, stream>>>(a);
    else
        expert_kernel<X, W, GATED, kParts, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename X, typename W>
static hipError_t experts_typed(const ExpertsCall& c, char* aux, hipStream_t stream)
{
    const int n = (int)(c.tokens * c.top_k);
    const ExpertsPlan p(sizeof(W) == 1, c);
    const ExpertsScratch s(n, c.experts, c.dim, c.hidden, p.chunk);
    char *h = aux, *part = aux + s.part_at;
    int32_t* plan = nullptr;
    uint16_t* list = nullptr;
    const int blocks = (int)p.blocks;
    if (n > kFindMax) {
        plan = reinterpret_cast<int32_t*>(aux + s.plan_at);
        list = reinterpret_cast<uint16_t*>(aux + s.list_at);
        expert_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, stream>>>(c.ids, n, c.experts, p.chunk, blocks, plan, list);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const ExpertArgs a{c.ids, c.x, c.w_in, c.w_in_scale, h, c.x_stride, s.h_stride, plan, list, n, c.top_k, c.experts,
                       blocks, 0, p.chunk, c.hidden, c.dim};
    hipError_t e = launch_expert_kernel<X, W, true>(a, p.in, stream);
    if (e != hipSuccess) return e;
    const ExpertArgs b{c.ids, h, c.w_out, c.w_out_scale, part, s.h_stride, s.part_stride, plan, list, n, c.top_k,
                       c.experts, blocks, 0, p.chunk, c.dim, c.hidden};
    e = launch_expert_kernel<X, W, false>(b, p.out, stream);
    if (e != hipSuccess) return e;
    const int64_t items = c.tokens * ceil_div(c.dim, 4);
    expert_sum_kernel<X><<<dim3((unsigned)ceil_div(items, kThreads)), dim3(kThreads), 0, stream>>>(
        (const float*)part, s.part_stride, c.ids, c.weights, (int)c.tokens, c.top_k, c.experts, c.dim, (X*)c.y,
        c.y_stride);
    return hipGetLastError();
}

hipError_t launch_moe_experts(ElemKind kind, bool eight_bit, const ExpertsCall& c, char* aux, hipStream_t stream)
{
    if (kind == kBF16)
        return eight_bit ? experts_typed<bf16, fp8>(c, aux, stream) : experts_typed<bf16, bf16>(c, aux, stream);
    if (kind == kF16)
        return eight_bit ? experts_typed<fp16, fp8>(c, aux, stream) : experts_typed<fp16, fp16>(c, aux, stream);
    return hipErrorInvalidValue;
}

}  // namespace ds
