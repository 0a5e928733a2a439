// Linear attention with a decay for each head: launch interface, and what its kernels share.
//
// Per (batch b, head h), state S in R^{d_v x d_k}, log decay g_t:
//
//     S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = S_t q_t
//
// Chunks of C tokens, G the inclusive prefix sums of g in the chunk, S the state before it:
//
//     O  = e^G (Q S^T) + P V,      P[s][t] = e^{G_s - G_t} (Q K^T)[s][t] for t <= s, else 0
//     S' = e^{G_C} S + sum_t e^{G_C - G_t} v_t k_t^T
//
// The gradients have the same form with the roles changed (dq with the state as it is, dk and
// dv backwards in time), so every kernel here is a walk over chunks that holds one or two
// states in registers:
//
//   A wave owns 16 columns of the state, each for every contraction index ("rows"): for o the
//   columns are value indices and the rows key indices.  Tile 2u + h of its accumulators holds
//   in lane (g = l / 16, c = l % 16), element i, column c and row 32 u + 8 g + 4 h' + i, h' = h for
//   even g and 1 - h for odd g.  That is at once what the 16x16x32 products take as operand, with
//   eight consecutive rows a lane, so the other operand is one 16-byte LDS read, and the state
//   never leaves the registers.  Outputs are formed transposed: a lane gets four consecutive
//   columns of one token.
//
// Precision.  States, sums and statistics are fp32.  A bf16 product rounds P and the state it
// reads to bf16 once each.  What enters a state (v_t e^{G_C - G_t}) is split into bf16 addends, a
// product each: three (24 bits, all of an fp32) where S_T, dS0 or dg, which are fp32, come of the
// state; two (16 bits) where only element outputs do, which a third rounding to 8 bits would put
// 1.7 instead of 1.4 roundings off.  Prefix sums of g are taken in 64 bits and kept as the sum of two fp32 numbers:
// e^{G_s - G_t} of near tokens behind strong decays would lose what the difference cancels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qd_device.h"

namespace qd {

enum LinDecay { kNoDecay = 0, kTokenDecay = 1, kHeadDecay = 2 };

// A chunk's sums of a and b and its decay, for the chain of qd_linattn_bwd.hip.  size_a, size_b: means
// of |a| and |b| over 64 tokens, which stay within fp32 where squares, and sums, would not.
struct LinSums {
    float a, b, size_a, size_b, all;
    float c;                         // by the chain, where it is a launch of its own
    __device__ __forceinline__ double weight() const { return static_cast<double>(size_a) * size_a + static_cast<double>(size_b) * size_b; }
};

struct LinArgs {
    const void *q, *k, *v;           // [B][T][H][DK], [B][T][H][DK], [B][T][H][DV]
    const float *g;                  // null, [B][T][H] or [H], by `decay`
    const float *S0;                 // [B][H][DV][DK] or null
    const int *lens;                 // [B] or null
    void *o;                         // [B][T][H][DV]
    float *S_T;                      // [B][H][DV][DK] or null
    int B, T, H, DK, DV;
    int decay;
    // backward only
    const void *d_o;                 // [B][T][H][DV]
    const float *dS_T;               // [B][H][DV][DK] or null
    void *dq, *dk, *dv;
    float *dg;                       // like g, or null
    float *dS0;                      // or null
    // schedule, filled in by the launch.  The time axis is cut into `segs` segments of seg_chunks
    // chunks, walked side by side.  Their first states come of `subs` shorter pieces a segment,
    // sub_chunks each, walked from zero by a launch before: fwd of every segment but the last, rev
    // of every one but the first
    int segs, seg_chunks, subs, sub_chunks;
    float *fwd, *rev;                // [B H][(segs - 1) subs][DV][DK]
    float *fac;                      // [2][B H][(segs - 1) subs]: the root of a piece's decay
    float *entry;                    // [B H][DV][DK]: S0, where S_T overwrites it; or null
    LinSums *sums;                   // [B H][chunks]
    float *tok;                      // [3][B H][T]: terms of dg
    float *edge;                     // [B H][segs + 1][8]: <S, R> at the segments' borders, by wave
    double *chain;                   // [B H][chunks][2]: c before what is missed is taken back, and its share of that
    float *head;                     // [B][chunks][H]: sums of dg over tokens
};

bool lin_supported(int dtype, int dk, int dv);
enum LinCall { kLinStep, kLinFwd, kLinBwd };
bool lin_fits(int dtype, int B, int T, int H, LinCall call);
size_t lin_fwd_workspace(int dtype, int B, int T, int H, int dk, int dv);
hipError_t launch_lin_fwd(int dtype, LinArgs a, void *ws, hipStream_t stream);
hipError_t launch_lin_step(int dtype, const LinArgs &a, float *S, hipStream_t stream);   // T = 1
size_t lin_bwd_workspace(int dtype, int B, int T, int H, int dk, int dv, bool dg);
hipError_t launch_lin_bwd(int dtype, LinArgs a, void *ws, hipStream_t stream);
// Workspace of the states at the segments' borders, and the launches that find them (exact: fp32
// results come of the states, not only element outputs).
size_t lin_states_floats(const LinArgs &a, int directions);
float *lin_states_place(LinArgs &a, float *ws, int directions);      // the workspace behind them
hipError_t launch_lin_states(int dtype, const LinArgs &a, bool fwd, bool rev, bool exact, hipStream_t stream);
// The segments for `units` walks (workgroups, one a compute unit) of a chunk sequence; `heads` of
// them times `directions` states
void lin_plan(int dtype, LinArgs &a, long long units, int directions, double state_cost);
hipError_t launch_lin_copy(float *to, const float *from, size_t n, hipStream_t stream);  // from null: zeros

// Tokens of a chunk.  fp32 rows of 64 would not fit the LDS twice.
template <class P>
constexpr int kLinChunk = P::kBytes == 2 ? 64 : 32;
inline int lin_chunk(int dtype) { return dtype == 1 ? 64 : 32; }

constexpr double kLinLog2e = 1.4426950408889634;

typedef __attribute__((ext_vector_type(4))) unsigned lin_u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned lin_u32x2;

// raw buffer (stride 0): reads at offsets >= bytes give 0, writes there are dropped.  base and
// bytes are the same in every lane; said so, or each access becomes a loop over the lanes' values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lin_rsrc(const void *base, int bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(static_cast<uint64_t>(hi) << 32 | lo), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

__device__ __forceinline__ float lin_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
// e^x for a decay.  What the product with log2 e rounds away is put back to first order; below
// -1000 (-inf too) the result is zero either way.
__device__ __forceinline__ float lin_exp(float x) {
    x = x < -1000.f ? -1000.f : x;
    const float p = x * 1.44269504088896341f;
    const float q = fmaf(x, 1.925963033500e-8f, fmaf(x, 1.44269504088896341f, -p));
    return lin_exp2(p) * fmaf(q, 0.69314718055994531f, 1.f);
}

// ---------------------------------------------------------------- rows of a chunk
// A matrix of ROWS x COLS elements in LDS, and the ways it is read as an operand:
//   oct:  row r0 + l % 16, eight columns 32 u + 8 g + .., g = l / 16 (contraction over columns)
//   down: rows 32 u + 8 g + .. of column c0 + l % 16 (contraction over rows)
//   across: the same rows of the columns that a state's tile has as its rows
// Each gives the eight as two halves, in the order of their index for even g and the other way
// round for odd g; products pair what has the same place, so any two of them agree.
//
// bf16: a 16 x 32 block is 64 slots of 16 bytes; columns 8 g .. 8 g + 7 of row r sit in slot
// 16 g + (r ^ 2 g), their halves swapped for odd g.  A cycle serves 128 bytes: eight lanes of an
// oct read one g and eight rows; the sixteen lanes of a transposing read take four rows of four
// g, whose slots and halves all differ; the 32-column strips are an odd number of slots long, so
// what is written together, sixteen pieces of a row, half by half, differs too.
// fp32: rows padded by 16 bytes.
//
// An address is a part that depends on the lane alone (LinLane) and one that the compiler knows.
__device__ __forceinline__ int lin_half(int e, int lane) { return 4 * (e ^ ((lane >> 4) & 1)); }

struct LinLane {
    int lane, oct, across, down, four;
    __device__ __forceinline__ LinLane(int l) : lane(l) {
        const int g = l >> 4, r = l & 15, i = r >> 2, p = r & 3;
        const int row = 8 * (g & 1) + 4 * (g & 1) + i, strip = (g >> 1) << 9;
        oct = 8 * (16 * g + (r ^ (2 * g)));
        // LDS transpose reads: lane 4i + p of a group of 16 reads row i, four columns at chunk p;
        // lane 4p + q receives element q of chunk p of the rows 0..3
        across = strip + 8 * (16 * p + (row ^ (2 * p)));
        down = strip + 8 * (16 * (p >> 1) + (row ^ (2 * (p >> 1)))) + 4 * ((p ^ (p >> 1)) & 1);
        four = 8 * (16 * (g >> 1) + (r ^ (2 * (g >> 1)))) + 4 * ((g ^ (g >> 1)) & 1);
    }
};

template <class P, int ROWS, int COLS>
struct LinTile {
    using R = typename P::R;
    using F = typename P::F;
    static constexpr bool kSwz = P::kBytes == 2;
    static constexpr int kStrip = ROWS / 16 * 512 + 8, kPitch = COLS + 4;
    static constexpr int kElems = kSwz ? COLS / 32 * kStrip : ROWS * kPitch;
    R m[kElems];

    // four elements of row 16 i + l % 16 from column 16 t + 4 (l / 16) on
    __device__ __forceinline__ R *four(int i, int t, const LinLane &l) {
        if constexpr (kSwz) return m + (t >> 1) * kStrip + 512 * i + 256 * (t & 1) + (l.four ^ (32 * (t & 1)));
        else return m + (16 * i + (l.lane & 15)) * kPitch + 16 * t + 4 * (l.lane >> 4);
    }
    // halves lo, hi of the eight columns 32 u + 8 g + .. of row 16 i + l % 16
    __device__ __forceinline__ void oct(int i, int u, const LinLane &l, F &lo, F &hi) {
        if constexpr (kSwz) {
            P::ld8(m + u * kStrip + 512 * i + l.oct, lo, hi);
        } else {
            const R *p = m + (16 * i + (l.lane & 15)) * kPitch + 32 * u + 8 * (l.lane >> 4);
            lo = P::ld4(p + lin_half(0, l.lane));
            hi = P::ld4(p + lin_half(1, l.lane));
        }
    }
    // half e of the eight rows 32 u + 8 g + .. of column 16 t + l % 16
    __device__ __forceinline__ F down(int u, int e, int t, const LinLane &l) {
        if constexpr (kSwz) return transposed(m + (t >> 1) * kStrip + 1024 * u + 256 * (t & 1) + (l.down ^ (32 * ((e ^ t) & 1))));
        else return P::ld4_strided(m + f32_row(u, e, l) * kPitch + 16 * t + (l.lane & 15), kPitch);
    }
    // the same of the column that is row l % 16 of a state's tile t
    __device__ __forceinline__ F across(int u, int e, int t, const LinLane &l) {
        if constexpr (kSwz) {
            return transposed(m + (t >> 1) * kStrip + 1024 * u + 4 * (t & 1) + (l.across ^ (32 * e)));
        } else {
            const int p = (l.lane & 15) >> 2;
            return P::ld4_strided(m + f32_row(u, e, l) * kPitch + 32 * (t >> 1) + 8 * p + 4 * ((t ^ p) & 1) + (l.lane & 3), kPitch);
        }
    }

private:
    __device__ __forceinline__ static int f32_row(int u, int e, const LinLane &l) { return 32 * u + 8 * (l.lane >> 4) + lin_half(e, l.lane); }
    __device__ __forceinline__ static F transposed(R *p) {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        return __builtin_bit_cast(F, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
    }
};

// How NT threads share the 16-byte pieces of C rows of COLS elements
template <class P, int C, int COLS, int NT>
struct LinPieces {
    using T = LinTile<P, C, COLS>;
    static constexpr int kPer = COLS * P::kBytes / 16, N = C * kPer / NT, kRows = NT / kPer;
    static_assert(C * kPer % NT == 0 && N >= 1 && (!T::kSwz || kRows % 16 == 0), "pieces must divide over the threads");
    int row, c;
    __device__ __forceinline__ LinPieces(int tid) : row(tid / kPer), c(tid % kPer) {}
    __device__ __forceinline__ int from(int j, int stride) const { return (row + j * kRows) * stride + 16 * c; }
    __device__ __forceinline__ typename P::R *at(T &t, int j, int half) const {
        if constexpr (T::kSwz) {
            const int g = c & 3;
            return t.m + (c >> 2) * T::kStrip + (row >> 4) * 512 + 8 * (16 * g + ((row & 15) ^ (2 * g))) + 4 * ((half ^ c) & 1) +
                   j * (kRows / 16) * 512;
        } else {
            return t.m + (row + j * kRows) * T::kPitch + 4 * c;
        }
    }
    __device__ __forceinline__ void put(T &t, int j, lin_u32x4 v) const {
        if constexpr (T::kSwz) {
            *reinterpret_cast<lin_u32x2 *>(at(t, j, 0)) = __builtin_shufflevector(v, v, 0, 1);
            *reinterpret_cast<lin_u32x2 *>(at(t, j, 1)) = __builtin_shufflevector(v, v, 2, 3);
        } else {
            *reinterpret_cast<lin_u32x4 *>(at(t, j, 0)) = v;
        }
    }
    __device__ __forceinline__ lin_u32x4 get(T &t, int j) const {
        if constexpr (T::kSwz)
            return __builtin_shufflevector(*reinterpret_cast<const lin_u32x2 *>(at(t, j, 0)),
                                           *reinterpret_cast<const lin_u32x2 *>(at(t, j, 1)), 0, 1, 2, 3);
        else
            return *reinterpret_cast<const lin_u32x4 *>(at(t, j, 0));
    }
};

// Rows of a tile to a buffer (what lies past its end is dropped), over NT threads
template <class P, int C, int COLS, int NT>
__device__ __forceinline__ void lin_store(LinTile<P, C, COLS> &from, __amdgpu_buffer_rsrc_t rs, int stride, int tid) {
    const LinPieces<P, C, COLS, NT> at(tid);
#pragma unroll
    for (int j = 0; j < at.N; ++j) __builtin_amdgcn_raw_buffer_store_b128(at.get(from, j), rs, at.from(j, stride), 0, 0);
}

// C rows of COLS elements (rows `stride` bytes apart) on their way to a tile, over NT threads
template <class P, int C, int COLS, int NT>
struct LinRows {
    using Pieces = LinPieces<P, C, COLS, NT>;
    lin_u32x4 r[Pieces::N];

    __device__ __forceinline__ void load(const void *base, int rows, int stride, int tid) {
        const Pieces at(tid);
        const __amdgpu_buffer_rsrc_t rs = lin_rsrc(base, rows > 0 ? (rows - 1) * stride + COLS * P::kBytes : 0);
#pragma unroll
        for (int j = 0; j < at.N; ++j) r[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, at.from(j, stride), 0, 0);
    }
    __device__ __forceinline__ void put(LinTile<P, C, COLS> &to, int tid) const {
        const Pieces at(tid);
#pragma unroll
        for (int j = 0; j < at.N; ++j) at.put(to, j, r[j]);
    }
};

// ---------------------------------------------------------------- decays of a chunk
template <int C>
struct LinGates {
    float before[C];                 // e^{G_t}: from the chunk's start to behind token t
    float after[C];                  // e^{G_C - G_t}
    float hi[C], lo[C];              // G in powers of two, as a sum
    float all[4];                    // e^{G_C}
};

// log decay of lane's token of the chunk at t0 with `live` tokens, 0 past them.  A buffer load like
// the rows', so that a wave always has the same number of loads on their way.
__device__ __forceinline__ float lin_gate(const LinArgs &a, int b, int h, int t0, int live, int lane) {
    const bool token = a.decay == kTokenDecay;
    const float *base = token ? a.g + (static_cast<size_t>(b) * a.T + t0) * a.H + h : a.g + h;
    const int stride = token ? a.H * 4 : 0;
    const __amdgpu_buffer_rsrc_t rs = lin_rsrc(base, a.decay == kNoDecay || live <= 0 ? 0 : (live - 1) * stride + 4);
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, lane < live ? lane * stride : 0x7ffffff0, 0, 0));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lin_dpp(double x) {
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xf, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// One wave.  A decay of zero (g = -inf) forgets all that came before: 4096 powers of two make
// every factor across it zero, and prefix sums stay finite.
template <int C>
__device__ __forceinline__ double lin_gates(LinGates<C> &t, float g, int lane) {
    double x = static_cast<double>(g) * kLinLog2e;
    x = x < -4096.0 ? -4096.0 : x;
    // inclusive prefix sums over the wave
    x += lin_dpp<0x111, 0xf>(x);   // row_shr:1
    x += lin_dpp<0x112, 0xf>(x);   // row_shr:2
    x += lin_dpp<0x114, 0xf>(x);   // row_shr:4
    x += lin_dpp<0x118, 0xf>(x);   // row_shr:8
    x += lin_dpp<0x142, 0xa>(x);   // row_bcast:15 into rows 1 and 3
    x += lin_dpp<0x143, 0xc>(x);   // row_bcast:31 into rows 2 and 3
    const uint64_t bits = __builtin_bit_cast(uint64_t, x);
    const uint32_t e0 = __builtin_amdgcn_readlane(static_cast<int>(bits), C - 1);
    const uint32_t e1 = __builtin_amdgcn_readlane(static_cast<int>(bits >> 32), C - 1);
    const double end = __builtin_bit_cast(double, static_cast<uint64_t>(e1) << 32 | e0);
    if (lane < C) {
        const float hi = static_cast<float>(x);
        t.hi[lane] = hi;
        t.lo[lane] = static_cast<float>(x - hi);
        t.before[lane] = lin_exp2(hi);
        t.after[lane] = lin_exp2(static_cast<float>(end - x));
        if (lane == 0) t.all[0] = lin_exp2(static_cast<float>(end));
    }
    return end;
}
// e^{G_s - G_t} for the tokens t..t+3 (an infinity or nonsense where t > s: not used there)
template <int C>
__device__ __forceinline__ f32x4 lin_between(const LinGates<C> &g, int s, int t) {
    const f32x4 hi = g.hi[s] - lds_f32x4(g.hi + t), lo = g.lo[s] - lds_f32x4(g.lo + t);
    f32x4 d;
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = lin_exp2(hi[e] + lo[e]);
    return d;
}

// ---------------------------------------------------------------- operands
// x as a sum of NS operands of the element type; fp32 takes one.
template <class P, int NS>
struct LinSplit {
    static constexpr int N = P::kBytes == 2 ? NS : 1;
    typename P::F p[N];
    __device__ __forceinline__ void of(f32x4 x) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p[j] = P::cvt(x);
            if (j + 1 < N) x -= P::f32(p[j]);
        }
    }
};

// state += its chunk's part: S = all S + sum_t (row_t) (col_t weight_t), the rows from LDS and the
// wave's columns, NC tiles of 16, in operand registers.
template <class P, int C, int NS, int D, int NC>
__device__ __forceinline__ void lin_update(f32x4 (&S)[NC][D / 16], LinTile<P, C, D> &rows,
                                           const typename P::F (&col)[NC][C / 32][2], const float *weight, float all,
                                           const LinLane &l) {
    const float *w = weight + 8 * (l.lane >> 4);
    constexpr bool kApart = P::kBytes == 4;      // the chunk's sum by itself: fewer roundings at the state's size
    if constexpr (!kApart) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int b = 0; b < D / 16; ++b) S[c][b] *= all;
    }
#pragma unroll
    for (int u = 0; u < C / 32; ++u) {
        LinSplit<P, NS> lo[NC], hi[NC];
        const f32x4 w0 = lds_f32x4(w + 32 * u + lin_half(0, l.lane)), w1 = lds_f32x4(w + 32 * u + lin_half(1, l.lane));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            lo[c].of(P::f32(col[c][u][0]) * w0);
            hi[c].of(P::f32(col[c][u][1]) * w1);
        }
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {
            const typename P::F r0 = rows.across(u, 0, b, l), r1 = rows.across(u, 1, b, l);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if constexpr (kApart) {
                    static_assert(C == 32, "one sum a chunk");
                    const f32x4 sum = P::mma2(zero4(), r0, r1, lo[c].p[0], hi[c].p[0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[c][b][e] = fmaf(S[c][b][e], all, sum[e]);
                } else {
#pragma unroll
                    for (int j = 0; j < LinSplit<P, NS>::N; ++j) S[c][b] = P::mma2(S[c][b], r0, r1, lo[c].p[j], hi[c].p[j]);
                }
            }
        }
    }
}

// The chunk's rows with the state (NS addends of it): acc[c][i] gets four columns of one token a
// lane, token 16 i + l % 16.
template <class P, int NS, int C, int D, int NC>
__device__ __forceinline__ void lin_read(f32x4 (&acc)[NC][C / 16], const f32x4 (&S)[NC][D / 16], LinTile<P, C, D> &rows,
                                         const LinLane &l) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < C / 16; ++i) acc[c][i] = zero4();
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        LinSplit<P, NS> s0[NC], s1[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            s0[c].of(S[c][2 * u]);
            s1[c].of(S[c][2 * u + 1]);
        }
#pragma unroll
        for (int i = 0; i < C / 16; ++i) {
            typename P::F x0, x1;
            rows.oct(i, u, l, x0, x1);
            if constexpr (P::kBytes == 4) {      // sums of 32 products, then their sum
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c][i] += P::mma2(zero4(), s0[c].p[0], s1[c].p[0], x0, x1);
            } else {
#pragma unroll
                for (int j = LinSplit<P, NS>::N - 1; j >= 0; --j)
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[c][i] = P::mma2(acc[c][i], s0[c].p[j], s1[c].p[j], x0, x1);
            }
        }
    }
}

// The wave's columns of a tile as operands: from tile of columns t0 on.
template <class P, int C, int D, int NC>
__device__ __forceinline__ void lin_columns(typename P::F (&col)[NC][C / 32][2], LinTile<P, C, D> &rows, int t0, const LinLane &l) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int u = 0; u < C / 32; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) col[c][u][e] = rows.down(u, e, t0 + c, l);
}

// acc += the chunk's own part: the rows of p (element [token][other token]) with the columns.
// LOWER: others up to the token; else from the token on.
template <class P, bool LOWER, int C, int NC>
__device__ __forceinline__ void lin_near(f32x4 (&acc)[NC][C / 16], LinTile<P, C, C> &p, const typename P::F (&col)[NC][C / 32][2],
                                         const LinLane &l) {
#pragma unroll
    for (int i = 0; i < C / 16; ++i)
#pragma unroll
        for (int u = LOWER ? 0 : i / 2; u < (LOWER ? i / 2 + 1 : C / 32); ++u) {
            typename P::F p0, p1;
            p.oct(i, u, l, p0, p1);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c][i] = P::mma2(acc[c][i], col[c][u][0], col[c][u][1], p0, p1);
        }
}

// A 16 x 16 block of products of LDS rows: lane l gets rows 16 i + 4 (l / 16) + e with row 16 j + l % 16.
template <class P, int C, int D>
__device__ __forceinline__ f32x4 lin_block(LinTile<P, C, D> &rows, LinTile<P, C, D> &cols, int i, int j, const LinLane &l) {
    f32x4 acc = zero4();
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        typename P::F x0, x1, y0, y1;
        rows.oct(i, u, l, x0, x1);
        cols.oct(j, u, l, y0, y1);
        acc = P::mma2(acc, x0, x1, y0, y1);
    }
    return acc;
}

// First of the four rows that tile t of a state has in this lane
__device__ __forceinline__ int lin_row(int t, int lane) { return 32 * (t >> 1) + 8 * (lane >> 4) + lin_half(t & 1, lane); }

// A state's tiles from and to [columns][D]: the lane's column, four rows at a time
template <int D>
__device__ __forceinline__ void lin_load(f32x4 (&S)[D / 16], const float *from, int col, int lane) {
#pragma unroll
    for (int t = 0; t < D / 16; ++t) S[t] = zero4();
    if (!from) return;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) S[t] = *reinterpret_cast<const f32x4 *>(from + static_cast<size_t>(col) * D + lin_row(t, lane));
}
template <int D>
__device__ __forceinline__ void lin_keep(const f32x4 (&S)[D / 16], float *to, int col, int lane) {
#pragma unroll
    for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4 *>(to + static_cast<size_t>(col) * D + lin_row(t, lane)) = S[t];
}

// Lower block triangle of at most four rows, row by row: p -> (i, j), j <= i
__device__ __forceinline__ void lin_pair(int p, int &i, int &j) {
    i = (p >= 1) + (p >= 3) + (p >= 6);
    j = p - i * (i + 1) / 2;
}
// The index of a wave, known to be the same in its lanes
__device__ __forceinline__ int lin_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }
// Two waves a SIMD: what the LDS leaves room for, and registers for loads ahead
#define LIN_TWO_WAVES __attribute__((amdgpu_waves_per_eu(2, 2)))

// The state before segment seg of head bh, and its gradient behind it: of the last piece before,
// of the first one behind
__device__ __forceinline__ const float *lin_before(const LinArgs &a, int bh, int seg) {
    const size_t state = static_cast<size_t>(a.DV) * a.DK;
    if (seg == 0) return a.S0 ? a.S0 + bh * state : nullptr;
    return a.fwd + (static_cast<size_t>(bh) * (a.segs - 1) * a.subs + seg * a.subs - 1) * state;
}
__device__ __forceinline__ const float *lin_behind(const LinArgs &a, int bh, int seg) {
    const size_t state = static_cast<size_t>(a.DV) * a.DK;
    if (seg == a.segs - 1) return a.dS_T ? a.dS_T + bh * state : nullptr;
    return a.rev + (static_cast<size_t>(bh) * (a.segs - 1) * a.subs + seg * a.subs) * state;
}

// Tokens of sequence b
__device__ __forceinline__ int lin_len(const LinArgs &a, int b) { return a.lens ? min(max(a.lens[b], 0), a.T) : a.T; }

}  // namespace qd
