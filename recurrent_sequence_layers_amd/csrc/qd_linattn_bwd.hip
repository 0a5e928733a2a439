// Gradients of linear attention with a decay for each head (formulas and layouts: qd_linattn.h).
//
// With R the gradient of the state behind a chunk (C tokens, entry state S, P and D as in the
// forward, D[s][t] = e^{G_s - G_t}):
//
//   dq_s = e^{G_s} S^T do_s + sum_{t<=s} D[s][t] (do_s . v_t) k_t
//   dk_t = e^{G_C - G_t} R^T v_t + sum_{s>=t} D[s][t] (do_s . v_t) q_s
//   dv_t = e^{G_C - G_t} R k_t + sum_{s>=t} P[s][t] do_s
//   R <- e^{G_C} R + sum_s e^{G_s} do_s q_s^T
//
// dq is the forward's form over (do, v, k), dk and dv the same backwards in time over (v, do, q)
// and (k, q, do).  So there are two walks and neither needs what the other finds: one workgroup
// goes forwards with S and forms dq, another one backwards with R, once by its value and once by
// its key columns, and forms dk and dv.  No state goes through memory.  q, k, v and do are read
// twice, once by each walk, which is less than the chunks' states would be.
//
// dg_t collects every pair of a token before t and one not before t:
//
//   dg_t = sum_{s>=t} a_s + sum_{i<t} b_i + sum_{i<t<=s} M[s][i] + c         within a chunk,
//   a_s = e^{G_s} do_s S q_s,  b_i = e^{G_C - G_i} v_i R k_i,  M = D o (Q K^T) o (dO V^T),
//   c = e^{G_C} <S, R>.
//
// Every term is one that g_t scales, and within a chunk each sum is of such terms alone, so behind a
// strong decay they are as small as dg is.  The walks write a, b and the third term: sums over
// parts of M's rows and columns, block by block.  c comes from a chain over the chunks: with
// E_n = <S, R> behind chunk n, c_n = E_n - sum b and E_{n-1} = c_n + sum a, from the segment's end on
// (<S_T, dS_T>, or what the states at the border give).  That is a difference: c is as exact as <S, R>
// at its chunk's ends is, not as itself, unless the chunk's whole decay is zero in fp32.  Then c is
// zero, and the chain ends on either side of the chunk with its own sums.
// a and b are taken before anything is rounded (the state split as in qd_linattn.h), since dg is fp32.
// The chain adds up their roundings; what it misses <S, R> by at its start is taken back in
// proportion to the squares of the sizes of the terms that it has passed, which is where it came from.
#include "qd_internal.h"
#include "qd_linattn.h"
#include "qd_mixer.h"

namespace qd {
namespace {

__device__ __forceinline__ float sum16(float x) { return group_sum(x, 16); }
__device__ __forceinline__ float sum64(float x) { return group_sum(x, 64); }
// Sums over 16 lanes: from this one on, and of those before it
__device__ __forceinline__ float behind16(float x) {
    x += dpp_src<0x101, 0xf>(x);   // row_shl:1
    x += dpp_src<0x102, 0xf>(x);
    x += dpp_src<0x104, 0xf>(x);
    return x + dpp_src<0x108, 0xf>(x);
}
__device__ __forceinline__ float before16(float x) {
    x = dpp_src<0x111, 0xf>(x);    // row_shr:1
    x += dpp_src<0x111, 0xf>(x);
    x += dpp_src<0x112, 0xf>(x);
    x += dpp_src<0x114, 0xf>(x);
    return x + dpp_src<0x118, 0xf>(x);
}

// 8 x 4096 tokens, 16 heads, 128 x 128, bf16, the decays' gradient too: 394 to 416 us, without it 323.
// The 944 MB would take 191 at the rate of a copy, and the two walks' 1.5 GB past the L2 305; the
// products, half of them for the 24 bits that dg is of, 242 at that of a large product.  The vector
// units, which split the states and their addends, are 56 % busy, the matrix units 36 %.  With dg the
// roles' registers do not quite fit the 168 that twelve waves leave each: 20 are spilled (fp32 30),
// without it 3.
//
// Twelve waves, two barriers a chunk.  Forwards four or eight waves hold the state, sixteen columns
// each; backwards four hold it by its key columns and four by its value columns, a quarter each (one
// of either a wave reads the LDS twice as often: 411 -> 443 us).  In a chunk's first interval they form
// its outputs, in the second they update the state.  The other waves meanwhile bring the next
// chunk: first from the registers, where its loads went a chunk before, to LDS, then its decayed
// products P, of which states' waves that have less to do take some.  Outputs wait in registers for
// the second interval, go to a tile of their chunk that nobody reads any more (dq to q, dk to k, dv to
// v) and leave in whole rows, each thread storing the pieces that it is about to replace.
constexpr int kBwdThreads = 768;
template <class P, int DK, int DV>
struct BwdLds {
    static constexpr int C = kLinChunk<P>, NB = (C / 16) * (C / 16 + 1) / 2;
    struct Chunk {
        LinTile<P, C, DK> q, k;
        LinTile<P, C, DV> v, o;
    } c[2];
    LinGates<C> gates[3];
    // Of do v forwards; of q k and of do v backwards.  Where the latter is read in the second interval,
    // bf16 forms it in the first one, fp32 in the second one before, so it has two in turn.
    // That is so for dg, whose three addends make reading the state the first interval's longest part
    // (fp32, 4096 x 16 x 128 x 128: 272 -> 261 us), and without it for bf16 while the registers last: 8 x
    // 1000 x 16 x 64 x 64 38.9 -> 37.4 us, 64 x 128 57.2 -> 55.5, but 128 x 128 spills, 324 -> 325.
    static constexpr bool later(bool dg) { return dg || (C == 64 && DK + DV < 256); }
    LinTile<P, C, C> p[P::kBytes == 4 ? 3 : 2];
    __device__ __forceinline__ LinTile<P, C, C> &second(bool dg, int m) { return p[P::kBytes == 4 && dg ? 1 + (m & 1) : 1]; }
    // Of M's blocks the sums of rows and of columns; of those on the diagonal, in rows, what is from
    // each token on and before it
    float rows[NB][16], cols[NB][16];
    float part[8][C];                  // a or b, by the columns' wave

    // Walks of one chunk have P as a sum of two: over few tokens its roundings would not average out.
    // What the first rounds away is in the second chunk's tiles, which have no other use then.
    using Tri = LinTile<P, C, C>;
    static_assert(sizeof(Tri) <= sizeof(c[1].q) && sizeof(Tri) <= sizeof(c[1].o), "a tile for the second addend");
    __device__ __forceinline__ Tri &low(int i) { return i ? reinterpret_cast<Tri &>(c[1].o) : reinterpret_cast<Tri &>(c[1].q); }
};

// Where a workgroup walks, and its tensors' first bytes.
template <class P, int DK, int DV>
struct Walk {
    static constexpr int C = kLinChunk<P>;
    const LinArgs &a;
    int b, h, bh, seg, c0, count, len, role, wave, lane, g4, r16;   // role: waves 0-3, 4-7, 8-11
    size_t sdk, sdv;
    LinLane l;

    __device__ __forceinline__ Walk(const LinArgs &a_, int unit) : a(a_), l(lane_id()) {
        seg = unit % a.segs;
        bh = unit / a.segs;
        b = bh / a.H;
        h = bh % a.H;
        role = lin_wave() >> 2;
        wave = lin_wave() & 3;
        lane = lane_id();
        g4 = lane >> 4;
        r16 = lane & 15;
        len = lin_len(a, b);
        c0 = seg * a.seg_chunks;
        count = min(a.seg_chunks, (a.T + C - 1) / C - c0);
        sdk = static_cast<size_t>(a.H) * DK * P::kBytes;
        sdv = static_cast<size_t>(a.H) * DV * P::kBytes;
    }
    // The m-th chunk of the walk
    template <bool REV>
    __device__ __forceinline__ int chunk(int m) const { return REV ? c0 + count - 1 - m : c0 + m; }
    __device__ __forceinline__ bool few() const { return P::kBytes == 2 && count == 1; }
    __device__ __forceinline__ int live(int n) const { return min(max(len - n * C, 0), C); }
    __device__ __forceinline__ size_t at(int t, size_t stride, int d) const {
        return (static_cast<size_t>(b) * a.T + t) * stride + static_cast<size_t>(h) * d * P::kBytes;
    }
    // Output rows of chunk n, padding's included: those are written as zeros
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t out(void *base, int n, bool valid, size_t stride, int d) const {
        const int rows = min(a.T - n * C, C);
        return lin_rsrc(static_cast<char *>(base) + (valid ? at(n * C, stride, d) : 0),
                        valid ? (rows - 1) * static_cast<int>(stride) + d * P::kBytes : 0);
    }
    // <S, R> before segment k
    __device__ __forceinline__ float *edge(int k) const { return a.edge + (static_cast<size_t>(bh) * (a.segs + 1) + k) * 8; }
    // One of the terms of dg for chunk n: a thread a token
    __device__ __forceinline__ void term(int which, int n, bool valid, int tid, float v) const {
        const float *to = a.tok + (static_cast<size_t>(which) * a.B * a.H + bh) * a.T + (valid ? n * C : 0);
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), lin_rsrc(to, valid ? min(a.T - n * C, C) * 4 : 0),
                                              tid * 4, 0, 0);
    }
    // a (backwards b) of chunk n from its NS parts, with its sum and mean size (forwards the chunk's
    // decay too): one wave
    template <bool REV, int NS, class L>
    __device__ __forceinline__ void terms(const L &lds, int n, float all) const {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NS; ++k) s += lds.part[k][lane & (C - 1)];
        term(REV ? 2 : 1, n, true, lane, s);
        s = lane < C ? s : 0.f;
        const float sum = wave_inclusive_sum(s), size = wave_inclusive_sum(fabsf(s) * (1.f / 64));
        LinSums &to = a.sums[static_cast<size_t>(bh) * ((a.T + C - 1) / C) + n];
        if (lane == 63) {
            (REV ? to.b : to.a) = sum;
            (REV ? to.size_b : to.size_a) = size;
            if (!REV) to.all = all;
        }
    }
};

// The decays, by one of the states' waves: those of chunk m + 2 in chunk m's second interval, where
// these waves have the least to do.
template <class P, int DK, int DV, bool REV>
struct Decays {
    const Walk<P, DK, DV> &w;
    float next;
    __device__ __forceinline__ float fetch(int m) const {
        const int n = m < w.count ? w.template chunk<REV>(m) : w.c0;
        return lin_gate(w.a, w.b, w.h, n * w.C, m < w.count ? w.live(n) : 0, w.lane);
    }
    // before the first chunk
    __device__ __forceinline__ Decays(const Walk<P, DK, DV> &w_, BwdLds<P, DK, DV> &lds) : w(w_), next(0.f) {
        if (w.role || w.wave) return;
        lin_gates(lds.gates[0], fetch(0), w.lane);
        lin_gates(lds.gates[1], fetch(1), w.lane);
        next = fetch(2);
    }
    __device__ __forceinline__ void ahead(BwdLds<P, DK, DV> &lds, int m) {
        if (w.role || w.wave) return;
        lin_gates(lds.gates[(m + 2) % 3], next, w.lane);
        next = fetch(m + 3);
    }
};

// A chunk's products, decayed.  Backwards by its earlier tokens' rows: blocks J .. J + N - 1 of earlier
// tokens with the later ones of block I, all of it in flight at once (block by block each waits for
// its own LDS reads).
template <class P, int I, int J, int N, int C, int D>
__device__ __forceinline__ void products_back(LinTile<P, C, D> &later, LinTile<P, C, D> &earlier, const LinGates<C> &gates,
                                              LinTile<P, C, C> &to, LinTile<P, C, C> *low, const LinLane &l) {
    static_assert(I < C / 16 && J + N - 1 <= I, "the lower triangle");
    const int g4 = l.lane >> 4, r16 = l.lane & 15, s = 16 * I + 4 * g4;
    f32x4 x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = zero4();
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        typename P::F a0, a1, b0[N], b1[N];
        later.oct(I, u, l, a0, a1);
#pragma unroll
        for (int n = 0; n < N; ++n) earlier.oct(J + n, u, l, b0[n], b1[n]);
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = P::mma2(x[n], a0, a1, b0[n], b1[n]);
    }
    const f32x4 hi = lds_f32x4(gates.hi + s), lo = lds_f32x4(gates.lo + s);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int t = 16 * (J + n) + r16;
        const float ht = gates.hi[t], lt = gates.lo[t];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = x[n][e] * lin_exp2((hi[e] - ht) + (lo[e] - lt));
            x[n][e] = J + n < I || t <= s + e ? v : 0.f;
        }
        P::st4(to.four(J + n, I, l), x[n]);
        if (low) P::st4(low->four(J + n, I, l), x[n] - P::f32(P::cvt(x[n])));
    }
}
// All of them by four waves: three, two, three and two blocks.
template <class P, int C, int D>
__device__ __forceinline__ void back_by_four(int wave, LinTile<P, C, D> &later, LinTile<P, C, D> &earlier, const LinGates<C> &gates,
                                             LinTile<P, C, C> &to, LinTile<P, C, C> *low, const LinLane &l) {
    if (wave == 0) {
        products_back<P, 3, 0, 2>(later, earlier, gates, to, low, l);
        products_back<P, 0, 0, 1>(later, earlier, gates, to, low, l);
    } else if (wave == 1) {
        products_back<P, 3, 2, 2>(later, earlier, gates, to, low, l);
    } else if (wave == 2) {
        products_back<P, 2, 0, 3>(later, earlier, gates, to, low, l);
    } else {
        products_back<P, 1, 0, 2>(later, earlier, gates, to, low, l);
    }
}
// By two waves, five blocks each (fp32: two and one).
template <class P, int C, int D>
__device__ __forceinline__ void back_by_two(int wave, LinTile<P, C, D> &later, LinTile<P, C, D> &earlier, const LinGates<C> &gates,
                                            LinTile<P, C, C> &to, LinTile<P, C, C> *low, const LinLane &l) {
    if constexpr (C == 64) {
        if (wave == 0) {
            products_back<P, 3, 0, 4>(later, earlier, gates, to, low, l);
            products_back<P, 0, 0, 1>(later, earlier, gates, to, low, l);
        } else {
            products_back<P, 2, 0, 3>(later, earlier, gates, to, low, l);
            products_back<P, 1, 0, 2>(later, earlier, gates, to, low, l);
        }
    } else {
        if (wave == 0) products_back<P, 0, 0, 1>(later, earlier, gates, to, low, l);
        else products_back<P, 1, 0, 2>(later, earlier, gates, to, low, l);
    }
}
// By eight waves: seven of ten by four of them, three by the others, with less time (few): the
// loading ones, or without dg those that hold dk.
template <class P, int C, int D>
__device__ __forceinline__ void back_by_eight(bool few, int wave, LinTile<P, C, D> &later, LinTile<P, C, D> &earlier,
                                              const LinGates<C> &gates, LinTile<P, C, C> &to, LinTile<P, C, C> *low, const LinLane &l) {
    if (!few) {
        if (wave == 0) products_back<P, 3, 0, 2>(later, earlier, gates, to, low, l);
        else if (wave == 1) products_back<P, 3, 2, 2>(later, earlier, gates, to, low, l);
        else if (wave == 2) products_back<P, 2, 0, 2>(later, earlier, gates, to, low, l);
        else products_back<P, 2, 2, 1>(later, earlier, gates, to, low, l);
    } else {
        if (wave == 0) products_back<P, 1, 0, 1>(later, earlier, gates, to, low, l);
        else if (wave == 1) products_back<P, 1, 1, 1>(later, earlier, gates, to, low, l);
        else if (wave == 2) products_back<P, 0, 0, 1>(later, earlier, gates, to, low, l);
    }
}
// Forwards by its later tokens' rows, of do v; for dg with M's sums over the block.
template <class P, int DK, int DV, bool DG>
__device__ __forceinline__ void product(const Walk<P, DK, DV> &w, BwdLds<P, DK, DV> &lds, int m, int p) {
    typename BwdLds<P, DK, DV>::Chunk &next = lds.c[(m + 1) & 1];
    const LinGates<kLinChunk<P>> &gates = lds.gates[(m + 1) % 3];
    int i, j;
    lin_pair(p, i, j);
    f32x4 ov = lin_block<P>(next.v, next.o, j, i, w.l);
    const int s = 16 * i + w.r16, t = 16 * j + 4 * w.g4;
    ov *= lin_between(gates, s, t);
    if (i == j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ov[e] = t + e <= s ? ov[e] : 0.f;
    }
    P::st4(lds.p[0].four(i, j, w.l), ov);
    if (w.few()) P::st4(lds.low(0).four(i, j, w.l), ov - P::f32(P::cvt(ov)));
    if constexpr (DG) {
        const f32x4 qk = lin_block<P>(next.k, next.q, j, i, w.l);
        float row = 0.f;
        if (i == j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {        // from token s on, the columns before it
                const float x = behind16(t + e < s ? ov[e] * qk[e] : 0.f);
                row += t + e < s ? x : 0.f;
            }
        } else {
            f32x4 col;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = ov[e] * qk[e];
                row += x;
                col[e] = sum16(x);
            }
            if (w.r16 == 0) *reinterpret_cast<f32x4 *>(&lds.cols[p][4 * w.g4]) = col;
        }
        row += __shfl_xor(row, 16);
        row += __shfl_xor(row, 32);
        if (w.lane < 16) lds.rows[p][w.r16] = row;
    }
}

// The loading waves, NW of them; `wave` counts from the first.  Forwards they form the blocks up to LAST.
template <class P, int DK, int DV, bool REV, bool DG, int NW, int LAST = BwdLds<P, DK, DV>::NB>
__device__ __forceinline__ void bring(const Walk<P, DK, DV> &w, BwdLds<P, DK, DV> &lds, int wave) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NT = 64 * NW;
    const LinArgs &a = w.a;
    const int sdk = static_cast<int>(w.sdk), sdv = static_cast<int>(w.sdv), tid = 64 * wave + w.lane;
    LinRows<P, C, DK, NT> rq, rk;
    LinRows<P, C, DV, NT> rv, ro;
    // every step has the same loads and stores, those past the walk's ends of nothing: with a
    // branch around stores the waits for older loads would wait for them too
    auto fetch = [&](int m) {
        const int n = m < w.count ? w.template chunk<REV>(m) : w.c0, t0 = n * C, live = m < w.count ? w.live(n) : 0;
        rq.load(static_cast<const char *>(a.q) + w.at(t0, w.sdk, DK), live, sdk, tid);
        rk.load(static_cast<const char *>(a.k) + w.at(t0, w.sdk, DK), live, sdk, tid);
        rv.load(static_cast<const char *>(a.v) + w.at(t0, w.sdv, DV), live, sdv, tid);
        ro.load(static_cast<const char *>(a.d_o) + w.at(t0, w.sdv, DV), live, sdv, tid);
    };
    auto emit = [&](int m) {                     // the outputs of chunk m - 1, from the tiles of chunk m + 1
        const bool valid = m >= 1 && m <= w.count;
        const int n = valid ? w.template chunk<REV>(m - 1) : 0;
        typename L::Chunk &c = lds.c[(m + 1) & 1];
        if constexpr (REV) {
            lin_store<P, C, DK, NT>(c.k, w.out(a.dk, n, valid, w.sdk, DK), sdk, tid);
            lin_store<P, C, DV, NT>(c.v, w.out(a.dv, n, valid, w.sdv, DV), sdv, tid);
        } else {
            lin_store<P, C, DK, NT>(c.q, w.out(a.dq, n, valid, w.sdk, DK), sdk, tid);
        }
    };
    fetch(0);
    for (int m = -1; m < w.count; ++m) {
        const bool valid = m >= 0;
        const int n = valid ? w.template chunk<REV>(m) : 0;
        typename L::Chunk &next = lds.c[(m + 1) & 1];
        emit(m);
        if (m < 0 || !w.few()) {
            rq.put(next.q, tid);
            rk.put(next.k, tid);
            rv.put(next.v, tid);
            ro.put(next.o, tid);
        }
        if constexpr (DG && REV && C == 64) {    // while the registers are free
            typename L::Chunk &x = lds.c[m & 1];
            if (valid) back_by_eight<P>(true, wave, x.o, x.v, lds.gates[m % 3], lds.p[1], w.few() ? &lds.low(1) : nullptr, w.l);
        }
        fetch(m + 2);
        if constexpr (DG && !REV) {
            // token e of block i: the rows from it on of the blocks to its left, the columns before it
            // of those below, all of what is both
            const int i = (tid >> 4) & (C / 16 - 1), e = tid & 15;
            float row = 0.f, col = 0.f;
#pragma unroll
            for (int j = 0; j < C / 16; ++j) {
                if (j < i) row += lds.rows[i * (i + 1) / 2 + j][e];
                if (j > i) col += lds.cols[j * (j + 1) / 2 + i][e];
            }
#pragma unroll
            for (int j = 2; j < C / 16; ++j)
#pragma unroll
                for (int k = 0; k < j - 1; ++k)
                    if (k < i && i < j) {        // e and the rows behind it, and those before it
                        const float x = lds.rows[j * (j + 1) / 2 + k][e];
                        row += x;
                        col += x;
                    }
            w.term(0, n, valid, tid, lds.rows[i * (i + 3) / 2][e] + behind16(row) + before16(col));
        }
        __syncthreads();
        if constexpr (REV) {
            const LinGates<C> &gates = lds.gates[(m + 1) % 3];
            const bool low = w.few() && m < 0;
            if constexpr (C == 64 && L::later(DG)) back_by_four<P>(wave, next.q, next.k, gates, lds.p[0], low ? &lds.low(0) : nullptr, w.l);
            else if (wave & 1) back_by_two<P>(wave >> 1, next.o, next.v, gates, lds.second(DG, m + 1), low ? &lds.low(1) : nullptr, w.l);
            else back_by_two<P>(wave >> 1, next.q, next.k, gates, lds.p[0], low ? &lds.low(0) : nullptr, w.l);
        } else {
            // two of eight waves take two of ten blocks: none of the diagonal's, whose sums take longer
            for (int p = wave; p < LAST; p += NW)
                product<P, DK, DV, DG>(w, lds, m, NW == 8 && L::NB == 10 ? 0x8764952031ull >> 4 * p & 15 : p);
        }
        __syncthreads();
    }
    emit(w.count);
}

// a or b: the state's part of each output row with the row's own q or k, over a wave's columns
template <class P, int C, int D, int NC>
__device__ __forceinline__ void row_parts(float *part, LinTile<P, C, D> &rows, const f32x4 (&acc)[NC][C / 16], int t0,
                                          const LinLane &l) {
#pragma unroll
    for (int i = 0; i < C / 16; ++i) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const f32x4 y = P::f32(P::ld4(rows.four(i, t0 + c, l)));
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fmaf(acc[c][i][e], y[e], s);
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (l.lane < 16) part[16 * i + l.lane] = s;
    }
}
template <int C, int NC>
__device__ __forceinline__ void scale(f32x4 (&acc)[NC][C / 16], const float *w, int r16) {
#pragma unroll
    for (int i = 0; i < C / 16; ++i) {
        const float x = w[16 * i + r16];
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c][i] *= x;
    }
}
// Outputs as elements, zeros in padding
template <class P, int C, int NC>
__device__ __forceinline__ void pack(typename P::F (&out)[NC][C / 16], f32x4 (&acc)[NC][C / 16], int live, int r16) {
    if (live < C) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < C / 16; ++i)
                if (16 * i + r16 >= live) acc[c][i] = zero4();
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < C / 16; ++i) out[c][i] = P::cvt(acc[c][i]);
}
template <class P, int C, int D, int NC>
__device__ __forceinline__ void spill_out(LinTile<P, C, D> &to, const typename P::F (&out)[NC][C / 16], int t0, const LinLane &l) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
            *reinterpret_cast<typename P::F *>(to.four(i, t0 + c, l)) = out[c][i];
}
// A state whose columns are key indices, from and to [DV][DK]
template <int DK, int DV, int NC>
__device__ __forceinline__ void load_across(f32x4 (&S)[NC][DV / 16], const float *from, int c0, int lane) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int t = 0; t < DV / 16; ++t) S[c][t] = zero4();
    if (!from) return;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int t = 0; t < DV / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[c][t][e] = from[(lin_row(t, lane) + e) * DK + c0 + 16 * c + (lane & 15)];
}

// The inner product of a wave's columns with those of [DV][DK] (null: zeros)
template <int DK, int DV, int NC>
__device__ __forceinline__ float inner(const f32x4 (&S)[NC][DV / 16], const float *other, int c0, int lane) {
    if (!other) return 0.f;
    f32x4 d[NC][DV / 16];
    load_across<DK, DV>(d, other, c0, lane);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int t = 0; t < DV / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fmaf(S[c][t][e], d[c][t][e], s);
    return sum64(s);
}

// ---------------------------------------------------------------- dq, forwards
template <class P, int DK, int DV, bool DG>
__device__ __forceinline__ void dq_walk(const LinArgs &a, BwdLds<P, DK, DV> &lds, int unit) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NC = 1, NS = DK / 16;
    const Walk<P, DK, DV> w(a, unit);
    const int wave = 4 * w.role + w.wave;
    // with eight waves on the state, whose second interval is short, six of them take a block each
    constexpr int LAST = NS == 8 && L::NB == 10 ? 4 : L::NB;
    if (wave >= NS) return bring<P, DK, DV, false, DG, 12 - NS, LAST>(w, lds, wave - NS);
    const int lane = w.lane, t0 = wave, c0 = 16 * t0;
    const size_t state = static_cast<size_t>(DV) * DK;
    f32x4 S[NC][DV / 16];
    load_across<DK, DV>(S, lin_before(a, w.bh, w.seg), c0, lane);
    if constexpr (DG) {
        if (w.seg > 0) {
            const float s = inner<DK, DV>(S, lin_behind(a, w.bh, w.seg - 1), c0, lane);
            if (lane == 0) w.edge(w.seg)[wave] = s;
        }
    }
    Decays<P, DK, DV, false> decays(w, lds);
    auto help = [&](int m) {
        if (LAST < L::NB && wave >= 2) product<P, DK, DV, DG>(w, lds, m, LAST + wave - 2);
    };
    __syncthreads();                             // the first chunk is brought
    help(-1);
    __syncthreads();
    for (int m = 0; m < w.count; ++m) {
        typename L::Chunk &x = lds.c[m & 1];
        const LinGates<C> &gates = lds.gates[m % 3];
        typename P::F kf[NC][C / 32][2], out[NC][C / 16];
        {
            f32x4 acc[NC][C / 16];
            lin_read<P, DG ? 3 : 1>(acc, S, x.o, w.l);
            scale<C>(acc, gates.before, w.r16);
            if constexpr (DG) row_parts<P>(lds.part[wave], x.q, acc, t0, w.l);
            lin_columns<P, C>(kf, x.k, t0, w.l);
            lin_near<P, true>(acc, lds.p[0], kf, w.l);
            if (w.few()) lin_near<P, true>(acc, lds.low(0), kf, w.l);
            pack<P, C>(out, acc, w.live(w.c0 + m), w.r16);
        }
        __syncthreads();
        help(m);
        spill_out<P, C>(x.q, out, t0, w.l);
        lin_update<P, C, DG ? 3 : 2>(S, x.v, kf, gates.after, gates.all[0], w.l);
        if (DG && wave == 1) w.template terms<false, NS>(lds, w.c0 + m, gates.all[0]);
        decays.ahead(lds, m);
        __syncthreads();
    }
    if constexpr (DG) {
        if (w.seg == a.segs - 1) {               // <S_T, dS_T>
            const float s = inner<DK, DV>(S, a.dS_T ? a.dS_T + w.bh * state : nullptr, c0, lane);
            if (lane == 0) w.edge(a.segs)[wave] = s;
        }
    }
}

// ---------------------------------------------------------------- dk and dv, backwards
// dv: the gradient's columns are value indices.
template <class P, int DK, int DV, bool DG>
__device__ __forceinline__ void dv_walk(const Walk<P, DK, DV> &w, BwdLds<P, DK, DV> &lds, const float *from) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NC = DV / 64;
    const int lane = w.lane, t0 = NC * w.wave, c0 = 16 * t0;
    f32x4 R[NC][DK / 16];
#pragma unroll
    for (int c = 0; c < NC; ++c) lin_load<DK>(R[c], from, c0 + 16 * c + w.r16, lane);
    __syncthreads();                             // the first chunk is brought
    __syncthreads();
    for (int m = 0; m < w.count; ++m) {
        typename L::Chunk &x = lds.c[m & 1];
        const LinGates<C> &gates = lds.gates[m % 3];
        typename P::F of[NC][C / 32][2], out[NC][C / 16];
        // dk's products, where they are for the second interval
        if constexpr (C == 64 && L::later(DG)) back_by_eight<P>(false, w.wave, x.o, x.v, gates, lds.p[1], w.few() ? &lds.low(1) : nullptr, w.l);
        {
            f32x4 acc[NC][C / 16];
            lin_columns<P, C>(of, x.o, t0, w.l);
            lin_read<P, 1>(acc, R, x.k, w.l);
            scale<C>(acc, gates.after, w.r16);
            lin_near<P, false>(acc, lds.p[0], of, w.l);
            if (w.few()) lin_near<P, false>(acc, lds.low(0), of, w.l);
            pack<P, C>(out, acc, w.live(w.template chunk<true>(m)), w.r16);
        }
        __syncthreads();
        spill_out<P, C>(x.v, out, t0, w.l);
        lin_update<P, C, 2>(R, x.q, of, gates.before, gates.all[0], w.l);
        __syncthreads();
    }
}
// dk: its columns are key indices.
template <class P, int DK, int DV, bool DG, int NS>
__device__ __forceinline__ void dk_walk(const Walk<P, DK, DV> &w, BwdLds<P, DK, DV> &lds, const float *from) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NC = DK / 64;
    const int lane = w.lane, t0 = NC * w.wave, c0 = 16 * t0;
    f32x4 R[NC][DV / 16];
    load_across<DK, DV>(R, from, c0, lane);
    Decays<P, DK, DV, true> decays(w, lds);
    __syncthreads();                             // the first chunk is brought
    __syncthreads();
    for (int m = 0; m < w.count; ++m) {
        typename L::Chunk &x = lds.c[m & 1];
        const LinGates<C> &gates = lds.gates[m % 3];
        typename P::F qf[NC][C / 32][2], out[NC][C / 16];
        if constexpr (!DG && C == 64 && L::later(DG)) back_by_eight<P>(true, w.wave, x.o, x.v, gates, lds.p[1], w.few() ? &lds.low(1) : nullptr, w.l);
        f32x4 acc[NC][C / 16];
        lin_read<P, DG ? 3 : 1>(acc, R, x.v, w.l);
        scale<C>(acc, gates.after, w.r16);
        // the chunk's own part
        auto own = [&] {
            lin_columns<P, C>(qf, x.q, t0, w.l);
            lin_near<P, false>(acc, lds.second(DG, m), qf, w.l);
            if (w.few()) lin_near<P, false>(acc, lds.low(1), qf, w.l);
            pack<P, C>(out, acc, w.live(w.template chunk<true>(m)), w.r16);
        };
        if constexpr (DG) row_parts<P>(lds.part[w.wave], x.k, acc, t0, w.l);
        if constexpr (!L::later(DG)) own();
        __syncthreads();
        if constexpr (L::later(DG)) own();
        spill_out<P, C>(x.k, out, t0, w.l);
        lin_update<P, C, NS>(R, x.o, qf, gates.before, gates.all[0], w.l);
        if (DG && w.wave == 1) w.template terms<true, 4>(lds, w.template chunk<true>(m), 0.f);
        decays.ahead(lds, m);
        __syncthreads();
    }
    const LinArgs &a = w.a;
    if (DG && w.seg == 0) {                      // <S0, dS0>
        const float s = inner<DK, DV>(R, a.S0 ? a.S0 + static_cast<size_t>(w.bh) * DV * DK : nullptr, c0, lane);
        if (lane == 0) w.edge(0)[w.wave] = s;
    }
    if (a.dS0 && w.seg == 0) {
        float *to = a.dS0 + static_cast<size_t>(w.bh) * DV * DK;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int t = 0; t < DV / 16; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) to[(lin_row(t, lane) + e) * DK + c0 + 16 * c + w.r16] = R[c][t][e];
    }
}
template <class P, int DK, int DV, bool DG, int NS>
__device__ __forceinline__ void dkv_walk(const LinArgs &a, BwdLds<P, DK, DV> &lds, int unit) {
    const Walk<P, DK, DV> w(a, unit);
    if (w.role == 2) return bring<P, DK, DV, true, DG, 4>(w, lds, w.wave);
    const float *from = lin_behind(a, w.bh, w.seg);
    if (w.role == 0) dk_walk<P, DK, DV, DG, NS>(w, lds, from);
    else dv_walk<P, DK, DV, DG>(w, lds, from);
}

template <class P, int DK, int DV, bool DG, int NS>
__global__ __launch_bounds__(kBwdThreads) __attribute__((amdgpu_waves_per_eu(3, 3))) void lin_bwd_kernel(const LinArgs a) {
    using L = BwdLds<P, DK, DV>;
    extern __shared__ __align__(16) char smem[];
    L &lds = *reinterpret_cast<L *>(smem);
    // blocks of P off its triangle that a pair of tiles reads: never written again
    for (int e = threadIdx.x; e < LinTile<P, L::C, L::C>::kElems; e += kBwdThreads) lds.p[0].m[e] = lds.p[1].m[e] = lds.p[sizeof(lds.p) / sizeof(lds.p[0]) - 1].m[e] = lds.low(0).m[e] = lds.low(1).m[e] = 0;
    __syncthreads();
    const int unit = blockIdx.x >> 1;
    if (blockIdx.x & 1) dq_walk<P, DK, DV, DG>(a, lds, unit);
    else dkv_walk<P, DK, DV, DG, NS>(a, lds, unit);
}

// ---------------------------------------------------------------- dg
constexpr int kDgWaves = 16, kDgChunks = 1024;

// Sum over a wave, in every lane
__device__ __forceinline__ double lin_total(double x) {
    x += lin_dpp<0x111, 0xf>(x);
    x += lin_dpp<0x112, 0xf>(x);
    x += lin_dpp<0x114, 0xf>(x);
    x += lin_dpp<0x118, 0xf>(x);
    x += lin_dpp<0x142, 0xa>(x);
    x += lin_dpp<0x143, 0xc>(x);
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), 63), hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), 63);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
struct Ends {
    int first, count;                // the segment's chunks
    double before, behind;           // <S, R> at its borders
    __device__ __forceinline__ Ends(const LinArgs &a, size_t bh, int nc, int seg)
        : first(seg * a.seg_chunks), count(min(a.seg_chunks, nc - first)), before(0), behind(0) {
        const float *e = a.edge + (bh * (a.segs + 1) + seg) * 8;
        for (int w = 0; w < (seg ? a.DK / 16 : 4); ++w) before += e[w];
        for (int w = 0; w < a.DK / 16; ++w) behind += e[8 + w];
    }
};
// The chain of c for chunk n by one wave, from all the chunks' sums.
__device__ __forceinline__ float chain_at(const LinArgs &a, size_t bh, int nc, int n, int lane) {
    const Ends e(a, bh, nc, n / a.seg_chunks);
    const LinSums *sums = a.sums + bh * nc + e.first;
    const int at = n - e.first;
    double start = e.before, end = e.behind, D, V, later, passed, own;
    auto chunks = [&](int lo, int hi) {          // sums over those between; whether one of them forgets
        bool forgets = false;
        D = V = later = passed = own = 0;
        for (int m = lane; m < hi; m += kWave) {
            if (m <= lo) continue;
            const LinSums x = sums[m];
            const double d = static_cast<double>(x.a) - x.b, v = x.weight();
            D += d;
            V += v;
            later += m > at ? d : 0;
            passed += m > at ? v : m == at ? 0.5 * v : 0;
            own += m == at ? x.b : 0;
            forgets = forgets || x.all == 0.f;
        }
        return __any(forgets);
    };
    if (chunks(-1, e.count)) {
        // what forgets all ends the chain: behind it <S, R> is its sum of b, before it that of a
        int lo = -1, hi = e.count;
        for (int m = lane; m < e.count; m += kWave) {
            if (sums[m].all != 0.f) continue;
            if (m <= at) lo = m;
            else hi = min(hi, m);
        }
#pragma unroll
        for (int k = 1; k < kWave; k *= 2) {
            lo = max(lo, __shfl_xor(lo, k));
            hi = min(hi, __shfl_xor(hi, k));
        }
        if (lo == at) return 0.f;
        if (lo >= 0) start = sums[lo].b;
        if (hi < e.count) end = sums[hi].a;
        chunks(lo, hi);
    }
    D = lin_total(D);
    V = lin_total(V);
    return static_cast<float>(end + lin_total(later) - lin_total(own) - (V > 0 ? (end + D - start) / V * lin_total(passed) : 0));
}

// The same for all of a segment's chunks, where they are many: one workgroup, 1024 chunks at a time, from
// the last one on; then from the first one on, since what a chain misses is known at its start.
// A call of 7 chunks 34 us, by this launch 39; 64 399, 410; 256 782, 783; 512 1617, 1573; 2048 7212, 6630.
constexpr int kFewChunks = 256;
__global__ __launch_bounds__(64 * kDgWaves) void lin_chain_kernel(const LinArgs a, const int nc) {
    __shared__ float sa[kDgChunks], sb[kDgChunks];
    __shared__ double sv[kDgChunks];             // negative: the chunk forgets all
    __shared__ double missed, part[kDgWaves];    // by a term's weight: of the first chain, and of a wave's last chunk that forgets
    __shared__ bool any[kDgWaves];
    const size_t bh = blockIdx.x / a.segs;
    const int wave = wave_id(), lane = lane_id();
    const Ends ends(a, bh, nc, blockIdx.x % a.segs);
    LinSums *sums = a.sums + bh * nc + ends.first;
    double *far = a.chain + 2 * (bh * nc + ends.first);
    double E = ends.behind, passed = 0;
    for (int last = ends.count; last > 0; last -= kDgChunks) {
        const int first = max(last - kDgChunks, 0), count = last - first;
        for (int m = threadIdx.x; m < count; m += 64 * kDgWaves) {
            const LinSums x = sums[first + m];
            sa[m] = x.a;
            sb[m] = x.b;
            sv[m] = x.all == 0.f ? -1. : x.weight();
        }
        __syncthreads();
        if (wave == 0) {
            // a lane's chunks are consecutive, from the last on.  cut: one of them, or of those of the
            // lanes before, forgets, and d and v are of what is behind it
            constexpr int PER = kDgChunks / 64;
            double d = 0, v = 0;
            int cut = 0;
            for (int i = 0; i < PER; ++i) {
                const int m = count - 1 - (lane * PER + i);
                if (m < 0) break;
                if (sv[m] < 0) {
                    cut = 1;
                    d = sa[m];
                    v = 0;
                } else {
                    d += static_cast<double>(sa[m]) - sb[m];
                    v += sv[m];
                }
            }
            for (int s = 1; s < 64; s *= 2) {
                const double y = __shfl_up(d, s), z = __shfl_up(v, s);
                const int q = __shfl_up(cut, s);
                if (lane >= s && !cut) {
                    d += y;
                    v += z;
                    cut = q;
                }
            }
            double e = __shfl_up(d, 1), p = __shfl_up(v, 1);
            const int before = __shfl_up(cut, 1);
            if (lane == 0) e = p = 0;
            if (lane == 0 || !before) {
                e += E;
                p += passed;
            }
            for (int i = 0; i < PER; ++i) {
                const int m = count - 1 - (lane * PER + i);
                if (m < 0) break;
                double *to = far + 2 * static_cast<size_t>(first + m);
                const double own = e - sb[m];
                if (sv[m] < 0) {                 // what the chain behind it has missed
                    to[0] = 0;
                    to[1] = p > 0 ? own / p : 0;
                    e = sa[m];
                    p = 0;
                } else {
                    to[0] = own;
                    to[1] = p + 0.5 * sv[m];
                    e = own + sa[m];
                    p += sv[m];
                }
            }
            const bool cut_all = __shfl(cut, 63);
            E = __shfl(d, 63) + (cut_all ? 0 : E);
            passed = __shfl(v, 63) + (cut_all ? 0 : passed);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) missed = passed > 0 ? (E - ends.before) / passed : 0;
    __syncthreads();
    double share = missed;                       // of the chain that goes on into these chunks
    for (int first = 0; first < ends.count; first += 64 * kDgWaves) {
        const int m = first + threadIdx.x;
        const bool valid = m < ends.count, forgets = valid && sums[m].all == 0.f;
        const double own = valid ? far[2 * static_cast<size_t>(m)] : 0, weight = valid ? far[2 * static_cast<size_t>(m) + 1] : 0;
        const uint64_t mask = __ballot(forgets), lower = mask & ((1ull << lane) - 1);
        if (lane == 0) any[wave] = mask != 0;
        if (mask && lane == 63 - __builtin_clzll(mask)) part[wave] = weight;
        const double near = __shfl(weight, lower ? 63 - __builtin_clzll(lower) : 0);
        __syncthreads();
        double mine = share;
        for (int w = 0; w < kDgWaves; ++w) {
            if (!any[w]) continue;
            if (w < wave) mine = part[w];
            share = part[w];
        }
        if (lower) mine = near;
        if (valid) sums[m].c = forgets ? 0.f : static_cast<float>(own - mine * weight);
        __syncthreads();
    }
}

// dg of a chunk of sixteen heads: a wave a head, rows of heads through LDS.
template <int C>
__global__ __launch_bounds__(64 * kDgWaves) void lin_dg_kernel(const LinArgs a) {
    __shared__ float out[64][kDgWaves + 1];
    const int nc = (a.T + C - 1) / C, n = blockIdx.x % nc, b = blockIdx.x / nc, h0 = blockIdx.y * kDgWaves;
    const int wave = wave_id(), lane = lane_id(), h = h0 + wave;
    const size_t bhs = static_cast<size_t>(a.B) * a.H, bh = static_cast<size_t>(b) * a.H + h;
    const int len = lin_len(a, b), live = min(max(len - n * C, 0), C);
    float v = 0.f;
    if (h < a.H && live > 0) {
        const float *x = a.tok + bh * a.T + n * C, *ta = x + bhs * a.T, *tb = ta + bhs * a.T;
        const int back = 63 - lane;
        const float pairs = lane < live ? x[lane] : 0.f, y = lane < live ? tb[lane] : 0.f, z = back < live ? ta[back] : 0.f;
        const float upto = __shfl_up(wave_inclusive_sum(y), 1), before = lane ? upto : 0.f;
        const float behind = __shfl(wave_inclusive_sum(z), back);
        const float c = a.seg_chunks <= kFewChunks ? chain_at(a, bh, nc, n, lane) : a.sums[bh * nc + n].c;
        v = lane < live ? c + (pairs + (before + behind)) : 0.f;
    }
    if (a.decay == kHeadDecay) {
        v = sum64(v);
        if (h < a.H && lane == 0) a.head[(static_cast<size_t>(b) * nc + n) * a.H + h] = v;
        return;
    }
    out[lane][wave] = v;
    __syncthreads();
    const int t = threadIdx.x / kDgWaves, k = threadIdx.x % kDgWaves;
    if (t < C && n * C + t < a.T && h0 + k < a.H)
        a.dg[(static_cast<size_t>(b) * a.T + n * C + t) * a.H + h0 + k] = out[t][k];
}
struct HeadStore {
    float *to;
    __device__ __forceinline__ void operator()(long long h, float v) const { to[h] = v; }
};

template <class P, int DK, int DV>
hipError_t bwd_sized(const LinArgs &a, hipStream_t stream) {
    using L = BwdLds<P, DK, DV>;
    static_assert(sizeof(L) <= 160 * 1024, "LDS of a workgroup");
    const dim3 grid(static_cast<unsigned>(2LL * a.B * a.H * a.segs)), blk(kBwdThreads);
    if (a.dg) hipLaunchKernelGGL((lin_bwd_kernel<P, DK, DV, true, 3>), grid, blk, sizeof(L), stream, a);
    else if (a.dS0) hipLaunchKernelGGL((lin_bwd_kernel<P, DK, DV, false, 3>), grid, blk, sizeof(L), stream, a);
    else hipLaunchKernelGGL((lin_bwd_kernel<P, DK, DV, false, 2>), grid, blk, sizeof(L), stream, a);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.dg) {
        const unsigned nc = (a.T + L::C - 1) / L::C;
        if (a.seg_chunks > kFewChunks) hipLaunchKernelGGL(lin_chain_kernel, dim3(static_cast<unsigned>(a.B * a.H * a.segs)), dim3(64 * kDgWaves), 0, stream, a, static_cast<int>(nc));
        hipLaunchKernelGGL(lin_dg_kernel<L::C>, dim3(nc * a.B, (a.H + kDgWaves - 1) / kDgWaves), dim3(64 * kDgWaves), 0, stream, a);
        if (a.decay == kHeadDecay) column_sum(a.head, static_cast<int>(nc * a.B), a.H, HeadStore{a.dg}, stream);
    }
    return hipGetLastError();
}
template <class P>
hipError_t bwd_typed(const LinArgs &a, hipStream_t stream) {
    if (a.DK == 128) return a.DV == 128 ? bwd_sized<P, 128, 128>(a, stream) : bwd_sized<P, 128, 64>(a, stream);
    return a.DV == 128 ? bwd_sized<P, 64, 128>(a, stream) : bwd_sized<P, 64, 64>(a, stream);
}

// Both walks of every head are 2 B H workgroups.  A chunk's step is long here, and the states of
// both directions cost a quarter of it.
void bwd_plan(int dtype, LinArgs &a) { lin_plan(dtype, a, 2LL * a.B * a.H, 2, 0.25); }

}  // namespace

size_t lin_bwd_workspace(int dtype, int B, int T, int H, int dk, int dv, bool dg) {
    if (static_cast<long long>(B) * H * T == 0) return 0;
    LinArgs a{};
    a.B = B; a.T = T; a.H = H; a.DK = dk; a.DV = dv;
    bwd_plan(dtype, a);
    const size_t bh = static_cast<size_t>(B) * H;
    const size_t chunks = bh * ((T + lin_chunk(dtype) - 1) / lin_chunk(dtype));
    const size_t terms = dg ? chunks * (sizeof(LinSums) + 2 * sizeof(double) + sizeof(float)) + (3 * bh * T + bh * 8 * (a.segs + 1)) * sizeof(float) : 0;
    return lin_states_floats(a, 2) * sizeof(float) + terms;
}

hipError_t launch_lin_bwd(int dtype, LinArgs a, void *ws, hipStream_t stream) {
    const size_t bh = static_cast<size_t>(a.B) * a.H, state = static_cast<size_t>(a.DV) * a.DK;
    if (a.T == 0 || bh == 0) {
        // no tokens: dS0 = dS_T, and sums over tokens are zero
        if (a.dS0 && bh)
            if (hipError_t e = launch_lin_copy(a.dS0, a.dS_T, bh * state, stream)) return e;
        if (a.dg && a.decay == kHeadDecay && a.H) column_sum(a.dg, 0, a.H, HeadStore{a.dg}, stream);
        return hipGetLastError();
    }
    bwd_plan(dtype, a);
    float *p = lin_states_place(a, static_cast<float *>(ws), 2);
    if (a.segs > 1)
        if (hipError_t e = launch_lin_states(dtype, a, true, true, a.dg || a.dS0, stream)) return e;
    if (a.dg) {
        const size_t chunks = bh * ((a.T + lin_chunk(dtype) - 1) / lin_chunk(dtype));
        a.chain = reinterpret_cast<double *>(p);
        a.sums = reinterpret_cast<LinSums *>(a.chain + 2 * chunks);
        a.tok = reinterpret_cast<float *>(a.sums + chunks);
        a.edge = a.tok + 3 * bh * a.T;
        a.head = a.edge + bh * 8 * (a.segs + 1);
    }
    return dtype == 1 ? bwd_typed<Bf16>(a, stream) : bwd_typed<F32>(a, stream);
}

}  // namespace qd
