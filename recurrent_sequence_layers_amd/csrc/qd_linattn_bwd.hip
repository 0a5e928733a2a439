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
// Every term is one that g_t scales: no difference of large sums.  The walks write a, b and
// x_t = sum_{s>t} M[s][t] - sum_{i<t} M[t][i], whose prefix sums are the third term, and c comes
// from a chain over the chunks: with E_n = <S, R> behind chunk n, c_n = E_n - sum b and
// E_{n-1} = c_n + sum a, from E = <S_T, dS_T> on.  a and b are taken before anything is rounded
// (the state split as in qd_linattn.h), since dg is fp32.
#include "qd_internal.h"
#include "qd_linattn.h"

namespace qd {
namespace {

template <class P, int DK, int DV>
struct BwdLds {
    static constexpr int C = kLinChunk<P>, NW = (DK > DV ? DK : DV) / 16, NT = 64 * NW;
    static constexpr int NB = (C / 16) * (C / 16 + 1) / 2;
    using QK = LinRows<P, C, DK, NT>;
    using VV = LinRows<P, C, DV, NT>;
    LinTile<P, C, DK> q, k;
    LinTile<P, C, DV> v, o;
    LinTile<P, C, C> p[2];
    LinGates<C> gates;
    float rows[NB][16], cols[NB][16];  // strict row and column sums of M's blocks
    float part[NW][C];                 // a or b, by the columns' wave
};

// Where a walk reads and writes.
template <class P, int DK, int DV>
struct Walk {
    using L = BwdLds<P, DK, DV>;
    static constexpr int C = L::C, NT = L::NT;
    const LinArgs &a;
    int b, h, bh, seg, c0, c1, len, tid, wave, lane, g4, r16;
    size_t sdk, sdv;
    const char *gq, *gk, *gv, *go;
    typename L::QK rq, rk;
    typename L::VV rv, ro;
    float gate = 0.f;

    __device__ __forceinline__ Walk(const LinArgs &a_, int unit) : a(a_) {
        seg = unit % a.segs;
        bh = unit / a.segs;
        b = bh / a.H;
        h = bh % a.H;
        tid = threadIdx.x;
        wave = lin_wave();
        lane = lane_id();
        g4 = lane >> 4;
        r16 = lane & 15;
        len = lin_len(a, b);
        c0 = seg * a.seg_chunks;
        c1 = min(c0 + a.seg_chunks, (a.T + C - 1) / C);
        sdk = static_cast<size_t>(a.H) * DK * P::kBytes;
        sdv = static_cast<size_t>(a.H) * DV * P::kBytes;
        gq = static_cast<const char *>(a.q) + at(0, sdk, DK);
        gk = static_cast<const char *>(a.k) + at(0, sdk, DK);
        gv = static_cast<const char *>(a.v) + at(0, sdv, DV);
        go = static_cast<const char *>(a.d_o) + at(0, sdv, DV);
    }
    __device__ __forceinline__ size_t at(int t, size_t stride, int d) const {
        return (static_cast<size_t>(b) * a.T + t) * stride + static_cast<size_t>(h) * d * P::kBytes;
    }
    __device__ __forceinline__ int live(int n) const { return min(max(len - n * C, 0), C); }
    __device__ __forceinline__ void fetch(int n) {
        const int t0 = n * C, rows = live(n);
        rq.load(gq + static_cast<size_t>(t0) * sdk, rows, static_cast<int>(sdk), tid);
        rk.load(gk + static_cast<size_t>(t0) * sdk, rows, static_cast<int>(sdk), tid);
        rv.load(gv + static_cast<size_t>(t0) * sdv, rows, static_cast<int>(sdv), tid);
        ro.load(go + static_cast<size_t>(t0) * sdv, rows, static_cast<int>(sdv), tid);
        if (wave == 0) gate = lin_gate(a, b, h, t0, rows, lane);
    }
    __device__ __forceinline__ void put(L &lds) const {
        rq.put(lds.q, tid);
        rk.put(lds.k, tid);
        rv.put(lds.v, tid);
        ro.put(lds.o, tid);
        if (wave == 0) lin_gates(lds.gates, gate, lane);
    }
    // Output rows of chunk n, padding's included: they are written as zeros
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t out(void *base, int n, size_t stride, int d) const {
        const int rows = min(a.T - n * C, C);
        return lin_rsrc(static_cast<char *>(base) + at(n * C, stride, d), (rows - 1) * static_cast<int>(stride) + d * P::kBytes);
    }
    __device__ __forceinline__ float *tok(int which, int n) const {
        return a.tok + (static_cast<size_t>(which) * a.B * a.H + bh) * a.T + n * C;
    }
};

// a or b of one row: the product of the state's part with the row's own q or k, summed over columns
template <class P, int C, int D>
__device__ __forceinline__ void row_part(float *part, LinTile<P, C, D> &rows, int row, int col, f32x4 acc, int lane) {
    const f32x4 y = P::f32(P::ld4(rows.four(row, col)));
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(acc[e], y[e], s);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) part[row] = s;
}
__device__ __forceinline__ float sum16(float x) {
    x += dpp_src<0xB1, 0xf>(x);    // quad_perm 1,0,3,2
    x += dpp_src<0x4E, 0xf>(x);    // quad_perm 2,3,0,1
    x += dpp_src<0x141, 0xf>(x);   // row_half_mirror
    return x + dpp_src<0x140, 0xf>(x);   // row_mirror
}

// ---------------------------------------------------------------- dq, forwards
template <class P, int DK, int DV, bool DG>
__device__ __forceinline__ void dq_walk(const LinArgs &a, BwdLds<P, DK, DV> &lds, int unit) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NB = L::NB, NW = L::NW, KC = DK / 16;
    Walk<P, DK, DV> w(a, unit);
    const int wave = w.wave, lane = w.lane, g4 = w.g4, r16 = w.r16;
    const bool mine = wave < KC;
    const size_t state = static_cast<size_t>(DV) * DK;
    const int col = 16 * wave + r16;             // key column of the state
    f32x4 S[DV / 16];
    const float *from = w.seg > 0 ? a.fwd + (static_cast<size_t>(w.bh) * (a.segs - 1) + w.seg - 1) * state
                                  : a.S0 ? a.S0 + w.bh * state : nullptr;
#pragma unroll
    for (int t = 0; t < DV / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[t][e] = from && mine ? from[(lin_row(t, lane) + e) * DK + col] : 0.f;
    for (int e = w.tid; e < LinTile<P, C, C>::kElems; e += L::NT) lds.p[0].m[e] = 0;
    w.fetch(w.c0);
    for (int n = w.c0; n < w.c1; ++n) {
        __syncthreads();
        w.put(lds);
        __syncthreads();
        if (n + 1 < w.c1) w.fetch(n + 1);
        const int live = w.live(n);
        for (int p = wave; p < NB; p += NW) {
            int i, j;
            lin_pair(p, i, j);
            f32x4 acc = lin_block<P>(lds.v, lds.o, 16 * j, 16 * i, lane);
            const int s = 16 * i + r16, t = 16 * j + 4 * g4;
            const f32x4 d = lin_between(lds.gates, s, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = t + e <= s ? d[e] * acc[e] : 0.f;
            P::st4(lds.p[0].four(s, t), acc);
            if constexpr (DG) {
                const f32x4 qk = lin_block<P>(lds.k, lds.q, 16 * j, 16 * i, lane);
                float row = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float m = t + e < s ? acc[e] * qk[e] : 0.f;
                    row += m;
                    const float c = sum16(m);
                    if (r16 == 0) lds.cols[p][4 * g4 + e] = c;
                }
                row += __shfl_xor(row, 16);
                row += __shfl_xor(row, 32);
                if (lane < 16) lds.rows[p][r16] = row;
            }
        }
        __syncthreads();
        if (mine) {
            typename P::F kf[C / 32][2];
#pragma unroll
            for (int u = 0; u < C / 32; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) kf[u][e] = lds.k.down(u, e, 16 * wave, lane);
            LinSplit<P, DG ? 3 : 1> sf[DV / 16];
#pragma unroll
            for (int t = 0; t < DV / 16; ++t) sf[t].of(S[t]);
            const __amdgpu_buffer_rsrc_t rs = w.out(a.dq, n, w.sdk, DK);
#pragma unroll
            for (int i = 0; i < C / 16; ++i) {
                const int row = 16 * i + r16;
                f32x4 acc = lin_read<P>(sf, lds.o, 16 * i, lane);
                acc *= lds.gates.before[row];
                if constexpr (DG) row_part<P>(lds.part[wave], lds.q, row, 16 * wave + 4 * g4, acc, lane);
#pragma unroll
                for (int u = 0; u <= i / 2; ++u) {
                    typename P::F p0, p1;
                    lds.p[0].oct(16 * i, u, lane, p0, p1);
                    acc = P::mma2(acc, kf[u][0], kf[u][1], p0, p1);
                }
                lin_store4<P>(rs, row * static_cast<int>(w.sdk) + (16 * wave + 4 * g4) * P::kBytes, row < live ? acc : zero4());
            }
            lin_update<P, C, 3, DV>(S, lds.v, kf, lds.gates.after, lds.gates.all[0], lane);
        }
        if constexpr (DG) {
            __syncthreads();
            if (w.tid < C && n * C + w.tid < a.T) {
                const int i = w.tid >> 4, r = w.tid & 15;
                float x = 0.f, s = 0.f;
                for (int m = i; m < C / 16; ++m) x += lds.cols[m * (m + 1) / 2 + i][r];
                for (int m = 0; m <= i; ++m) x -= lds.rows[i * (i + 1) / 2 + m][r];
#pragma unroll
                for (int m = 0; m < KC; ++m) s += lds.part[m][w.tid];
                w.tok(0, n)[w.tid] = x;
                w.tok(1, n)[w.tid] = s;
            }
        }
    }
    if constexpr (DG) {
        if (w.seg == a.segs - 1) {               // <S_T, dS_T>
            float s = 0.f;
            if (a.dS_T && mine) {
                const float *d = a.dS_T + w.bh * state;
#pragma unroll
                for (int t = 0; t < DV / 16; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s = fmaf(S[t][e], d[(lin_row(t, lane) + e) * DK + col], s);
            }
            for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
            if (lane == 0) a.edge[static_cast<size_t>(w.bh) * 8 + wave] = s;
        }
    }
}

// ---------------------------------------------------------------- dk and dv, backwards
template <class P, int DK, int DV, bool DG>
__device__ __forceinline__ void dkv_walk(const LinArgs &a, BwdLds<P, DK, DV> &lds, int unit) {
    using L = BwdLds<P, DK, DV>;
    constexpr int C = L::C, NB = L::NB, NW = L::NW, KC = DK / 16, VC = DV / 16;
    Walk<P, DK, DV> w(a, unit);
    const int wave = w.wave, lane = w.lane, g4 = w.g4, r16 = w.r16;
    const bool mine_k = wave < KC, mine_v = wave < VC;
    const size_t state = static_cast<size_t>(DV) * DK;
    const int col = 16 * wave + r16;
    f32x4 Rv[KC], Rk[VC];                        // columns are value indices; key indices
    const float *from = w.seg < a.segs - 1 ? a.rev + (static_cast<size_t>(w.bh) * (a.segs - 1) + w.seg) * state
                                           : a.dS_T ? a.dS_T + w.bh * state : nullptr;
#pragma unroll
    for (int t = 0; t < KC; ++t)
        Rv[t] = from && mine_v ? *reinterpret_cast<const f32x4 *>(from + col * DK + lin_row(t, lane)) : zero4();
#pragma unroll
    for (int t = 0; t < VC; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            Rk[t][e] = from && mine_k ? from[(lin_row(t, lane) + e) * DK + col] : 0.f;
    for (int e = w.tid; e < LinTile<P, C, C>::kElems; e += L::NT) lds.p[0].m[e] = lds.p[1].m[e] = 0;
    w.fetch(w.c1 - 1);
    for (int n = w.c1 - 1; n >= w.c0; --n) {
        __syncthreads();
        w.put(lds);
        __syncthreads();
        if (n > w.c0) w.fetch(n - 1);
        const int live = w.live(n);
        // by the earlier token t's row: p[0] for dv, p[1] for dk
        for (int p = wave; p < NB; p += NW) {
            int i, j;
            lin_pair(p, i, j);                        // s in block i, t in block j
            const int t = 16 * j + r16, s = 16 * i + 4 * g4;
            f32x4 qk = lin_block<P>(lds.q, lds.k, 16 * i, 16 * j, lane);
            f32x4 ov = lin_block<P>(lds.o, lds.v, 16 * i, 16 * j, lane);
            const f32x4 hi = lds_f32x4(lds.gates.hi + s) - lds.gates.hi[t], lo = lds_f32x4(lds.gates.lo + s) - lds.gates.lo[t];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = lin_exp2(hi[e] + lo[e]);
                qk[e] = t <= s + e ? d * qk[e] : 0.f;
                ov[e] = t <= s + e ? d * ov[e] : 0.f;
            }
            P::st4(lds.p[0].four(t, s), qk);
            P::st4(lds.p[1].four(t, s), ov);
        }
        __syncthreads();
        if (mine_v) {
            typename P::F of[C / 32][2];
#pragma unroll
            for (int u = 0; u < C / 32; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) of[u][e] = lds.o.down(u, e, 16 * wave, lane);
            LinSplit<P, 1> sf[KC];
#pragma unroll
            for (int t = 0; t < KC; ++t) sf[t].of(Rv[t]);
            const __amdgpu_buffer_rsrc_t rs = w.out(a.dv, n, w.sdv, DV);
#pragma unroll
            for (int i = 0; i < C / 16; ++i) {
                const int row = 16 * i + r16;
                f32x4 acc = lin_read<P>(sf, lds.k, 16 * i, lane);
                acc *= lds.gates.after[row];
#pragma unroll
                for (int u = i / 2; u < C / 32; ++u) {
                    typename P::F p0, p1;
                    lds.p[0].oct(16 * i, u, lane, p0, p1);
                    acc = P::mma2(acc, of[u][0], of[u][1], p0, p1);
                }
                lin_store4<P>(rs, row * static_cast<int>(w.sdv) + (16 * wave + 4 * g4) * P::kBytes, row < live ? acc : zero4());
            }
            lin_update<P, C, 2, DK>(Rv, lds.q, of, lds.gates.before, lds.gates.all[0], lane);
        }
        if (mine_k) {
            typename P::F qf[C / 32][2];
#pragma unroll
            for (int u = 0; u < C / 32; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) qf[u][e] = lds.q.down(u, e, 16 * wave, lane);
            LinSplit<P, DG ? 3 : 1> sf[VC];
#pragma unroll
            for (int t = 0; t < VC; ++t) sf[t].of(Rk[t]);
            const __amdgpu_buffer_rsrc_t rs = w.out(a.dk, n, w.sdk, DK);
#pragma unroll
            for (int i = 0; i < C / 16; ++i) {
                const int row = 16 * i + r16;
                f32x4 acc = lin_read<P>(sf, lds.v, 16 * i, lane);
                acc *= lds.gates.after[row];
                if constexpr (DG) row_part<P>(lds.part[wave], lds.k, row, 16 * wave + 4 * g4, acc, lane);
#pragma unroll
                for (int u = i / 2; u < C / 32; ++u) {
                    typename P::F p0, p1;
                    lds.p[1].oct(16 * i, u, lane, p0, p1);
                    acc = P::mma2(acc, qf[u][0], qf[u][1], p0, p1);
                }
                lin_store4<P>(rs, row * static_cast<int>(w.sdk) + (16 * wave + 4 * g4) * P::kBytes, row < live ? acc : zero4());
            }
            lin_update<P, C, 3, DV>(Rk, lds.o, qf, lds.gates.before, lds.gates.all[0], lane);
        }
        if constexpr (DG) {
            __syncthreads();
            if (w.tid < C && n * C + w.tid < a.T) {
                float s = 0.f;
#pragma unroll
                for (int m = 0; m < KC; ++m) s += lds.part[m][w.tid];
                w.tok(2, n)[w.tid] = s;
            }
        }
    }
    if (a.dS0 && w.seg == 0 && mine_k) {
        float *to = a.dS0 + w.bh * state;
#pragma unroll
        for (int t = 0; t < VC; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) to[(lin_row(t, lane) + e) * DK + col] = Rk[t][e];
    }
}

template <class P, int DK, int DV, bool DG>
__global__ __launch_bounds__(64 * ((DK > DV ? DK : DV) / 16)) LIN_TWO_WAVES void lin_bwd_kernel(const LinArgs a) {
    extern __shared__ __align__(16) char smem[];
    auto &lds = *reinterpret_cast<BwdLds<P, DK, DV> *>(smem);
    const int unit = blockIdx.x >> 1;
    if (blockIdx.x & 1) dq_walk<P, DK, DV, DG>(a, lds, unit);
    else dkv_walk<P, DK, DV, DG>(a, lds, unit);
}

// ---------------------------------------------------------------- dg
// One workgroup a (sequence, head): the chain of c over the chunks from the last, 64 at a time, a
// chunk a wave.  Bound by the latency of its few passes over three numbers a token.
constexpr int kDgWaves = 16, kDgChunks = 512;
template <int C>
__global__ __launch_bounds__(64 * kDgWaves) void lin_dg_kernel(const LinArgs a) {
    __shared__ double sa[kDgChunks], sb[kDgChunks];
    __shared__ double carry, wsum[kDgWaves];
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, wave = wave_id(), lane = lane_id();
    const size_t bhs = static_cast<size_t>(a.B) * a.H;
    const float *x = a.tok + static_cast<size_t>(bh) * a.T, *ta = x + bhs * a.T, *tb = ta + bhs * a.T;
    const int len = lin_len(a, b), nc = (a.T + C - 1) / C;
    auto get = [&](const float *p, int n, int i) { return i < C && n * C + i < a.T ? p[n * C + i] : 0.f; };
    if (threadIdx.x == 0) {
        double e = 0;
        for (int w = 0; w < (a.DK > a.DV ? a.DK : a.DV) / 16; ++w) e += a.edge[static_cast<size_t>(bh) * 8 + w];
        carry = e;
    }
    double total = 0;
    for (int last = nc; last > 0; last -= kDgChunks) {
        const int first = max(last - kDgChunks, 0), count = last - first;
        for (int m = wave; m < count; m += kDgWaves) {
            float va = get(ta, first + m, lane), vb = get(tb, first + m, lane);
            for (int d = 1; d < 64; d *= 2) {
                va += __shfl_xor(va, d);
                vb += __shfl_xor(vb, d);
            }
            if (lane == 0) {
                sa[m] = va;
                sb[m] = vb;
            }
        }
        __syncthreads();
        if (wave == 0) {
            // c_n = E + sum of (a - b) over later chunks - b_n; a lane's chunks are consecutive, from the last on
            constexpr int PER = kDgChunks / 64;
            double d[PER], mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int m = count - 1 - (lane * PER + i);
                d[i] = m >= 0 ? sa[m] - sb[m] : 0.0;
                mine += d[i];
            }
            double run = mine;
            for (int s = 1; s < 64; s *= 2) {
                const double y = __shfl_up(run, s);
                if (lane >= s) run += y;
            }
            double e = carry + run - mine;
            const double end = carry + __shfl(run, 63);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int m = count - 1 - (lane * PER + i);
                if (m >= 0) sa[m] = e - sb[m];
                e += d[i];
            }
            if (lane == 0) carry = end;
        }
        __syncthreads();
        for (int m = wave; m < count; m += kDgWaves) {
            const int n = first + m;
            const float y = get(x, n, lane) + get(tb, n, lane);
            const float before = wave_inclusive_sum(y) - y;
            const float back = wave_inclusive_sum(get(ta, n, 63 - lane));
            const float behind = __shfl(back, 63 - lane);
            const int t = n * C + lane;
            if (lane < C && t < a.T) {
                const float v = t < len ? static_cast<float>(sa[m] + static_cast<double>(before + behind)) : 0.f;
                if (a.decay == kTokenDecay) a.dg[(static_cast<size_t>(b) * a.T + t) * a.H + h] = v;
                else total += v;
            }
        }
        __syncthreads();
    }
    if (a.decay == kHeadDecay) {
        for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
        if (lane == 0) wsum[wave] = total;
        __syncthreads();
        if (threadIdx.x == 0) {
            double s = 0;
            for (int w = 0; w < kDgWaves; ++w) s += wsum[w];
            a.head[bh] = static_cast<float>(s);
        }
    }
}
__global__ __launch_bounds__(256) void lin_dg_head_kernel(const LinArgs a) {
    const int h = blockIdx.x * 256 + threadIdx.x;
    if (h >= a.H) return;
    double s = 0;
    for (int b = 0; b < (a.T ? a.B : 0); ++b) s += a.head[static_cast<size_t>(b) * a.H + h];
    a.dg[h] = static_cast<float>(s);
}

template <class P, int DK, int DV>
hipError_t bwd_sized(const LinArgs &a, hipStream_t stream) {
    using L = BwdLds<P, DK, DV>;
    static_assert(sizeof(L) <= 160 * 1024, "LDS of a workgroup");
    const dim3 grid(static_cast<unsigned>(2LL * a.B * a.H * a.segs)), blk(L::NT);
    if (a.dg) hipLaunchKernelGGL((lin_bwd_kernel<P, DK, DV, true>), grid, blk, sizeof(L), stream, a);
    else hipLaunchKernelGGL((lin_bwd_kernel<P, DK, DV, false>), grid, blk, sizeof(L), stream, a);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.dg) {
        hipLaunchKernelGGL(lin_dg_kernel<L::C>, dim3(static_cast<unsigned>(a.B * a.H)), dim3(64 * kDgWaves), 0, stream, a);
        if (a.decay == kHeadDecay) hipLaunchKernelGGL(lin_dg_head_kernel, dim3((a.H + 255) / 256), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}
template <class P>
hipError_t bwd_typed(const LinArgs &a, hipStream_t stream) {
    if (a.DK == 128) return a.DV == 128 ? bwd_sized<P, 128, 128>(a, stream) : bwd_sized<P, 128, 64>(a, stream);
    return a.DV == 128 ? bwd_sized<P, 64, 128>(a, stream) : bwd_sized<P, 64, 64>(a, stream);
}

// Both walks of every head are 2 B H workgroups, one a compute unit; fewer than the card has cut
// the time axis.
void bwd_plan(int dtype, int B, int T, int H, int &segs, int &seg_chunks) {
    const int C = lin_chunk(dtype);
    const long long units = 2LL * B * H, nc = (static_cast<long long>(T) + C - 1) / C;
    long long s = units > 0 ? 256 / units : 1;
    if (s > nc / 4) s = nc / 4;
    if (s < 1) s = 1;
    const long long per = nc ? (nc + s - 1) / s : 1;
    segs = static_cast<int>(nc ? (nc + per - 1) / per : 1);
    seg_chunks = static_cast<int>(per);
}

}  // namespace

size_t lin_bwd_workspace(int dtype, int B, int T, int H, int dk, int dv, bool dg) {
    if (static_cast<long long>(B) * H * T == 0) return 0;
    int segs, per;
    bwd_plan(dtype, B, T, H, segs, per);
    const size_t bh = static_cast<size_t>(B) * H;
    size_t n = 0;
    if (segs > 1) n += 2 * bh * (segs - 1) * dk * dv + 2 * bh * segs;
    if (dg) n += 3 * bh * T + 9 * bh;
    return n * sizeof(float);
}

hipError_t launch_lin_bwd(int dtype, LinArgs a, void *ws, hipStream_t stream) {
    const size_t bh = static_cast<size_t>(a.B) * a.H, state = static_cast<size_t>(a.DV) * a.DK;
    if (a.T == 0 || bh == 0) {
        // no tokens: dS0 = dS_T, and sums over tokens are zero
        if (a.dS0 && bh)
            if (hipError_t e = launch_lin_copy(a.dS0, a.dS_T, bh * state, stream)) return e;
        if (a.dg && a.decay == kHeadDecay && a.H) {
            a.T = 0;
            hipLaunchKernelGGL(lin_dg_head_kernel, dim3((a.H + 255) / 256), dim3(256), 0, stream, a);
        }
        return hipGetLastError();
    }
    bwd_plan(dtype, a.B, a.T, a.H, a.segs, a.seg_chunks);
    float *p = static_cast<float *>(ws);
    if (a.segs > 1) {
        a.fwd = p;
        a.rev = a.fwd + bh * (a.segs - 1) * state;
        a.fac = a.rev + bh * (a.segs - 1) * state;
        p = a.fac + 2 * bh * a.segs;
        if (hipError_t e = launch_lin_states(dtype, a, true, true, a.dg || a.dS0, stream)) return e;
    }
    if (a.dg) {
        a.tok = p;
        a.edge = a.tok + 3 * bh * a.T;
        a.head = a.edge + 8 * bh;
    }
    return dtype == 1 ? bwd_typed<Bf16>(a, stream) : bwd_typed<F32>(a, stream);
}

}  // namespace qd
