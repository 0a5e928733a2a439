// Linear attention with a decay for each head, forward and single tokens (the formulas and the
// layout of the state are in qd_linattn.h).
//
// Bound by HBM: q, k, v read once, o written once.  A workgroup walks the chunks of one (sequence,
// head, 64 value columns): four waves hold the state, sixteen columns each, and four more bring what
// they need.  The column blocks of a head are put on the same XCD, so its L2 serves the second
// reading of q and k.  8 x 4096 tokens, 16 heads, 128 x 128, bf16 (539 MB): 129 to 135 us, 4.0 to 4.2
// TB/s of the 4.9 that a copy reaches; the same loads, barriers and stores without the products take
// 127.  Four waves that load, compute and store in turn took 294 us, the two roles 179, and outputs in
// whole rows instead of eight bytes a lane 149 where they had been 175.
//
// Where (sequence, head, column block) leaves the card short of workgroups the time axis is cut into
// segments: a first launch walks each segment but the last from zero, a second one joins the
// segments' states, and the main one starts every segment from its own.  65536 tokens of 16 heads:
// 1617 us uncut, 402 to 414 cut in eight, 138 of them for the states, which read k and v once more.
#include "qd_internal.h"
#include "qd_linattn.h"

namespace qd {
namespace {

constexpr int kNT = 256;             // four waves, 64 columns

// Block index -> (unit, column block): the ncb blocks of a unit are 8 apart, on the same XCD.
__device__ __forceinline__ bool lin_place(int units, int ncb, int &unit, int &cb) {
    const int x = blockIdx.x & 7, y = blockIdx.x >> 3;
    cb = y % ncb;
    unit = (y / ncb) * 8 + x;
    return unit < units;
}
dim3 lin_grid(long long units, int ncb) { return dim3(static_cast<unsigned>((units + 7) / 8 * 8 * ncb)); }

// Eight waves in two roles, a barrier a step.  At step n waves 0-3 hold the state and do chunk n's
// part with it: the outputs, then the state's update.  Waves 4-7 are ahead of them: they bring chunk
// n + 2 from the registers, where the loads of two steps before put it, to LDS.  All of them form P of
// chunk n + 1, two blocks of a row at a time, shared so that the roles take equally long.
template <class P, int DK>
struct FwdLds {
    static constexpr int C = kLinChunk<P>;
    LinTile<P, C, DK> q[3], k[3];
    LinTile<P, C, 64> v[3], o[2];
    LinTile<P, C, C> p[2];
    LinGates<C> gates[3];
};

// Blocks J .. J + N - 1 of row I of P, all in flight at once.  low: what the bf16 of it rounds away
template <class P, int I, int J, int N, int C, int D>
__device__ __forceinline__ void lin_products(LinTile<P, C, D> &q, LinTile<P, C, D> &k, const LinGates<C> &gates, LinTile<P, C, C> &to,
                                             LinTile<P, C, C> *low, const LinLane &l) {
    static_assert(I < C / 16 && J + N - 1 <= I, "the lower triangle");
    f32x4 x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = zero4();
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        typename P::F q0, q1, k0[N], k1[N];
        q.oct(I, u, l, q0, q1);
#pragma unroll
        for (int n = 0; n < N; ++n) k.oct(J + n, u, l, k0[n], k1[n]);
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = P::mma2(x[n], k0[n], k1[n], q0, q1);
    }
    const int s = 16 * I + (l.lane & 15);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int t = 16 * (J + n) + 4 * (l.lane >> 4);
        const f32x4 d = lin_between(gates, s, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = J + n < I || t + e <= s ? d[e] * x[n][e] : 0.f;
        P::st4(to.four(I, J + n, l), x[n]);
        if (P::kBytes == 2 && low) P::st4(low->four(I, J + n, l), x[n] - P::f32(P::cvt(x[n])));
    }
}
// A wave's share of them: the loading waves (role 1) take seven of ten, the states' waves three. With
// all ten on the loading waves the size above takes 144 us, and seven prompts of up to 1900 tokens,
// 12 heads, 46 instead of 38 (other lengths up to 1900: up to 42). In fp32, where the states' waves
// have more to do, the loading waves take all three.
template <class P, int C, int D>
__device__ __forceinline__ void lin_share(int role, int wave, LinTile<P, C, D> &q, LinTile<P, C, D> &k, const LinGates<C> &gates,
                                          LinTile<P, C, C> &to, LinTile<P, C, C> *low, const LinLane &l) {
    if constexpr (C == 64) {
        if (role == 1) {
            if (wave == 0) lin_products<P, 3, 0, 2>(q, k, gates, to, low, l);
            else if (wave == 1) lin_products<P, 3, 2, 2>(q, k, gates, to, low, l);
            else if (wave == 2) lin_products<P, 2, 0, 2>(q, k, gates, to, low, l);
            else lin_products<P, 2, 2, 1>(q, k, gates, to, low, l);
        } else {
            if (wave == 0) lin_products<P, 1, 0, 1>(q, k, gates, to, low, l);
            else if (wave == 1) lin_products<P, 1, 1, 1>(q, k, gates, to, low, l);
            else if (wave == 2) lin_products<P, 0, 0, 1>(q, k, gates, to, low, l);
        }
    } else if (role == 1) {
        if (wave == 0) lin_products<P, 1, 0, 1>(q, k, gates, to, low, l);
        else if (wave == 1) lin_products<P, 1, 1, 1>(q, k, gates, to, low, l);
        else if (wave == 2) lin_products<P, 0, 0, 1>(q, k, gates, to, low, l);
    }
}

template <class P, int DK, int NS>
__global__ __launch_bounds__(2 * kNT) LIN_TWO_WAVES void lin_fwd_kernel(const LinArgs a) {
    using L = FwdLds<P, DK>;
    constexpr int C = L::C;
    extern __shared__ __align__(16) char smem[];
    L &lds = *reinterpret_cast<L *>(smem);
    const int ncb = a.DV / 64;
    int unit, cb;
    if (!lin_place(a.B * a.H * a.segs, ncb, unit, cb)) return;
    const int seg = unit % a.segs, bh = unit / a.segs, b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x & (kNT - 1), role = lin_wave() >> 2, wave = lin_wave() & 3, lane = lane_id(), r16 = lane & 15;
    const LinLane l(lane);
    const int len = lin_len(a, b);
    // a sequence that ends before the segment leaves it without chunks
    const int c0 = seg * a.seg_chunks, c1 = max(c0, min(c0 + a.seg_chunks, (len + C - 1) / C));
    if (c1 == c0 && !(a.S_T && seg == a.segs - 1)) return;
    // in one chunk P is a sum of two: over few tokens its roundings would not average out, and the
    // other chunks' tile is free
    const bool few = c1 - c0 == 1;
    const size_t sdk = static_cast<size_t>(a.H) * DK * P::kBytes, sdv = static_cast<size_t>(a.H) * a.DV * P::kBytes;
    const size_t tok0 = static_cast<size_t>(b) * a.T;
    const size_t vcol = (static_cast<size_t>(h) * a.DV + 64 * cb) * P::kBytes;

    // blocks above the diagonal that a pair of tiles reads: never written again
    for (int e = threadIdx.x; e < LinTile<P, C, C>::kElems; e += 2 * kNT) lds.p[0].m[e] = lds.p[1].m[e] = 0;
    __syncthreads();

    if (role == 1) {
        const char *gq = static_cast<const char *>(a.q) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
        const char *gk = static_cast<const char *>(a.k) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
        const char *gv = static_cast<const char *>(a.v) + tok0 * sdv + vcol;
        char *go = static_cast<char *>(a.o) + tok0 * sdv + vcol;
        // two chunks on their way: the loads of one step are waited for two steps later
        struct Ahead {
            LinRows<P, C, DK, kNT> q, k;
            LinRows<P, C, 64, kNT> v;
            float gate;
        } even, odd;
        auto fetch = [&](Ahead &r, int n) {
            const int t0 = n * C, live = n < c1 ? min(max(len - t0, 0), C) : 0;
            r.q.load(gq + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
            r.k.load(gk + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
            r.v.load(gv + static_cast<size_t>(t0) * sdv, live, static_cast<int>(sdv), tid);
            r.gate = lin_gate(a, b, h, t0, live, lane);
        };
        int put = 0, now = 2;                    // slots of chunks n + 2 and n + 1
        auto step = [&](Ahead &r, int n) {
            // the outputs of chunk n - 1; rows past the buffer's end, that of the last token's row,
            // are dropped by their offset
            const int t0 = max(n - 1, c0) * C, live = n > c0 && n <= c1 ? min(max(len - t0, 0), C) : 0;
            lin_store<P, C, 64, kNT>(lds.o[(n - 1 - c0) & 1],
                                     lin_rsrc(go + static_cast<size_t>(t0) * sdv,
                                              live > 0 ? (live - 1) * static_cast<int>(sdv) + 64 * P::kBytes : 0),
                                     static_cast<int>(sdv), tid);
            // also past the last chunk, with zeros: a branch here would make the waits for one
            // chunk's loads wait for the next one's too
            r.q.put(lds.q[put], tid);
            r.k.put(lds.k[put], tid);
            r.v.put(lds.v[put], tid);
            if (wave == 3) lin_gates(lds.gates[put], r.gate, lane);
            fetch(r, n + 4);
            if (n + 1 >= c0 && n + 1 < c1)
                lin_share<P>(1, wave, lds.q[now], lds.k[now], lds.gates[now], lds.p[(n + 1 - c0) & 1], few ? &lds.p[1] : nullptr, l);
            now = put;
            put = put == 2 ? 0 : put + 1;
            __syncthreads();
        };
        fetch(even, c0);
        fetch(odd, c0 + 1);
        for (int n = c0 - 2; n <= c1; n += 2) {
            step(even, n);
            step(odd, n + 1);
        }
        return;
    }

    const size_t state = static_cast<size_t>(a.DV) * DK;
    const int col = 64 * cb + 16 * wave + r16;
    f32x4 S[1][DK / 16];
    lin_load<DK>(S[0], lin_before(a, bh, seg), col, lane);
    __syncthreads();
    if (c0 < c1) lin_share<P>(0, wave, lds.q[0], lds.k[0], lds.gates[0], lds.p[0], few ? &lds.p[1] : nullptr, l);
    __syncthreads();
    int now = 0;
    for (int n = c0; n < c1; ++n) {
        LinTile<P, C, DK> &q = lds.q[now], &k = lds.k[now];
        LinTile<P, C, C> &p = lds.p[(n - c0) & 1];
        const LinGates<C> &gates = lds.gates[now];
        if (n + 1 < c1) {
            const int next = now == 2 ? 0 : now + 1;
            lin_share<P>(0, wave, lds.q[next], lds.k[next], lds.gates[next], lds.p[(n + 1 - c0) & 1], few ? &lds.p[1] : nullptr, l);
        }
        typename P::F vf[1][C / 32][2];
        lin_columns<P, C>(vf, lds.v[now], wave, l);
        f32x4 acc[1][C / 16];
        lin_read<P, 1>(acc, S, q, l);
#pragma unroll
        for (int i = 0; i < C / 16; ++i) acc[0][i] *= gates.before[16 * i + r16];
        lin_near<P, true>(acc, p, vf, l);
        if (P::kBytes == 2 && few) lin_near<P, true>(acc, lds.p[1], vf, l);
#pragma unroll
        for (int i = 0; i < C / 16; ++i) P::st4(lds.o[(n - c0) & 1].four(i, wave, l), acc[0][i]);
        lin_update<P, C, NS>(S, k, vf, gates.after, gates.all[0], l);
        now = now == 2 ? 0 : now + 1;
        __syncthreads();
    }
    __syncthreads();                             // the last chunk's outputs go in a step of their own
    if (!((c1 - c0) & 1)) __syncthreads();       // and that role goes by pairs of steps
    if (a.S_T && seg == a.segs - 1) lin_keep<DK>(S[0], a.S_T + bh * state, col, lane);
}

// The states alone, from zero (or S0, dS_T) over one piece of a segment: forwards with k, v and the
// decay to the piece's end, backwards with q, do and the decay from its start.  Four waves; the
// next chunk goes to LDS while this one is used.  Short of HBM's rate: 470 MB of the 65536 tokens above
// at 3.4 TB/s with three addends, 3.8 with two; vector units 40 % busy, matrix units 28 %.
template <class P, int DK>
struct StateLds {
    static constexpr int C = kLinChunk<P>;
    LinTile<P, C, DK> k[2];
    LinTile<P, C, 64> v[2];
    LinGates<C> gates[2];
};
template <class P, int DK, int NS>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(3, 3))) void lin_state_kernel(const LinArgs a, const int first_rev) {
    using L = StateLds<P, DK>;
    constexpr int C = L::C;
    extern __shared__ __align__(16) char smem[];
    L &lds = *reinterpret_cast<L *>(smem);
    const int ncb = a.DV / 64, slots = (a.segs - 1) * a.subs, bhs = a.B * a.H;
    int unit, cb;
    if (!lin_place(bhs * slots, ncb, unit, cb)) return;
    const bool rev = first_rev + static_cast<int>(blockIdx.y) > 0;
    const int slot = unit % slots, bh = unit / slots, b = bh / a.H, h = bh % a.H, piece = rev ? slot + a.subs : slot;
    const int tid = threadIdx.x, wave = lin_wave(), lane = lane_id(), r16 = lane & 15;
    const LinLane l(lane);
    const int len = lin_len(a, b);
    const int c0 = piece / a.subs * a.seg_chunks + piece % a.subs * a.sub_chunks, nc = (len + C - 1) / C;
    const int count = max(0, min(min(a.sub_chunks, a.seg_chunks - piece % a.subs * a.sub_chunks), nc - c0));
    const size_t sdk = static_cast<size_t>(a.H) * DK * P::kBytes, sdv = static_cast<size_t>(a.H) * a.DV * P::kBytes;
    const size_t tok0 = static_cast<size_t>(b) * a.T;
    const char *gk = static_cast<const char *>(rev ? a.q : a.k) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
    const char *gv = static_cast<const char *>(rev ? a.d_o : a.v) + tok0 * sdv + (static_cast<size_t>(h) * a.DV + 64 * cb) * P::kBytes;
    const size_t state = static_cast<size_t>(a.DV) * DK;
    const int col = 64 * cb + 16 * wave + r16;

    f32x4 S[1][DK / 16];
    const bool first = rev ? slot == slots - 1 : slot == 0;
    const float *from = rev ? a.dS_T : a.S0;
    lin_load<DK>(S[0], first && from ? from + bh * state : nullptr, col, lane);
    if (first && !rev && a.entry) lin_keep<DK>(S[0], a.entry + bh * state, col, lane);
    LinRows<P, C, DK, kNT> rk;
    LinRows<P, C, 64, kNT> rv;
    float gate = 0.f;
    double total = 0;
    auto fetch = [&](int m) {
        const int t0 = (rev ? c0 + count - 1 - m : c0 + m) * C, live = min(max(len - t0, 0), C);
        rk.load(gk + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
        rv.load(gv + static_cast<size_t>(t0) * sdv, live, static_cast<int>(sdv), tid);
        if (wave == 3) gate = lin_gate(a, b, h, t0, live, lane);
    };
    auto put = [&](int m) {
        rk.put(lds.k[m & 1], tid);
        rv.put(lds.v[m & 1], tid);
        if (wave == 3) total += lin_gates(lds.gates[m & 1], gate, lane);
    };
    if (count > 0) {
        fetch(0);
        put(0);
        if (count > 1) fetch(1);
    }
    __syncthreads();
    for (int m = 0; m < count; ++m) {
        if (m + 1 < count) {
            put(m + 1);
            if (m + 2 < count) fetch(m + 2);
        }
        const LinGates<C> &gates = lds.gates[m & 1];
        typename P::F vf[1][C / 32][2];
        lin_columns<P, C>(vf, lds.v[m & 1], wave, l);
        lin_update<P, C, NS>(S, lds.k[m & 1], vf, rev ? gates.before : gates.after, gates.all[0], l);
        __syncthreads();
    }
    lin_keep<DK>(S[0], (rev ? a.rev : a.fwd) + (static_cast<size_t>(bh) * slots + slot) * state, col, lane);
    if (cb == 0 && wave == 3 && lane == 0)
        a.fac[(static_cast<size_t>(rev) * bhs + bh) * slots + slot] = lin_exp2(static_cast<float>(0.5 * total));
}

// The pieces' own states to the states at the segments' borders: forwards slot j becomes the state
// behind piece j, backwards the gradient of the state before its piece; written where a segment
// begins.  Eight pieces are on their way at a time.  A piece's decay is there as its root: it may
// lie beyond fp32 where its product with a state does not.
__global__ __launch_bounds__(kNT) void lin_join_kernel(const LinArgs a, const int first_rev) {
    constexpr int AHEAD = 8;
    const bool rev = first_rev + static_cast<int>(blockIdx.y) > 0;
    const int slots = (a.segs - 1) * a.subs, per = a.DV * a.DK / 4, bhs = a.B * a.H;
    const long long idx = static_cast<long long>(blockIdx.x) * kNT + threadIdx.x;
    if (idx >= static_cast<long long>(bhs) * per) return;
    const int bh = static_cast<int>(idx / per);
    f32x4 *p = reinterpret_cast<f32x4 *>(rev ? a.rev : a.fwd) + static_cast<size_t>(bh) * slots * per + idx % per;
    const float *fac = a.fac + (static_cast<size_t>(rev) * bhs + bh) * slots;
    f32x4 S = zero4();
    for (int m = 0; m < slots; m += AHEAD) {
        f32x4 x[AHEAD];
        float f[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int j = rev ? slots - 1 - min(m + k, slots - 1) : min(m + k, slots - 1);
            x[k] = p[static_cast<size_t>(j) * per];
            f[k] = fac[j];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (m + k >= slots) break;
            const int j = rev ? slots - 1 - (m + k) : m + k;
            S = m + k == 0 ? x[k] : x[k] + S * f[k] * f[k];
            if ((rev ? j : j + 1) % a.subs == 0) p[static_cast<size_t>(j) * per] = S;
        }
    }
}

// ---------------------------------------------------------------- one token
// Bound by the state's reading and writing: 541 MB of 256 sequences x 16 heads in 104 us, 5.2 TB/s (82
// where part of the states is still in the Infinity Cache).  One sequence is a launch, 4.3 us.  Eight
// lanes share a row, 128 contiguous bytes a load; all of a wave's rows are loaded before any
// arithmetic:
//   s_j <- e^g s_j + v_j k,   o_j = e^g (s_j . q) + v_j (k . q)
template <class P, int DK, int DV>
__global__ __launch_bounds__(kNT) void lin_step_kernel(const LinArgs a, float *__restrict__ states) {
    using R = typename P::R;
    constexpr int LPR = 8, NG = DK / (4 * LPR), ROWS = DV / 4, NPASS = ROWS / (kWave / LPR);
    const size_t nh = blockIdx.x;
    const int lane = lane_id(), wave = wave_id(), sub = lane % LPR, grp = lane / LPR;
    const R *gq = static_cast<const R *>(a.q) + nh * DK, *gk = static_cast<const R *>(a.k) + nh * DK;
    const R *gv = static_cast<const R *>(a.v) + nh * DV;
    R *go = static_cast<R *>(a.o) + nh * DV;
    float *S = states + nh * DV * DK;
    f32x4 s[NPASS][NG];
#pragma unroll
    for (int p = 0; p < NPASS; ++p)
#pragma unroll
        for (int m = 0; m < NG; ++m)
            s[p][m] = *reinterpret_cast<const f32x4 *>(S + (wave * ROWS + p * (kWave / LPR) + grp) * DK + 4 * (m * LPR + sub));
    const float x = a.decay == kNoDecay ? 0.f : a.decay == kHeadDecay ? a.g[nh % a.H] : a.g[nh];
    const float decay = lin_exp(x);
    f32x4 kk[NG], qq[NG];
    float kq = 0.f;
#pragma unroll
    for (int m = 0; m < NG; ++m) {
        kk[m] = P::f32(P::ld4(gk + 4 * (m * LPR + sub)));
        qq[m] = P::f32(P::ld4(gq + 4 * (m * LPR + sub)));
#pragma unroll
        for (int i = 0; i < 4; ++i) kq = fmaf(kk[m][i], qq[m][i], kq);
    }
    auto sum8 = [](float v) {
        v += __shfl_xor(v, 1, LPR);
        v += __shfl_xor(v, 2, LPR);
        return v + __shfl_xor(v, 4, LPR);
    };
    kq = sum8(kq);
#pragma unroll
    for (int p = 0; p < NPASS; ++p) {
        const int row = wave * ROWS + p * (kWave / LPR) + grp;
        const float vj = P::to_f32(gv[row]);
        float c = 0.f;
#pragma unroll
        for (int m = 0; m < NG; ++m) {
            f32x4 ns;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c = fmaf(s[p][m][i], qq[m][i], c);
                ns[i] = fmaf(vj, kk[m][i], decay * s[p][m][i]);
            }
            *reinterpret_cast<f32x4 *>(S + row * DK + 4 * (m * LPR + sub)) = ns;
        }
        c = sum8(c);
        if (sub == 0) go[row] = P::from_f32(fmaf(vj, kq, decay * c));
    }
}

__global__ __launch_bounds__(kNT) void lin_copy_kernel(f32x4 *to, const f32x4 *from, size_t n) {
    for (size_t i = static_cast<size_t>(blockIdx.x) * kNT + threadIdx.x; i < n; i += static_cast<size_t>(gridDim.x) * kNT)
        to[i] = from ? from[i] : zero4();
}

template <class P, int DK>
void fwd_sized(const LinArgs &a, hipStream_t stream) {
    const dim3 grid = lin_grid(static_cast<long long>(a.B) * a.H * a.segs, a.DV / 64), blk(2 * kNT);
    if (a.S_T) hipLaunchKernelGGL((lin_fwd_kernel<P, DK, 3>), grid, blk, sizeof(FwdLds<P, DK>), stream, a);
    else hipLaunchKernelGGL((lin_fwd_kernel<P, DK, 2>), grid, blk, sizeof(FwdLds<P, DK>), stream, a);
}
template <class P>
hipError_t fwd_typed(const LinArgs &a, hipStream_t stream) {
    if (a.DK == 128) fwd_sized<P, 128>(a, stream);
    else fwd_sized<P, 64>(a, stream);
    return hipGetLastError();
}
template <class P, int DK>
void states_sized(const LinArgs &a, dim3 grid, int first, bool exact, hipStream_t stream) {
    if (exact) hipLaunchKernelGGL((lin_state_kernel<P, DK, 3>), grid, dim3(kNT), sizeof(StateLds<P, DK>), stream, a, first);
    else hipLaunchKernelGGL((lin_state_kernel<P, DK, 2>), grid, dim3(kNT), sizeof(StateLds<P, DK>), stream, a, first);
}
template <class P>
void states_typed(const LinArgs &a, dim3 grid, int first, bool exact, hipStream_t stream) {
    if (a.DK == 128) states_sized<P, 128>(a, grid, first, exact, stream);
    else states_sized<P, 64>(a, grid, first, exact, stream);
}
template <class P>
hipError_t step_typed(const LinArgs &a, float *S, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.B) * a.H), blk(kNT);
    if (a.DK == 128 && a.DV == 128) hipLaunchKernelGGL((lin_step_kernel<P, 128, 128>), grid, blk, 0, stream, a, S);
    else if (a.DK == 128) hipLaunchKernelGGL((lin_step_kernel<P, 128, 64>), grid, blk, 0, stream, a, S);
    else if (a.DV == 128) hipLaunchKernelGGL((lin_step_kernel<P, 64, 128>), grid, blk, 0, stream, a, S);
    else hipLaunchKernelGGL((lin_step_kernel<P, 64, 64>), grid, blk, 0, stream, a, S);
    return hipGetLastError();
}

}  // namespace

bool lin_supported(int dtype, int dk, int dv) {
    return (dtype == 0 || dtype == 1) && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}
// Row offsets inside a chunk stay within 31 bits, and launches within 2^32 threads: of the walks,
// 256 threads a head for a token, 1024 forwards, 1536 backwards, and of dg, 1024 a chunk.
bool lin_fits(int dtype, int B, int T, int H, LinCall call) {
    const long long lim = (1LL << 32) - (1 << 16), per = call == kLinStep ? 256 : call == kLinFwd ? 1024 : 1536;
    const long long chunks = B * ((static_cast<long long>(T) + lin_chunk(dtype) - 1) / lin_chunk(dtype));
    return H <= (1 << 15) && T <= 0x7fff0000 && static_cast<long long>(B) * H * per < lim &&
           (call != kLinBwd || chunks * 1024 < lim);
}

// A walk of n chunks takes n + 3 steps, workgroups go in rounds of one a compute unit, and cutting
// the axis costs two launches (about five steps) and the states: a chunk of a piece costs
// state_cost of a step, three workgroups a compute unit side by side.  Uncut and cut, in us: forward
// 2048 x 16 heads 50 and 29, 2 x 4096 x 16 96 and 57; gradients 2048 x 8 heads 165 and 49, 2 x 1024 x
// 16 89 and 56, 4096 x 4 heads of 64 x 64 in fp32 442 and 41.  A sequence of seven chunks is left
// whole.  Pieces: as long as their segments, 65536 x 16 takes 504 us instead of 414, 2 x 4096 x 16 63
// instead of 57.
void lin_plan(int dtype, LinArgs &a, long long units, int directions, double state_cost) {
    const long long C = lin_chunk(dtype), nc = (a.T + C - 1) / C, cus = 256;
    double best = 0;
    a.segs = 1;
    a.seg_chunks = static_cast<int>(nc);
    for (long long want = 1; want <= 64 && want * 4 <= nc + 3; ++want) {
        const long long per = (nc + want - 1) / want, segs = (nc + per - 1) / per;
        const double rounds = static_cast<double>((units * segs + cus - 1) / cus);
        double cost = rounds * (per + 3);
        if (segs > 1) cost += 5 + state_cost * units * per * (segs - 1) / cus;
        if (want == 1 || cost < best) {
            best = cost;
            a.segs = static_cast<int>(segs);
            a.seg_chunks = static_cast<int>(per);
        }
    }
    a.subs = 1;
    a.sub_chunks = a.seg_chunks;
    if (a.segs > 1) {
        const long long walks = static_cast<long long>(a.B) * a.H * (a.DV / 64) * (a.segs - 1) * directions;
        long long subs = 3 * cus / walks;
        if (subs > a.seg_chunks / 4) subs = a.seg_chunks / 4;
        if (subs > 1) {
            a.sub_chunks = static_cast<int>((a.seg_chunks + subs - 1) / subs);
            a.subs = (a.seg_chunks + a.sub_chunks - 1) / a.sub_chunks;
        }
    }
}
size_t lin_states_floats(const LinArgs &a, int directions) {
    if (a.segs == 1) return 0;
    const size_t slots = static_cast<size_t>(a.B) * a.H * (a.segs - 1) * a.subs;
    return directions * slots * a.DK * a.DV + (2 * slots + 3) / 4 * 4;
}
float *lin_states_place(LinArgs &a, float *ws, int directions) {
    if (a.segs == 1) return ws;
    const size_t n = static_cast<size_t>(a.B) * a.H * (a.segs - 1) * a.subs * a.DK * a.DV;
    a.fwd = ws;
    a.rev = ws + n;
    a.fac = ws + directions * n;
    return ws + lin_states_floats(a, directions);
}

namespace {
// A step with the state alone takes half of one with the outputs.
void fwd_plan(int dtype, LinArgs &a) { lin_plan(dtype, a, static_cast<long long>(a.B) * a.H * (a.DV / 64), 1, 0.5); }
}  // namespace

size_t lin_fwd_workspace(int dtype, int B, int T, int H, int dk, int dv) {
    LinArgs a{};
    a.B = B; a.T = T; a.H = H; a.DK = dk; a.DV = dv;
    fwd_plan(dtype, a);
    return (lin_states_floats(a, 1) + (a.segs > 1 ? static_cast<size_t>(B) * H * dk * dv : 0)) * sizeof(float);
}

hipError_t launch_lin_states(int dtype, const LinArgs &a, bool fwd, bool rev, bool exact, hipStream_t stream) {
    const int first = fwd ? 0 : 1, count = (fwd ? 1 : 0) + (rev ? 1 : 0);
    dim3 grid = lin_grid(static_cast<long long>(a.B) * a.H * (a.segs - 1) * a.subs, a.DV / 64);
    grid.y = count;
    if (dtype == 1) states_typed<Bf16>(a, grid, first, exact, stream);
    else states_typed<F32>(a, grid, first, exact, stream);
    const long long n = static_cast<long long>(a.B) * a.H * (a.DV * a.DK / 4);
    hipLaunchKernelGGL(lin_join_kernel, dim3(static_cast<unsigned>((n + kNT - 1) / kNT), count), dim3(kNT), 0, stream, a, first);
    return hipGetLastError();
}

hipError_t launch_lin_copy(float *to, const float *from, size_t n, hipStream_t stream) {
    const size_t blocks = (n / 4 + kNT - 1) / kNT;
    hipLaunchKernelGGL(lin_copy_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(kNT), 0, stream,
                       reinterpret_cast<f32x4 *>(to), reinterpret_cast<const f32x4 *>(from), n / 4);
    return hipGetLastError();
}

hipError_t launch_lin_fwd(int dtype, LinArgs a, void *ws, hipStream_t stream) {
    const size_t bh = static_cast<size_t>(a.B) * a.H, state = static_cast<size_t>(a.DV) * a.DK;
    if (a.T == 0) return a.S_T && a.S_T != a.S0 ? launch_lin_copy(a.S_T, a.S0, bh * state, stream) : hipSuccess;
    fwd_plan(dtype, a);
    float *entry = lin_states_place(a, static_cast<float *>(ws), 1);
    if (a.segs > 1) {
        // a last segment may be done before a first one begins
        if (a.S_T && a.S_T == a.S0) a.entry = entry;
        if (hipError_t e = launch_lin_states(dtype, a, true, false, a.S_T != nullptr, stream)) return e;
        if (a.entry) a.S0 = a.entry;
    }
    return dtype == 1 ? fwd_typed<Bf16>(a, stream) : fwd_typed<F32>(a, stream);
}

hipError_t launch_lin_step(int dtype, const LinArgs &a, float *S, hipStream_t stream) {
    return dtype == 1 ? step_typed<Bf16>(a, S, stream) : step_typed<F32>(a, S, stream);
}

}  // namespace qd
