// Linear attention with a decay for each head, forward and single tokens (the formulas and the
// layout of the state are in qd_linattn.h).
//
// Bound by HBM: q, k, v read once, o written once.  A workgroup of four waves walks the chunks of
// one (sequence, head, 64 value columns); the column blocks of a head are put on the same XCD, so
// its L2 serves the second reading of q and k.  Where that leaves the card short of workgroups the
// time axis is cut into segments: a first launch walks each segment but the last from zero, a
// second one joins the segments' states, and the main one starts every segment from its own.
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

template <class P, int DK>
struct FwdLds {
    static constexpr int C = kLinChunk<P>;
    using QK = LinRows<P, C, DK, kNT>;
    using VV = LinRows<P, C, 64, kNT>;
    static constexpr int kPitchP = C + 16 / P::kBytes;
    typename P::R q[QK::kElems], k[QK::kElems], v[VV::kElems], p[C * kPitchP];
    LinGates<C> gates;
};

template <class P, int DK>
__global__ __launch_bounds__(kNT) void lin_fwd_kernel(const LinArgs a) {
    using L = FwdLds<P, DK>;
    constexpr int C = L::C, NB = (C / 16) * (C / 16 + 1) / 2;
    extern __shared__ __align__(16) char smem[];
    L &lds = *reinterpret_cast<L *>(smem);
    const int ncb = a.DV / 64;
    int unit, cb;
    if (!lin_place(a.B * a.H * a.segs, ncb, unit, cb)) return;
    const int seg = unit % a.segs, bh = unit / a.segs, b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), g4 = lane >> 4, r16 = lane & 15;
    const int len = lin_len(a, b);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, (a.T + C - 1) / C);
    const int col = 64 * cb + 16 * wave;
    const size_t sdk = static_cast<size_t>(a.H) * DK * P::kBytes, sdv = static_cast<size_t>(a.H) * a.DV * P::kBytes;
    const size_t tok0 = static_cast<size_t>(b) * a.T;
    const char *gq = static_cast<const char *>(a.q) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
    const char *gk = static_cast<const char *>(a.k) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
    const char *gv = static_cast<const char *>(a.v) + tok0 * sdv + (static_cast<size_t>(h) * a.DV + 64 * cb) * P::kBytes;
    char *go = static_cast<char *>(a.o) + tok0 * sdv + (static_cast<size_t>(h) * a.DV + 64 * cb) * P::kBytes;
    const size_t state = static_cast<size_t>(a.DV) * DK;

    f32x4 S[DK / 16];
    const float *from = seg > 0 ? a.fwd + (static_cast<size_t>(bh) * (a.segs - 1) + seg - 1) * state
                                : a.S0 ? a.S0 + bh * state : nullptr;
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
        S[t] = from ? *reinterpret_cast<const f32x4 *>(from + static_cast<size_t>(col + r16) * DK + 32 * (t >> 1) + 8 * g4 + 4 * (t & 1))
                    : zero4();
    // blocks above the diagonal that a pair of tiles reads: never written again
    for (int e = tid; e < C * L::kPitchP; e += kNT) lds.p[e] = 0;

    typename L::QK rq, rk;
    typename L::VV rv;
    float gate = 0.f;
    auto fetch = [&](int n) {
        const int t0 = n * C, live = min(max(len - t0, 0), C);
        rq.load(gq + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
        rk.load(gk + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
        rv.load(gv + static_cast<size_t>(t0) * sdv, live, static_cast<int>(sdv), tid);
        if (wave == 0) gate = lin_gate(a, b, h, t0, live, lane);
    };
    fetch(c0);
    for (int n = c0; n < c1; ++n) {
        const int t0 = n * C, live = min(max(len - t0, 0), C);
        __syncthreads();
        rq.put(lds.q, tid);
        rk.put(lds.k, tid);
        rv.put(lds.v, tid);
        if (wave == 0) lin_gates(lds.gates, gate, lane);
        __syncthreads();
        if (n + 1 < c1) fetch(n + 1);
        for (int p = wave; p < NB; p += 4) {
            int i, j;
            lin_pair(p, i, j);
            f32x4 acc = lin_block<P, DK>(lds.k, lds.q, L::QK::kPitch, 16 * j, 16 * i, lane);
            const int s = 16 * i + r16, t = 16 * j + 4 * g4;
            const float hs = lds.gates.hi[s], ls = lds.gates.lo[s];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = t + e <= s ? lin_between(lds.gates, hs, ls, t + e) * acc[e] : 0.f;
            P::st4(lds.p + s * L::kPitchP + t, acc);
        }
        __syncthreads();
        typename P::F vf[C / 32][2];
#pragma unroll
        for (int u = 0; u < C / 32; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) vf[u][e] = lin_down<P>(lds.v, L::VV::kPitch, 32 * u + 4 * e, 16 * wave, 4, lane);
        const __amdgpu_buffer_rsrc_t ro = lin_rsrc(go + static_cast<size_t>(t0) * sdv,
                                                   live > 0 ? (live - 1) * static_cast<int>(sdv) + 64 * P::kBytes : 0);
        LinSplit<P, 1> sf[DK / 16];
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) sf[t].of(S[t]);
#pragma unroll
        for (int i = 0; i < C / 16; ++i) {
            f32x4 acc = lin_read<P>(sf, lds.q, L::QK::kPitch, 16 * i, lane);
            acc *= lds.gates.before[16 * i + r16];
#pragma unroll
            for (int u = 0; u <= i / 2; ++u) {
                typename P::F p0, p1;
                frag_oct<P>(lds.p, L::kPitchP, 16 * i, 32 * u, p0, p1, lane);
                acc = P::mma2(acc, vf[u][0], vf[u][1], p0, p1);
            }
            const int row = 16 * i + r16;
            // the end of a buffer is that of its last row: rows past it are dropped by their offset
            lin_store4<P>(ro, row * static_cast<int>(sdv) + (16 * wave + 4 * g4) * P::kBytes, acc);
        }
        lin_update<P, C, 3>(S, lds.k, L::QK::kPitch, vf, lds.gates.after, lds.gates.all[0], lane);
    }
    if (a.S_T && seg == a.segs - 1) {
        float *to = a.S_T + bh * state;
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
            *reinterpret_cast<f32x4 *>(to + static_cast<size_t>(col + r16) * DK + 32 * (t >> 1) + 8 * g4 + 4 * (t & 1)) = S[t];
    }
}

// The states alone, from zero (or S0, dS_T) over one segment: forwards with k, v and the decay to
// the segment's end, backwards with q, do and the decay from its start.
template <class P, int DK>
struct StateLds {
    static constexpr int C = kLinChunk<P>;
    using QK = LinRows<P, C, DK, kNT>;
    using VV = LinRows<P, C, 64, kNT>;
    typename P::R k[QK::kElems], v[VV::kElems];
    LinGates<C> gates;
};
template <class P, int DK>
__global__ __launch_bounds__(kNT) void lin_state_kernel(const LinArgs a, const int first_rev) {
    using L = StateLds<P, DK>;
    constexpr int C = L::C;
    extern __shared__ __align__(16) char smem[];
    L &lds = *reinterpret_cast<L *>(smem);
    const int ncb = a.DV / 64, nseg = a.segs - 1, bhs = a.B * a.H;
    int unit, cb;
    if (!lin_place(bhs * nseg, ncb, unit, cb)) return;
    const bool rev = first_rev + static_cast<int>(blockIdx.y) > 0;
    const int slot = unit % nseg, bh = unit / nseg, b = bh / a.H, h = bh % a.H, seg = rev ? slot + 1 : slot;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), g4 = lane >> 4, r16 = lane & 15;
    const int len = lin_len(a, b);
    const int nc = (a.T + C - 1) / C, c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nc);
    const int col = 64 * cb + 16 * wave;
    const size_t sdk = static_cast<size_t>(a.H) * DK * P::kBytes, sdv = static_cast<size_t>(a.H) * a.DV * P::kBytes;
    const size_t tok0 = static_cast<size_t>(b) * a.T;
    const char *gk = static_cast<const char *>(rev ? a.q : a.k) + tok0 * sdk + static_cast<size_t>(h) * DK * P::kBytes;
    const char *gv = static_cast<const char *>(rev ? a.d_o : a.v) + tok0 * sdv + (static_cast<size_t>(h) * a.DV + 64 * cb) * P::kBytes;
    const size_t state = static_cast<size_t>(a.DV) * DK;

    f32x4 S[DK / 16];
    const float *from = rev ? (seg == a.segs - 1 && a.dS_T ? a.dS_T + bh * state : nullptr)
                            : (seg == 0 && a.S0 ? a.S0 + bh * state : nullptr);
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
        S[t] = from ? *reinterpret_cast<const f32x4 *>(from + static_cast<size_t>(col + r16) * DK + 32 * (t >> 1) + 8 * g4 + 4 * (t & 1))
                    : zero4();
    typename L::QK rk;
    typename L::VV rv;
    float gate = 0.f;
    auto fetch = [&](int n) {
        const int t0 = n * C, live = min(max(len - t0, 0), C);
        rk.load(gk + static_cast<size_t>(t0) * sdk, live, static_cast<int>(sdk), tid);
        rv.load(gv + static_cast<size_t>(t0) * sdv, live, static_cast<int>(sdv), tid);
        if (wave == 0) gate = lin_gate(a, b, h, t0, live, lane);
    };
    double total = 0;
    fetch(rev ? c1 - 1 : c0);
    for (int m = c0; m < c1; ++m) {
        const int n = rev ? c1 - 1 - (m - c0) : m;
        __syncthreads();
        rk.put(lds.k, tid);
        rv.put(lds.v, tid);
        if (wave == 0) total += lin_gates(lds.gates, gate, lane);
        __syncthreads();
        if (m + 1 < c1) fetch(rev ? n - 1 : n + 1);
        typename P::F vf[C / 32][2];
#pragma unroll
        for (int u = 0; u < C / 32; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) vf[u][e] = lin_down<P>(lds.v, L::VV::kPitch, 32 * u + 4 * e, 16 * wave, 4, lane);
        lin_update<P, C, 3>(S, lds.k, L::QK::kPitch, vf, rev ? lds.gates.before : lds.gates.after, lds.gates.all[0], lane);
    }
    float *to = (rev ? a.rev : a.fwd) + (static_cast<size_t>(bh) * nseg + slot) * state;
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
        *reinterpret_cast<f32x4 *>(to + static_cast<size_t>(col + r16) * DK + 32 * (t >> 1) + 8 * g4 + 4 * (t & 1)) = S[t];
    if (cb == 0 && tid == 0) a.fac[(static_cast<size_t>(rev) * bhs + bh) * a.segs + seg] = lin_exp2(static_cast<float>(total));
}

// Local states to states at the borders: forwards slot j becomes the state behind segment j,
// backwards the gradient of the state before segment j + 1.
__global__ __launch_bounds__(kNT) void lin_join_kernel(const LinArgs a, const int first_rev) {
    const bool rev = first_rev + static_cast<int>(blockIdx.y) > 0;
    const int nseg = a.segs - 1, per = a.DV * a.DK / 4, bhs = a.B * a.H;
    const long long idx = static_cast<long long>(blockIdx.x) * kNT + threadIdx.x;
    if (idx >= static_cast<long long>(bhs) * per) return;
    const int bh = static_cast<int>(idx / per);
    f32x4 *p = reinterpret_cast<f32x4 *>((rev ? a.rev : a.fwd)) + static_cast<size_t>(bh) * nseg * per + idx % per;
    const float *fac = a.fac + (static_cast<size_t>(rev) * bhs + bh) * a.segs;
    f32x4 S = p[static_cast<size_t>(rev ? nseg - 1 : 0) * per];
    for (int m = 1; m < nseg; ++m) {
        const int j = rev ? nseg - 1 - m : m;
        S = p[static_cast<size_t>(j) * per] + S * fac[rev ? j + 1 : j];
        p[static_cast<size_t>(j) * per] = S;
    }
}

// ---------------------------------------------------------------- one token
// Bound by the state's reading and writing.  Eight lanes share a row, 128 contiguous bytes a load;
// all of a wave's rows are loaded before any arithmetic:
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

template <class K>
hipError_t lin_launch(K kernel, dim3 grid, size_t lds, hipStream_t stream, const LinArgs &a) {
    hipLaunchKernelGGL(kernel, grid, dim3(kNT), static_cast<unsigned>(lds), stream, a);
    return hipGetLastError();
}

template <class P>
hipError_t fwd_typed(const LinArgs &a, hipStream_t stream) {
    const dim3 grid = lin_grid(static_cast<long long>(a.B) * a.H * a.segs, a.DV / 64);
    if (a.DK == 128) return lin_launch(lin_fwd_kernel<P, 128>, grid, sizeof(FwdLds<P, 128>), stream, a);
    return lin_launch(lin_fwd_kernel<P, 64>, grid, sizeof(FwdLds<P, 64>), stream, a);
}
template <class P>
void states_typed(const LinArgs &a, dim3 grid, int first, hipStream_t stream) {
    if (a.DK == 128) hipLaunchKernelGGL((lin_state_kernel<P, 128>), grid, dim3(kNT), sizeof(StateLds<P, 128>), stream, a, first);
    else hipLaunchKernelGGL((lin_state_kernel<P, 64>), grid, dim3(kNT), sizeof(StateLds<P, 64>), stream, a, first);
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

// Segments of the forward: from two workgroups a compute unit on, the time axis stays whole.
struct LinPlan {
    int segs, seg_chunks;
};
LinPlan fwd_plan(int dtype, int B, int T, int H, int dv) {
    const int C = lin_chunk(dtype);
    const long long units = static_cast<long long>(B) * H * (dv / 64), nc = (static_cast<long long>(T) + C - 1) / C;
    long long segs = 1;
    if (units > 0 && units < 256) segs = 512 / units;
    if (segs > nc / 4) segs = nc / 4;
    if (segs < 1) segs = 1;
    const long long per = nc ? (nc + segs - 1) / segs : 1;
    return LinPlan{static_cast<int>(nc ? (nc + per - 1) / per : 1), static_cast<int>(per)};
}

}  // namespace

bool lin_supported(int dtype, int dk, int dv) {
    return (dtype == 0 || dtype == 1) && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}
// 32-bit row offsets inside a chunk, and grids
bool lin_fits(int B, int T, int H) {
    return H <= (1 << 15) && static_cast<long long>(B) * H < (1LL << 26) && T <= 0x7fffff00;
}

size_t lin_fwd_workspace(int dtype, int B, int T, int H, int dk, int dv) {
    const LinPlan p = fwd_plan(dtype, B, T, H, dv);
    if (p.segs == 1) return 0;
    const size_t bh = static_cast<size_t>(B) * H;
    return (bh * (p.segs - 1) * dk * dv + 2 * bh * p.segs) * sizeof(float);
}

hipError_t launch_lin_states(int dtype, const LinArgs &a, bool fwd, bool rev, hipStream_t stream) {
    const int first = fwd ? 0 : 1, count = (fwd ? 1 : 0) + (rev ? 1 : 0);
    dim3 grid = lin_grid(static_cast<long long>(a.B) * a.H * (a.segs - 1), a.DV / 64);
    grid.y = count;
    if (dtype == 1) states_typed<Bf16>(a, grid, first, stream);
    else states_typed<F32>(a, grid, first, stream);
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
    const LinPlan p = fwd_plan(dtype, a.B, a.T, a.H, a.DV);
    a.segs = p.segs;
    a.seg_chunks = p.seg_chunks;
    if (p.segs > 1) {
        a.fwd = static_cast<float *>(ws);
        a.fac = a.fwd + bh * (p.segs - 1) * state;
        if (hipError_t e = launch_lin_states(dtype, a, true, false, stream)) return e;
    }
    return dtype == 1 ? fwd_typed<Bf16>(a, stream) : fwd_typed<F32>(a, stream);
}

hipError_t launch_lin_step(int dtype, const LinArgs &a, float *S, hipStream_t stream) {
    return dtype == 1 ? step_typed<Bf16>(a, S, stream) : step_typed<F32>(a, S, stream);
}

}  // namespace qd
