// Short causal depthwise convolution for gfx950, channels last, with an optional SiLU:
//
//   pre[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - W + 1 + j, c],   y = pre or silu(pre)
//
// Rows before the sequence come from the state S0 (the W - 1 inputs before the first, oldest
// first), or are zero; S_T is the same window at the sequence's end.  The gradients are
//
//   dpre = dy f'(pre),  dx[t, c] = sum_j w[c, j] dpre[t + W - 1 - j, c],
//   dw[c, j] = sum_{b, t} dpre[t, c] x[t - W + 1 + j, c],  dbias[c] = sum_{b, t} dpre[t, c].
//
// Every element is read once and written once: the kernels are bound by HBM.  A thread owns
// kVec channels over a run of TL tokens and keeps the last W - 1 rows in registers, so a row
// is loaded once for all W taps; consecutive threads take consecutive channel vectors, so a
// wave's load covers 512 or 1024 contiguous bytes of a row.  Channel counts that kVec does not
// divide take one channel a thread.  At 8 x 4096 x 2048 bf16, W = 4: forward 62 us (268 MB, 4.3
// TB/s), backward 98 us (403 MB, 4.1 TB/s), 118 with lens.  These figures and those below are of one
// build: a call among others over three sets of inputs, the median of five runs.
#include "qd_internal.h"
#include "qd_mixer.h"

namespace qd {
namespace {

constexpr int kThreads = 256;
// Channels a thread: 8 bytes of bf16, 16 of fp32.  Eight bf16 channels (16 bytes) take twice the
// registers: forward 67 us against 62, backward 102 against 98 (with lens 102 against 118).  Two fp32
// channels, at four sequences: forward 59 against 55 us, backward 92 against 94.
constexpr int kVec = 4;
// Rows loaded before they are used: forward 62 us with eight, 66 with four; backward, which
// holds two rows for each and more registers besides, 109 with eight and 98 with four.
constexpr int kAhead = 8, kAheadBwd = 4;

// Row t of a sequence with its history: t < 0 comes from the state (or is zero).
template <class P, int V>
__device__ __forceinline__ void row_or_state(const typename P::R *x, const typename P::R *s0, int t, int W, size_t D,
                                             float (&v)[V]) {
    if (t >= 0) {
        load_vec<P, V>(x + static_cast<size_t>(t) * D, v);
    } else if (s0) {
        load_vec<P, V>(s0 + static_cast<size_t>(t + W - 1) * D, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <class P, int V, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(const ConvArgs a) {
    using R = typename P::R;
    const int nvec = a.D / V, ntile = max(1, (a.T + a.TL - 1) / a.TL);
    const long long idx = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (idx >= static_cast<long long>(a.B) * ntile * nvec) return;
    const int vec = static_cast<int>(idx % nvec);
    const int bt = static_cast<int>(idx / nvec);
    const int b = bt / ntile, tile = bt % ntile;
    const size_t D = a.D;
    const int c = vec * V;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const R *x = static_cast<const R *>(a.x) + static_cast<size_t>(b) * a.T * D + c;
    const R *s0 = a.S0 ? static_cast<const R *>(a.S0) + static_cast<size_t>(b) * (W - 1) * D + c : nullptr;
    R *y = static_cast<R *>(a.y) + static_cast<size_t>(b) * a.T * D + c;

    const int t0 = tile * a.TL, t1 = min(t0 + a.TL, len);
    if (t0 < t1) {
        float w[W][V], bias[V], win[W][V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = a.w[static_cast<size_t>(c + i) * W + j];
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) row_or_state<P, V>(x, s0, t0 - (W - 1) + k, W, D, win[k]);
        for (int t = t0; t < t1; t += kAhead) {
            float in[kAhead][V];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load_vec<P, V>(x + static_cast<size_t>(min(t + k, t1 - 1)) * D, in[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[W - 1][i] = in[k][i];
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                    out[i] = a.silu ? siluf(p) : p;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
                }
                if (t + k < t1) store_vec<P, V>(y + static_cast<size_t>(t + k) * D, out);
            }
        }
    }
    // The thread of the first tile, the only reader of the state, writes the new one: S_T may be S0.
    if (tile == 0 && a.S_T) {
        R *st = static_cast<R *>(a.S_T) + static_cast<size_t>(b) * (W - 1) * D + c;
        float v[W - 1][V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) row_or_state<P, V>(x, s0, len - (W - 1) + k, W, D, v[k]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_vec<P, V>(st + static_cast<size_t>(k) * D, v[k]);
    }
}

// A block covers NX channel vectors times 256 / NX runs of TL tokens; its threads' sums for
// dw and dbias are joined in LDS in a fixed order and written as one row of partial results.
// LENS: sequences end at their lengths.  A length is a register more in every lane, which at four
// taps takes a wave of four from each SIMD (136 registers against 128): 118 against 98 us.
template <class P, int V, int W, bool LENS>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(const ConvBwdArgs a) {
    using R = typename P::R;
    __shared__ float red[kThreads][V];
    const int nvec = a.D / V, ntile = (a.T + a.TL - 1) / a.TL;
    const int vx = threadIdx.x & (a.NX - 1), ty = threadIdx.x / a.NX, NY = kThreads / a.NX;
    const int nbx = (nvec + a.NX - 1) / a.NX, bx = blockIdx.x % nbx, by = blockIdx.x / nbx;
    const int vec = bx * a.NX + vx;
    const long long run = static_cast<long long>(by) * NY + ty;
    const bool live = vec < nvec && run < static_cast<long long>(a.B) * ntile;
    const size_t D = a.D;
    const int c = vec * V;
    float dw[W][V] = {}, db[V] = {};
    if (live) {
        const int b = static_cast<int>(run / ntile), tile = static_cast<int>(run % ntile);
        const R *x = static_cast<const R *>(a.x) + static_cast<size_t>(b) * a.T * D + c;
        const R *dy = static_cast<const R *>(a.dy) + static_cast<size_t>(b) * a.T * D + c;
        const R *s0 = a.S0 ? static_cast<const R *>(a.S0) + static_cast<size_t>(b) * (W - 1) * D + c : nullptr;
        const R *dst = a.dS_T ? static_cast<const R *>(a.dS_T) + static_cast<size_t>(b) * (W - 1) * D + c : nullptr;
        R *dx = static_cast<R *>(a.dx) + static_cast<size_t>(b) * a.T * D + c;
        R *ds0 = a.dS0 ? static_cast<R *>(a.dS0) + static_cast<size_t>(b) * (W - 1) * D + c : nullptr;
        float w[W][V], bias[V], win[W][V] = {}, dp[W][V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = a.w[static_cast<size_t>(c + i) * W + j];
        }
        const int len = LENS ? min(max(a.lens[b], 0), a.T) : a.T;
        const int t0 = tile * a.TL, t1 = max(min(t0 + a.TL, len), t0);
        if (t0 < len) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) row_or_state<P, V>(x, s0, t0 - (W - 1) + k, W, D, win[k]);
        }
        // At step t the window holds x[t-W+1 .. t] and dp the gradients dpre[t-W+1 .. t]; the
        // finished row is t - (W - 1): rows t0 .. t1-1 need t up to t1 + W - 2.  The first run
        // also finishes the rows before the sequence, which are the state's, also of one that
        // has no tokens: then the rows loaded are not used.
        const int end = t0 < t1 || tile == 0 ? t1 + W - 1 : t0;
        for (int tb = t0; tb < end; tb += kAheadBwd) {
            float in[kAheadBwd][V], gy[kAheadBwd][V];
#pragma unroll
            for (int k = 0; k < kAheadBwd; ++k) {
                const int tc = max(min(tb + k, len - 1), 0);
                load_vec<P, V>(x + static_cast<size_t>(tc) * D, in[k]);
                load_vec<P, V>(dy + static_cast<size_t>(tc) * D, gy[k]);
            }
            float cw[W][V] = {}, cb[V] = {};        // sums of these four rows, added to the run's below
#pragma unroll
            for (int k = 0; k < kAheadBwd; ++k) {
                const int t = tb + k, tr = t - (W - 1);
                const bool in_seq = t < len, mine = t < t1;
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[W - 1][i] = in[k][i];
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                    const float g = a.silu ? gy[k][i] * dsiluf(p) : gy[k][i];
                    dp[W - 1][i] = in_seq ? g : 0.f;
                    if (mine) {
                        cb[i] += g;
#pragma unroll
                        for (int j = 0; j < W; ++j) cw[j][i] = fmaf(g, win[j][i], cw[j][i]);
                    }
                    float s = 0.f;                   // w[W-1] dpre[tr] + ... + w[0] dpre[tr + W - 1]
#pragma unroll
                    for (int j = 0; j < W; ++j) s = fmaf(w[W - 1 - j][i], dp[j][i], s);
                    out[i] = s;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j][i] = win[j + 1][i];
                        dp[j][i] = dp[j + 1][i];
                    }
                }
                const bool row = tr >= t0 && tr < t1, state = tile == 0 && tr < 0 && ds0;
                if (row || state) {
                    const int ts = tr - (len - (W - 1));        // the row's place in the final state
                    if (dst && ts >= 0) {
                        float e[V];
                        load_vec<P, V>(dst + static_cast<size_t>(ts) * D, e);
#pragma unroll
                        for (int i = 0; i < V; ++i) out[i] += e[i];
                    }
                    if (row) store_vec<P, V>(dx + static_cast<size_t>(tr) * D, out);
                    else store_vec<P, V>(ds0 + static_cast<size_t>(tr + W - 1) * D, out);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                db[i] += cb[i];
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][i] += cw[j][i];
            }
        }
        const float none[V] = {};
        for (int t = t1; LENS && t < min(t0 + a.TL, a.T); ++t) store_vec<P, V>(dx + static_cast<size_t>(t) * D, none);   // padding
    }
    float *part = a.part + static_cast<size_t>(by) * (W + 1) * D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        if (j) __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) red[threadIdx.x][i] = j < W ? dw[j < W ? j : 0][i] : db[i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.NX * V; e += kThreads) {
            const int cx = bx * a.NX * V + e;
            if (cx < a.D) {
                float s = 0.f;
                for (int r = 0; r < NY; ++r) s += red[r * a.NX + e / V][e % V];
                part[static_cast<size_t>(j) * D + cx] = s;
            }
        }
    }
}

// Rows before the sequence when it has no tokens: the final state is the initial one.
template <class P>
__global__ __launch_bounds__(kThreads) void conv_bwd_empty_kernel(const ConvBwdArgs a) {
    using R = typename P::R;
    const size_t n = static_cast<size_t>(a.B) * (a.W - 1) * a.D, i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    for (size_t j = i; j < n && a.dS0; j += static_cast<size_t>(gridDim.x) * kThreads)
        static_cast<R *>(a.dS0)[j] = a.dS_T ? static_cast<const R *>(a.dS_T)[j] : P::from_f32(0.f);
    if (i < static_cast<size_t>(a.D) * a.W) a.dw[i] = 0.f;
    if (i < static_cast<size_t>(a.D) && a.dbias) a.dbias[i] = 0.f;
}

struct ConvStore {
    float *dw, *dbias;
    int D, W;
    __device__ __forceinline__ void operator()(long long c, float v) const {
        const int j = static_cast<int>(c / D), d = static_cast<int>(c % D);
        if (j < W) dw[static_cast<size_t>(d) * W + j] = v;
        else if (dbias) dbias[d] = v;
    }
};

int vec_of(int D) {
    return D % kVec == 0 ? kVec : 1;
}

template <class P, int V>
hipError_t fwd_w(const ConvArgs &a, hipStream_t stream) {
    const long long n = static_cast<long long>(a.B) * max(1, (a.T + a.TL - 1) / a.TL) * (a.D / V);
    const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads)), blk(kThreads);
    if (a.W == 2) hipLaunchKernelGGL((conv_fwd_kernel<P, V, 2>), grid, blk, 0, stream, a);
    else if (a.W == 3) hipLaunchKernelGGL((conv_fwd_kernel<P, V, 3>), grid, blk, 0, stream, a);
    else hipLaunchKernelGGL((conv_fwd_kernel<P, V, 4>), grid, blk, 0, stream, a);
    return hipGetLastError();
}

template <class P, int V, int W>
void bwd_l(const ConvBwdArgs &a, dim3 grid, dim3 blk, hipStream_t stream) {
    if (a.lens) hipLaunchKernelGGL((conv_bwd_kernel<P, V, W, true>), grid, blk, 0, stream, a);
    else hipLaunchKernelGGL((conv_bwd_kernel<P, V, W, false>), grid, blk, 0, stream, a);
}
template <class P, int V>
hipError_t bwd_w(const ConvBwdArgs &a, hipStream_t stream) {
    const int nvec = a.D / V;
    const dim3 grid(static_cast<unsigned>((nvec + a.NX - 1) / a.NX) * a.R), blk(kThreads);
    if (a.W == 2) bwd_l<P, V, 2>(a, grid, blk, stream);
    else if (a.W == 3) bwd_l<P, V, 3>(a, grid, blk, stream);
    else bwd_l<P, V, 4>(a, grid, blk, stream);
    column_sum(a.part, a.R, static_cast<long long>(a.W + 1) * a.D, ConvStore{a.dw, a.dbias, a.D, a.W}, stream);
    return hipGetLastError();
}

struct BwdPlan {
    int TL, NX, R;
};
// TL tokens a thread: long runs read fewer rows twice (the W - 1 rows on either side of a
// run) and leave fewer partial sums, short ones fill the card.  At the size above 32 tokens take
// 102 us, 64 take 98 and 128 take 112; in fp32, at four sequences, 102, 94 and 94.
BwdPlan bwd_plan(int B, int T, int D) {
    const int nvec = D / vec_of(D);
    BwdPlan p;
    p.NX = 8;
    while (p.NX < 64 && p.NX < nvec) p.NX *= 2;
    p.TL = 64;
    while (p.TL > 8 && static_cast<long long>(B) * ((T + p.TL - 1) / p.TL) * nvec < 131072) p.TL /= 2;
    const long long runs = static_cast<long long>(B) * ((T + p.TL - 1) / p.TL);
    const int NY = kThreads / p.NX;
    p.R = static_cast<int>((runs + NY - 1) / NY);
    return p;
}

// Tokens a thread walks in the forward: long runs read fewer rows twice, short ones fill the
// card.  At the size above 16 tokens take 63 us, 32 take 62 and 64 take 60; in fp32, at four
// sequences, all three 55.
int fwd_run(int B, int T, int D) {
    int TL = 32;
    while (TL > 4 && static_cast<long long>(B) * ((T + TL - 1) / TL) * (D / vec_of(D)) < 262144) TL /= 2;
    return TL;
}

}  // namespace

// The backward's runs are at least eight tokens, and its workgroups up to 32 runs of up to 64
// channel vectors.
bool conv_fits(int B, int T, int D) {
    const long long rows = static_cast<long long>(B) * T, nvec = D / vec_of(D);
    const long long runs = static_cast<long long>(B) * max(1, (T + 7) / 8);
    return rows < (1LL << 31) && D < (1 << 25) && (runs + 31) * ((nvec + 63) / 64 * 64) < (1LL << 32);
}

hipError_t launch_conv_fwd(int dtype, const ConvArgs &args, hipStream_t stream) {
    ConvArgs a = args;
    const int V = vec_of(a.D);
    a.TL = fwd_run(a.B, a.T, a.D);
    if (dtype == 1) return V == kVec ? fwd_w<Bf16, kVec>(a, stream) : fwd_w<Bf16, 1>(a, stream);
    return V == kVec ? fwd_w<F32, kVec>(a, stream) : fwd_w<F32, 1>(a, stream);
}

hipError_t launch_conv_step(int dtype, const ConvArgs &a, hipStream_t stream) { return launch_conv_fwd(dtype, a, stream); }

size_t conv_bwd_workspace(int B, int T, int D, int W) {
    if (static_cast<long long>(B) * T * D == 0) return 0;
    return static_cast<size_t>(bwd_plan(B, T, D).R) * (W + 1) * D * sizeof(float);
}

hipError_t launch_conv_bwd(int dtype, const ConvBwdArgs &args, hipStream_t stream) {
    ConvBwdArgs a = args;
    if (static_cast<long long>(a.B) * a.T == 0) {
        const dim3 grid(static_cast<unsigned>((static_cast<size_t>(a.D) * a.W + kThreads - 1) / kThreads)), blk(kThreads);
        if (dtype == 1) hipLaunchKernelGGL((conv_bwd_empty_kernel<Bf16>), grid, blk, 0, stream, a);
        else hipLaunchKernelGGL((conv_bwd_empty_kernel<F32>), grid, blk, 0, stream, a);
        return hipGetLastError();
    }
    const BwdPlan p = bwd_plan(a.B, a.T, a.D);
    a.TL = p.TL; a.NX = p.NX; a.R = p.R;
    const int V = vec_of(a.D);
    if (dtype == 1) return V == kVec ? bwd_w<Bf16, kVec>(a, stream) : bwd_w<Bf16, 1>(a, stream);
    return V == kVec ? bwd_w<F32, kVec>(a, stream) : bwd_w<F32, 1>(a, stream);
}

}  // namespace qd
