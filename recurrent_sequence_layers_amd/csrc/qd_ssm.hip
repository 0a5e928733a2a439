// Selective state space scan for gfx950.  Per sequence, channel d and state n:
//
//   delta_t = softplus(dt_t + dt_bias)      (or dt_t + dt_bias itself)
//   h_t[n]  = exp(delta_t A[d, n]) h_{t-1}[n] + delta_t u_t B_t[n]
//   o_t     = (sum_n C_t[n] h_t[n] + D_d u_t) silu(z_t)
//
// with B and C shared by the channels of a group.  One exponential and four multiply-adds a
// token, channel and state against four to eight bytes a token and channel: the vector
// units bound it, not HBM.  The decay differs by channel and state, so there is no matrix
// product in it; the design keeps everything else off the vector units:
//   - a lane owns one channel and a wave NS of its N states, so the recurrence and the sum
//     over the wave's states need no exchange between lanes, and B_t and C_t are the same
//     for all lanes: they come through the scalar cache into scalar registers;
//   - the N / NS waves of a workgroup share 64 channels.  They stage delta_t and delta_t u_t
//     of a tile of kTok tokens once, each wave a part of the tokens, double-buffered in LDS;
//   - the waves' partial sums over their states meet in LDS, and the wave that staged a
//     token adds them up, applies D and the gate from the u and z it kept, and stores.
// One barrier a tile.  States and sums are fp32.
//
// Few channels (B D / 64 workgroups below the card's size): the time axis is cut into P
// segments.  A first launch walks all but the last from zero for their local end states and
// sums of delta; each workgroup of the second composes the segments before its own.
#include "qd_ssm.h"

namespace qd {
namespace {

constexpr int kOut = 0, kSeg = 1, kKeep = 2;   // the full walk; a segment's effect only; the states only

struct ScanArgs {
    SsmArgs a;
    int Dg, nblk;                    // channels per group, 64-channel blocks per group
    Segments seg;
    SegBuf buf;
    float *keep;                     // kKeep: [B][ceil(T / kTok)][N][D]
};

template <class P, int N, int NS, int MODE>
__global__ __launch_bounds__(64 * N / NS) void scan_kernel(const ScanArgs k) {
    using R = typename P::R;
    constexpr int NW = N / NS, TPW = kTok / NW > 0 ? kTok / NW : 1;
    __shared__ float2 s_in[2][kTok][64];
    __shared__ float s_y[MODE == kOut ? 2 : 1][MODE == kOut ? NW : 1][kTok][64];
    const SsmArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk, nseg = MODE == kSeg ? k.seg.P - 1 : k.seg.P;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = bp % nseg, b = bp / nseg;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const bool live = c_in < k.Dg;
    const int ch = g * k.Dg + min(c_in, k.Dg - 1);
    const int n0 = wave * NS;
    const size_t D = a.D;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int tb = p * k.seg.len, te = min(len, tb + k.seg.len);

    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = a.A[static_cast<size_t>(ch) * N + n0 + i] * kLog2e;
        h[i] = 0.f;
    }
    float *seg_h = k.buf.h + (static_cast<size_t>(b) * k.seg.P * N + n0) * D + ch;   // slot q at q N D
    float *seg_s = k.buf.s + static_cast<size_t>(b) * k.seg.P * D + ch;
    if (p == 0) {
        if (a.S0) {
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = a.S0[(static_cast<size_t>(b) * D + ch) * N + n0 + i];
        }
        // The full walk's last workgroup may overwrite S0: this launch leaves a copy.
        if (MODE == kSeg && live) {
#pragma unroll
            for (int i = 0; i < NS; ++i) seg_h[i * D] = h[i];
        }
    }
    if (MODE != kSeg && k.seg.P > 1) {
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = seg_h[i * D];
        for (int q = 0; q < p; ++q) {
            const float *hq = seg_h + static_cast<size_t>(q + 1) * N * D;
            const float sum = seg_s[static_cast<size_t>(q) * D];
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), h[i], hq[i * D]);
        }
    }
    if (MODE == kSeg) {              // the local effect starts from zero
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = 0.f;
    }
    float sum_delta = 0.f;

    if (tb < te) {
        const size_t row0 = static_cast<size_t>(b) * a.T;
        const R *u = static_cast<const R *>(a.u) + row0 * D + ch;
        const R *dt = static_cast<const R *>(a.dt) + row0 * D + ch;
        const R *z = a.z ? static_cast<const R *>(a.z) + row0 * D + ch : nullptr;
        R *o = MODE == kOut ? static_cast<R *>(a.o) + row0 * D + ch : nullptr;
        const R *Bm = static_cast<const R *>(a.Bm) + (row0 * a.G + g) * N + n0;
        const R *Cm = static_cast<const R *>(a.Cm) + (row0 * a.G + g) * N + n0;
        const size_t bc_row = static_cast<size_t>(a.G) * N;
        const float dt_bias = a.dt_bias ? a.dt_bias[ch] : 0.f;
        const float skip = a.Dskip ? a.Dskip[ch] : 0.f;
        const int ntile = (te - tb + kTok - 1) / kTok;

        struct Raw {
            float u[TPW], dt[TPW], z[TPW];
        };
        // Rows at and past the end read the last row instead; what they give is not used.
        auto fetch = [&](int tile, Raw &r) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) {
                if (wave + j * NW >= kTok) continue;
                const size_t t = min(tb + tile * kTok + wave + j * NW, te - 1);
                r.u[j] = P::to_f32(u[t * D]);
                r.dt[j] = P::to_f32(dt[t * D]);
                if (MODE == kOut && z) r.z[j] = P::to_f32(z[t * D]);
            }
        };
        auto stage = [&](int tile, const Raw &r) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) {
                const int i = wave + j * NW;
                if (i >= kTok) continue;
                const float x = r.dt[j] + dt_bias;
                const float delta = a.softplus ? softplusf(x) : x;
                s_in[tile & 1][i][lane] = make_float2(delta, delta * r.u[j]);
            }
        };
        auto walk = [&](int tile, auto full) {
            const int t0 = tb + tile * kTok, nt = te - t0;
            if (MODE == kKeep && live) {
                const size_t nc = (a.T + kTok - 1) / kTok;
                float *keep = k.keep + ((b * nc + t0 / kTok) * N + n0) * D + ch;
#pragma unroll
                for (int i = 0; i < NS; ++i) keep[i * D] = h[i];
            }
            ScalarRow<P, NS> rb[kTok], rc[MODE == kOut ? kTok : 1];
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                const size_t row = static_cast<size_t>(full ? t0 + t : min(t0 + t, te - 1)) * bc_row;
                rb[t].load(Bm + row);
                if constexpr (MODE == kOut) rc[t].load(Cm + row);
            }
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                if (!full && t >= nt) break;
                const float2 in = s_in[tile & 1][t][lane];
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = fmaf(__builtin_amdgcn_exp2f(in.x * A2[i]), h[i], in.y * rb[t][i]);
                    if constexpr (MODE == kOut) y = fmaf(rc[t][i], h[i], y);
                }
                if constexpr (MODE == kOut) s_y[tile & 1][wave][t][lane] = y;
                else if constexpr (MODE == kSeg) sum_delta += in.x;
            }
        };
        auto finish = [&](int tile, const Raw &r) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) {
                const int i = wave + j * NW, t = tb + tile * kTok + i;
                if (i >= kTok || t >= te) continue;
                float y = skip * r.u[j];
#pragma unroll
                for (int w = 0; w < NW; ++w) y += s_y[tile & 1][w][i][lane];
                if (z) y *= siluf(r.z[j]);
                if (live) o[static_cast<size_t>(t) * D] = P::from_f32(y);
            }
        };

        Raw cur, nxt;
        fetch(0, cur);
        stage(0, cur);
        nxt = cur;
        if (ntile > 1) fetch(1, nxt);
        __syncthreads();
        for (int i = 0; i < ntile; ++i) {
            if (tb + (i + 1) * kTok <= te) walk(i, std::true_type{});
            else walk(i, std::false_type{});
            if (i + 1 < ntile) stage(i + 1, nxt);
            const Raw mine = cur;
            cur = nxt;
            if (i + 2 < ntile) fetch(i + 2, nxt);
            __syncthreads();
            if constexpr (MODE == kOut) finish(i, mine);
        }
    }
    if (!live) return;
    if constexpr (MODE == kOut) {
        if (p == k.seg.P - 1 && a.S_T) {
#pragma unroll
            for (int i = 0; i < NS; ++i) a.S_T[(static_cast<size_t>(b) * D + ch) * N + n0 + i] = h[i];
        }
    } else if constexpr (MODE == kSeg) {
#pragma unroll
        for (int i = 0; i < NS; ++i) seg_h[static_cast<size_t>(p + 1) * N * D + i * D] = h[i];
        if (wave == 0) seg_s[static_cast<size_t>(p) * D] = sum_delta;
    }
}

// One token for each of B sequences, the state updated in place: bound by reading and
// writing the fp32 state.  N / 4 lanes share a channel, four states (16 bytes) each, so a
// wave reads 1 KB in a row; kStepReps channels a lane are in flight.
constexpr int kStepThreads = 256, kStepReps = 2;
template <class P, int N>
__global__ __launch_bounds__(kStepThreads) void ssm_step_kernel(const SsmArgs a) {
    using R = typename P::R;
    constexpr int LPC = N / 4, CPB = kStepThreads / LPC;
    const int nb = (a.D + CPB * kStepReps - 1) / (CPB * kStepReps);
    const int sub = threadIdx.x % LPC, b = blockIdx.x / nb;
    const int c0 = (blockIdx.x % nb) * CPB * kStepReps + threadIdx.x / LPC;
    const int Dg = a.D / a.G;
    float4 h[kStepReps], A[kStepReps];
    float u[kStepReps], x[kStepReps], z[kStepReps];
#pragma unroll
    for (int r = 0; r < kStepReps; ++r) {
        const int ch = min(c0 + r * CPB, a.D - 1);
        const size_t at = static_cast<size_t>(b) * a.D + ch;
        h[r] = *reinterpret_cast<const float4 *>(a.S_T + at * N + 4 * sub);
        A[r] = *reinterpret_cast<const float4 *>(a.A + static_cast<size_t>(ch) * N + 4 * sub);
        u[r] = P::to_f32(static_cast<const R *>(a.u)[at]);
        x[r] = P::to_f32(static_cast<const R *>(a.dt)[at]) + (a.dt_bias ? a.dt_bias[ch] : 0.f);
        z[r] = a.z ? P::to_f32(static_cast<const R *>(a.z)[at]) : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kStepReps; ++r) {
        const int c = c0 + r * CPB, ch = min(c, a.D - 1);
        const size_t at = static_cast<size_t>(b) * a.D + ch;
        const size_t bc = (static_cast<size_t>(b) * a.G + ch / Dg) * N + 4 * sub;
        const R *Bm = static_cast<const R *>(a.Bm) + bc, *Cm = static_cast<const R *>(a.Cm) + bc;
        const float delta = a.softplus ? softplusf(x[r]) : x[r], du = delta * u[r];
        float *hp = &h[r].x;
        const float *Ap = &A[r].x;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hp[i] = fmaf(__builtin_amdgcn_exp2f(delta * (Ap[i] * kLog2e)), hp[i], du * P::to_f32(Bm[i]));
            y = fmaf(P::to_f32(Cm[i]), hp[i], y);
        }
        y = group_sum(y, LPC);
        if (c < a.D) {
            *reinterpret_cast<float4 *>(a.S_T + at * N + 4 * sub) = h[r];
            if (sub == 0) {
                y = fmaf(a.Dskip ? a.Dskip[ch] : 0.f, u[r], y);
                if (a.z) y *= siluf(z[r]);
                static_cast<R *>(a.o)[at] = P::from_f32(y);
            }
        }
    }
}

// Segments of the time axis: enough workgroups that every SIMD has two waves, as long as a
// segment keeps at least 128 tokens.
Segments fwd_segments(int B, int T, int D, int G, int N) {
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    const long long nblk = static_cast<long long>(B) * G * ((D / G + 63) / 64);
    const long long waves = nblk * (N / 4);
    if (nblk == 0 || waves >= 4LL * cus) return cut_time(T, 1);
    long long want = (8LL * cus + waves - 1) / waves;
    if (want > T / 128) want = T / 128;
    return cut_time(T, static_cast<int>(want > 64 ? 64 : want));
}

template <class P, int N, int MODE>
hipError_t run_scan(const ScanArgs &k, hipStream_t stream) {
    constexpr int NS = 4;
    const dim3 blk(64 * N / NS);
    const unsigned per = static_cast<unsigned>(k.a.B) * k.a.G * k.nblk;
    if (k.seg.P > 1)
        hipLaunchKernelGGL((scan_kernel<P, N, NS, kSeg>), dim3(per * (k.seg.P - 1)), blk, 0, stream, k);
    hipLaunchKernelGGL((scan_kernel<P, N, NS, MODE>), dim3(per * k.seg.P), blk, 0, stream, k);
    return hipGetLastError();
}

template <class P, int MODE>
hipError_t run_scan_n(const ScanArgs &k, hipStream_t stream) {
    if (k.a.N == 16) return run_scan<P, 16, MODE>(k, stream);
    if (k.a.N == 32) return run_scan<P, 32, MODE>(k, stream);
    return run_scan<P, 64, MODE>(k, stream);
}

ScanArgs scan_args(const SsmArgs &a, Segments seg) {
    ScanArgs k;
    k.a = a;
    k.Dg = a.D / a.G;
    k.nblk = (k.Dg + 63) / 64;
    k.seg = seg;
    k.buf = SegBuf{nullptr, nullptr};
    k.keep = nullptr;
    return k;
}

template <class P>
hipError_t run_step(const SsmArgs &a, hipStream_t stream) {
    const int cpb = kStepThreads / (a.N / 4) * kStepReps;
    const dim3 grid(static_cast<unsigned>((a.D + cpb - 1) / cpb) * a.B), blk(kStepThreads);
    if (a.N == 16) hipLaunchKernelGGL((ssm_step_kernel<P, 16>), grid, blk, 0, stream, a);
    else if (a.N == 32) hipLaunchKernelGGL((ssm_step_kernel<P, 32>), grid, blk, 0, stream, a);
    else hipLaunchKernelGGL((ssm_step_kernel<P, 64>), grid, blk, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

bool ssm_supported(int dtype, int N) { return (dtype == 0 || dtype == 1) && (N == 16 || N == 32 || N == 64); }

// Every launch: up to 64 segments a channel block, 16 N lanes a workgroup (N / 4 waves); the
// sums over blocks take a lane for four values of dB and dC, and 16 for a value of dA.
bool ssm_fits(int B, int T, int D, int G, int N) {
    const long long blocks = static_cast<long long>(B) * G * ((D / G + 63) / 64), tiles = T / 64 + 1;
    return blocks < (1LL << 31) && blocks * (tiles < 64 ? tiles : 64) * 16 * N < (1LL << 32) &&
           static_cast<long long>(B) * T < (1LL << 31) && static_cast<long long>(B) * T * G < (1LL << 32) / N * 2 - 1024 &&
           static_cast<long long>(D) * N < (1LL << 27);
}

size_t ssm_fwd_workspace(int dtype, int B, int T, int D, int G, int N) {
    (void)dtype;
    const Segments s = fwd_segments(B, T, D, G, N);
    return s.P > 1 ? static_cast<size_t>(B) * s.P * D * (N + 1) * sizeof(float) : 0;
}

hipError_t launch_ssm_fwd(int dtype, const SsmArgs &a, void *ws, hipStream_t stream) {
    ScanArgs k = scan_args(a, fwd_segments(a.B, a.T, a.D, a.G, a.N));
    if (k.seg.P > 1) {
        k.buf.h = static_cast<float *>(ws);
        k.buf.s = k.buf.h + static_cast<size_t>(a.B) * k.seg.P * a.N * a.D;
    }
    return dtype == 1 ? run_scan_n<Bf16, kOut>(k, stream) : run_scan_n<F32, kOut>(k, stream);
}

hipError_t launch_ssm_states(int dtype, const SsmArgs &a, Segments seg, SegBuf buf, float *keep, hipStream_t stream) {
    ScanArgs k = scan_args(a, seg);
    k.buf = buf;
    k.keep = keep;
    return dtype == 1 ? run_scan_n<Bf16, kKeep>(k, stream) : run_scan_n<F32, kKeep>(k, stream);
}

hipError_t launch_ssm_step(int dtype, const SsmArgs &a, hipStream_t stream) {
    return dtype == 1 ? run_step<Bf16>(a, stream) : run_step<F32>(a, stream);
}

}  // namespace qd
