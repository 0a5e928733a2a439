// Gradients of the selective scan (qd_ssm.hip) for gfx950: of sum(o d_o) + sum(S_T dS_T).
// With dy = d_o silu(z), and g_t the gradient with respect to h_t,
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1},   a_t = exp(delta_t A),   g_{T-1} also takes dS_T
//   q_t = a_t g_t h_{t-1}
//   du     = delta s1 + D dy                 s1 = sum_n g B
//   ddelta = s2 + u s1                       s2 = sum_n A q
//   dB = sum_d g delta u,  dC = sum_d dy h,  dA = sum_t delta q,  dD = sum dy u
//   dz = d_o y silu'(z),  ddt = ddelta sigmoid(dt + dt_bias),  dS0 = a_0 g_0.
//
// The states are needed in reverse order.  The forward walk keeps the state before every
// tile of kTok tokens in HBM (4 N / kTok bytes a token and channel); the reverse walk takes a
// tile's entry state, runs its kTok tokens forward with decays and states in registers, and
// then backward.  Lanes, waves, staging and segments are those of the forward kernel: a lane
// is a channel, a wave four of its states, B and C in scalar registers, s1, s2 and y joined
// through LDS by the wave that staged the token.
//
// dB and dC sum over channels, which are lanes: eight values a lane and token.  A chain of
// fp32 MFMAs does it without a cross-lane instruction: the 64 lanes' values are a 16 x 4
// operand, the other operand has ones in one column j, so the product adds four lanes into
// column j of each of 16 rows; two tokens fill the 16 columns, and a second product with
// ones joins the rows.  The fp32 products are by 1 and 0, so only the sum rounds.  (0 times
// a non-finite value is not 0: one non-finite value makes its pair of tokens' dB and dC
// non-finite.)  Each 64-channel block leaves its sums in the workspace and a second kernel
// adds the blocks in order, so the result does not depend on the order of workgroups.
#include "qd_ssm.h"

namespace qd {
namespace {

constexpr int kNs = 4;               // states a wave

struct RevArgs {
    SsmBwdArgs a;
    int Dg, nblk;
    Segments seg;
    float *keep;                     // [B][ceil(T / kTok)][N][D]
    SegBuf rev;                      // segment p's local gradient (slot p) and sum of delta (slot p)
    float *part_bc;                  // [nblk][B][T][G][2][N]
    float *part_a;                   // [B][P][D][N]
    float *part_d;                   // [B][P][2][D]: dD, ddt_bias
};

// A segment's effect on the gradient that enters at its end: g_out = exp(A sum(delta)) g_in + g_local.
template <class P, int N>
__global__ __launch_bounds__(64 * N / kNs) void seg_grad_kernel(const RevArgs k) {
    using R = typename P::R;
    constexpr int NS = kNs, NW = N / NS, TPW = kTok / NW > 0 ? kTok / NW : 1;
    __shared__ float2 s_in[2][kTok][64];
    const SsmBwdArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk, nseg = k.seg.P - 1;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = 1 + bp % nseg, b = bp / nseg;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const int ch = g * k.Dg + min(c_in, k.Dg - 1), n0 = wave * NS;
    const size_t D = a.D, row0 = static_cast<size_t>(b) * a.T;
    const int tb = p * k.seg.len, te = min(a.T, tb + k.seg.len), ntile = (te - tb + kTok - 1) / kTok;
    float A2[NS], G[NS] = {}, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = a.A[static_cast<size_t>(ch) * N + n0 + i] * kLog2e;
    const R *dt = static_cast<const R *>(a.dt) + row0 * D + ch;
    const R *z = a.z ? static_cast<const R *>(a.z) + row0 * D + ch : nullptr;
    const R *d_o = static_cast<const R *>(a.d_o) + row0 * D + ch;
    const R *Cm = static_cast<const R *>(a.Cm) + (row0 * a.G + g) * N + n0;
    const size_t bc_row = static_cast<size_t>(a.G) * N;
    const float dt_bias = a.dt_bias ? a.dt_bias[ch] : 0.f;

    struct Raw {
        float dt[TPW], z[TPW], d_o[TPW];
    };
    auto fetch = [&](int tile, Raw &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            if (wave + j * NW >= kTok) continue;
            const size_t t = min(tb + tile * kTok + wave + j * NW, te - 1);
            r.dt[j] = P::to_f32(dt[t * D]);
            r.d_o[j] = P::to_f32(d_o[t * D]);
            if (z) r.z[j] = P::to_f32(z[t * D]);
        }
    };
    auto stage = [&](int tile, const Raw &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int i = wave + j * NW;
            if (i >= kTok) continue;
            const float x = r.dt[j] + dt_bias;
            const float delta = a.softplus ? softplusf(x) : x;
            s_in[tile & 1][i][lane] = make_float2(delta, z ? r.d_o[j] * siluf(r.z[j]) : r.d_o[j]);
        }
    };
    Raw r;
    fetch(ntile - 1, r);
    stage(ntile - 1, r);
    if (ntile > 1) fetch(ntile - 2, r);
    __syncthreads();
    for (int tile = ntile - 1; tile >= 0; --tile) {
        const int t0 = tb + tile * kTok, nt = min(kTok, te - t0);
        ScalarRow<P, NS> rc[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) rc[t].load(Cm + static_cast<size_t>(min(t0 + t, te - 1)) * bc_row);
#pragma unroll
        for (int t = kTok - 1; t >= 0; --t) {
            if (t >= nt) continue;
            const float2 in = s_in[tile & 1][t][lane];
            sum += in.x;
#pragma unroll
            for (int i = 0; i < NS; ++i) G[i] = __builtin_amdgcn_exp2f(in.x * A2[i]) * fmaf(rc[t][i], in.y, G[i]);
        }
        if (tile > 0) stage(tile - 1, r);
        if (tile > 1) fetch(tile - 2, r);
        __syncthreads();
    }
    if (c_in >= k.Dg) return;
    float *out = k.rev.h + ((static_cast<size_t>(b) * k.seg.P + p) * N + n0) * D + ch;
#pragma unroll
    for (int i = 0; i < NS; ++i) out[i * D] = G[i];
    if (wave == 0) k.rev.s[(static_cast<size_t>(b) * k.seg.P + p) * D + ch] = sum;
}

template <class P, int N>
__global__ __launch_bounds__(64 * N / kNs) void ssm_bwd_kernel(const RevArgs k) {
    using R = typename P::R;
    constexpr int NS = kNs, NW = N / NS, TPW = kTok / NW > 0 ? kTok / NW : 1;
    // One or two buffers of the partial sums: two (one barrier a tile) while they fit with
    // room for a second workgroup.
    constexpr int NB = N <= 16 ? 2 : 1;
    __shared__ float2 s_in[2][kTok][64];
    __shared__ float s_dy[2][kTok][64];
    __shared__ float s_p[NB][NW][3][kTok][64];
    const SsmBwdArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = bp % k.seg.P, b = bp / k.seg.P;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const bool live = c_in < k.Dg;
    const int ch = g * k.Dg + min(c_in, k.Dg - 1), n0 = wave * NS;
    const size_t D = a.D, row0 = static_cast<size_t>(b) * a.T;
    const int tb = p * k.seg.len, te = min(a.T, tb + k.seg.len), ntile = (te - tb + kTok - 1) / kTok;
    const size_t st = (static_cast<size_t>(b) * D + ch) * N + n0;

    float A2[NS], G[NS], dA[NS] = {};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = a.A[static_cast<size_t>(ch) * N + n0 + i] * kLog2e;
        G[i] = a.dS_T && live ? a.dS_T[st + i] : 0.f;
    }
    for (int q = k.seg.P - 1; q > p; --q) {
        const float *gq = k.rev.h + ((static_cast<size_t>(b) * k.seg.P + q) * N + n0) * D + ch;
        const float sum = k.rev.s[(static_cast<size_t>(b) * k.seg.P + q) * D + ch];
#pragma unroll
        for (int i = 0; i < NS; ++i) G[i] = live ? fmaf(__builtin_amdgcn_exp2f(A2[i] * sum), G[i], gq[i * D]) : 0.f;
    }
    const R *u = static_cast<const R *>(a.u) + row0 * D + ch;
    const R *dt = static_cast<const R *>(a.dt) + row0 * D + ch;
    const R *z = a.z ? static_cast<const R *>(a.z) + row0 * D + ch : nullptr;
    const R *d_o = static_cast<const R *>(a.d_o) + row0 * D + ch;
    const R *Bm = static_cast<const R *>(a.Bm) + (row0 * a.G + g) * N + n0;
    const R *Cm = static_cast<const R *>(a.Cm) + (row0 * a.G + g) * N + n0;
    const size_t bc_row = static_cast<size_t>(a.G) * N;
    const float dt_bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.Dskip ? a.Dskip[ch] : 0.f;
    const size_t nc = (a.T + kTok - 1) / kTok;
    const float *keep = k.keep + ((static_cast<size_t>(b) * nc + tb / kTok) * N + n0) * D + ch;
    float *part_bc = k.part_bc + (((static_cast<size_t>(cb % k.nblk) * a.B + b) * a.T) * a.G + g) * 2 * N + n0;
    float acc_d = 0.f, acc_b = 0.f;

    struct Tok {                     // what a wave keeps of the tokens it stages
        float u[TPW], x[TPW], z[TPW], d_o[TPW], delta[TPW], dy[TPW];
    };
    auto fetch = [&](int tile, Tok &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            if (wave + j * NW >= kTok) continue;
            const size_t t = min(tb + tile * kTok + wave + j * NW, te - 1);
            r.u[j] = P::to_f32(u[t * D]);
            r.x[j] = P::to_f32(dt[t * D]);
            r.d_o[j] = P::to_f32(d_o[t * D]);
            if (z) r.z[j] = P::to_f32(z[t * D]);
        }
    };
    // Tokens past the end and lanes past the channels enter with delta, u and dy zero: the
    // state passes through them and they add nothing to any sum.
    auto stage = [&](int tile, Tok &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int i = wave + j * NW;
            if (i >= kTok) continue;
            const bool in = live && tb + tile * kTok + i < te;
            r.x[j] += dt_bias;
            const float delta = a.softplus ? softplusf(r.x[j]) : r.x[j];
            const float dy = z ? r.d_o[j] * siluf(r.z[j]) : r.d_o[j];
            r.delta[j] = delta;
            r.dy[j] = dy;
            s_in[tile & 1][i][lane] = in ? make_float2(delta, delta * r.u[j]) : make_float2(0.f, 0.f);
            s_dy[tile & 1][i][lane] = in ? dy : 0.f;
        }
    };
    auto entry = [&](int tile, float (&h)[NS]) {
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = live ? keep[static_cast<size_t>(tile) * N * D + i * D] : 0.f;
    };
    float one[16], row_one[4];       // the selecting operands
#pragma unroll
    for (int j = 0; j < 16; ++j) one[j] = (lane & 15) == j ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) row_one[j] = ((lane & 15) >> 2) == j ? 1.f : 0.f;

    auto walk = [&](int tile, const float (&h_in)[NS]) {
        const int t0 = tb + tile * kTok, buf = tile & 1;
        ScalarRow<P, NS> rb[kTok], rc[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const size_t row = static_cast<size_t>(min(t0 + t, te - 1)) * bc_row;
            rb[t].load(Bm + row);
            rc[t].load(Cm + row);
        }
        float dec[kTok][NS], h[kTok][NS];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const float2 in = s_in[buf][t][lane];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                dec[t][i] = __builtin_amdgcn_exp2f(in.x * A2[i]);
                h[t][i] = fmaf(dec[t][i], t ? h[t - 1][i] : h_in[i], in.y * rb[t][i]);
            }
        }
        float dAt[NS] = {};          // this tile's part of dA: fewer roundings against the long sum
        f32x4 pair = zero4(), joined = zero4();
#pragma unroll
        for (int t = kTok - 1; t >= 0; --t) {
            const float2 in = s_in[buf][t][lane];
            const float dy = s_dy[buf][t][lane];
            float y = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float gi = fmaf(rc[t][i], dy, G[i]);
                y = fmaf(rc[t][i], h[t][i], y);
                s1 = fmaf(gi, rb[t][i], s1);
                G[i] = dec[t][i] * gi;
                const float q = G[i] * (t ? h[t - 1][i] : h_in[i]);
                s2 = fmaf(A2[i], q, s2);
                dAt[i] = fmaf(in.x, q, dAt[i]);
                pair = __builtin_amdgcn_mfma_f32_16x16x4f32(gi * in.y, one[(t & 1) * 8 + i], pair, 0, 0, 0);
                pair = __builtin_amdgcn_mfma_f32_16x16x4f32(dy * h[t][i], one[(t & 1) * 8 + 4 + i], pair, 0, 0, 0);
            }
            float *sp = &s_p[NB == 2 ? buf : 0][wave][0][t][lane];
            sp[0] = y;
            sp[kTok * 64] = s1;
            sp[2 * kTok * 64] = s2;
            if ((t & 1) == 0) {      // both tokens of a pair are in: add the 16 rows
                joined = __builtin_amdgcn_mfma_f32_16x16x4f32(row_one[t / 2], (pair[0] + pair[1]) + (pair[2] + pair[3]),
                                                              joined, 0, 0, 0);
                pair = zero4();
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) dA[i] += dAt[i];
        // lane l now holds column l % 16 of pair l / 16
        const int j = lane & 15, t = t0 + 2 * (lane >> 4) + (j >> 3), e = j & 7;
        if (t < te) part_bc[static_cast<size_t>(t) * a.G * 2 * N + (e >> 2) * N + (e & 3)] = joined[0];
    };
    auto finish = [&](int tile, const Tok &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int i = wave + j * NW, t = tb + tile * kTok + i;
            if (i >= kTok || t >= te) continue;
            float y = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float *sp = &s_p[NB == 2 ? tile & 1 : 0][w][0][i][lane];
                y += sp[0];
                s1 += sp[kTok * 64];
                s2 += sp[2 * kTok * 64];
            }
            float dd = fmaf(r.u[j], s1, s2 * kLn2);
            if (a.softplus) dd *= sigmoidf(r.x[j]);
            acc_d = fmaf(r.dy[j], r.u[j], acc_d);
            acc_b += dd;
            if (!live) continue;
            const size_t at = (row0 + t) * D + ch;
            static_cast<R *>(a.du)[at] = P::from_f32(fmaf(r.delta[j], s1, skip * r.dy[j]));
            static_cast<R *>(a.ddt)[at] = P::from_f32(dd);
            if (z) static_cast<R *>(a.dz)[at] = P::from_f32(r.d_o[j] * fmaf(skip, r.u[j], y) * dsiluf(r.z[j]));
        }
    };

    Tok cur, nxt;
    float h_cur[NS], h_nxt[NS];
    fetch(ntile - 1, cur);
    entry(ntile - 1, h_cur);
    stage(ntile - 1, cur);
    nxt = cur;
    if (ntile > 1) fetch(ntile - 2, nxt);
    __syncthreads();
    for (int tile = ntile - 1; tile >= 0; --tile) {
        if (tile > 0) entry(tile - 1, h_nxt);
        walk(tile, h_cur);
        if (tile > 0) stage(tile - 1, nxt);
        const Tok mine = cur;
        cur = nxt;
        if (tile > 1) fetch(tile - 2, nxt);
#pragma unroll
        for (int i = 0; i < NS; ++i) h_cur[i] = h_nxt[i];
        __syncthreads();
        finish(tile, mine);
        if (NB == 1) __syncthreads();
    }
    __syncthreads();
    float (*ends)[NW][64] = reinterpret_cast<float (*)[NW][64]>(&s_p[0][0][0][0][0]);
    ends[0][wave][lane] = acc_d;
    ends[1][wave][lane] = acc_b;
    __syncthreads();
    if (!live) return;
    if (wave == 0) {
        float sd = 0.f, sb = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            sd += ends[0][w][lane];
            sb += ends[1][w][lane];
        }
        float *out = k.part_d + (static_cast<size_t>(b) * k.seg.P + p) * 2 * D + ch;
        out[0] = sd;
        out[D] = sb;
    }
    float *pa = k.part_a + ((static_cast<size_t>(b) * k.seg.P + p) * D + ch) * N + n0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        pa[i] = dA[i];
        if (p == 0 && a.dS0) a.dS0[st + i] = G[i];
    }
}

// dB and dC from the channel blocks' sums, added in block order.
template <class P>
__global__ __launch_bounds__(256) void bc_sum_kernel(const RevArgs k) {
    using R = typename P::R;
    const int N = k.a.N;
    const long long rows = static_cast<long long>(k.a.B) * k.a.T * k.a.G;
    const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;   // four states of one row
    if (i >= rows * 2 * N) return;
    f32x4 s = zero4();
    for (int blk = 0; blk < k.nblk; ++blk) s += *reinterpret_cast<const f32x4 *>(k.part_bc + static_cast<size_t>(blk) * rows * 2 * N + i);
    const long long row = i / (2 * N);
    const int e = static_cast<int>(i % (2 * N));
    R *out = static_cast<R *>(e < N ? k.a.dB : k.a.dC) + row * N + (e < N ? e : e - N);
    P::st4(out, s);
}

struct StoreA {
    float *dA;
    __device__ __forceinline__ void operator()(long long c, float v) const { dA[c] = v; }
};
struct StoreD {
    float *dD, *db;
    int D;
    __device__ __forceinline__ void operator()(long long c, float v) const {
        if (c < D) {
            if (dD) dD[c] = v;
        } else if (db) {
            db[c - D] = v;
        }
    }
};

// With no tokens the gradients of what the tokens share are zero and dS0 is dS_T.
__global__ __launch_bounds__(256) void ssm_bwd_empty_kernel(const SsmBwdArgs a) {
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x, DN = static_cast<size_t>(a.D) * a.N;
    if (i < DN) a.dA[i] = 0.f;
    if (i < static_cast<size_t>(a.D)) {
        if (a.dD) a.dD[i] = 0.f;
        if (a.ddt_bias) a.ddt_bias[i] = 0.f;
    }
    if (a.dS0 && i < a.B * DN) a.dS0[i] = a.dS_T ? a.dS_T[i] : 0.f;
}

// Segments of the time axis: two waves a SIMD, as long as a segment keeps 64 tokens.
Segments bwd_segments(int B, int T, int D, int G, int N) {
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    const long long waves = static_cast<long long>(B) * G * ((D / G + 63) / 64) * (N / kNs);
    if (waves == 0) return cut_time(T, 1);
    long long want = (8LL * cus + waves - 1) / waves;
    if (want > T / 64) want = T / 64;
    return cut_time(T, static_cast<int>(want > 64 ? 64 : want));
}

struct Sizes {                       // floats of each part of the workspace, every one a multiple of four
    size_t seg_h, seg_s, keep, bc, pa, pd;
    size_t total() const { return 2 * (seg_h + seg_s) + keep + bc + pa + pd; }
};
size_t up4(size_t n) { return (n + 3) & ~static_cast<size_t>(3); }
Sizes sizes(int B, int T, int D, int G, int N, Segments s) {
    Sizes z;
    const size_t b = B, d = D, n = N, P = s.P, nc = (T + kTok - 1) / kTok, nblk = (D / G + 63) / 64;
    z.seg_h = s.P > 1 ? up4(b * P * n * d) : 0;
    z.seg_s = s.P > 1 ? up4(b * P * d) : 0;
    z.keep = up4(b * nc * n * d);
    z.bc = up4(nblk * b * T * G * 2 * n);
    z.pa = up4(b * P * d * n);
    z.pd = up4(b * P * 2 * d);
    return z;
}

template <class P, int N>
hipError_t run_bwd(const RevArgs &k, hipStream_t stream) {
    const dim3 blk(64 * N / kNs);
    const unsigned per = static_cast<unsigned>(k.a.B) * k.a.G * k.nblk;
    if (k.seg.P > 1) hipLaunchKernelGGL((seg_grad_kernel<P, N>), dim3(per * (k.seg.P - 1)), blk, 0, stream, k);
    hipLaunchKernelGGL((ssm_bwd_kernel<P, N>), dim3(per * k.seg.P), blk, 0, stream, k);
    const long long n4 = static_cast<long long>(k.a.B) * k.a.T * k.a.G * 2 * N / 4;
    hipLaunchKernelGGL((bc_sum_kernel<P>), dim3(static_cast<unsigned>((n4 + 255) / 256)), dim3(256), 0, stream, k);
    const int rows = k.a.B * k.seg.P;
    column_sum(k.part_a, rows, static_cast<long long>(k.a.D) * N, StoreA{k.a.dA}, stream);
    if (k.a.dD || k.a.ddt_bias) column_sum(k.part_d, rows, 2LL * k.a.D, StoreD{k.a.dD, k.a.ddt_bias, k.a.D}, stream);
    return hipGetLastError();
}
template <class P>
hipError_t run_bwd_n(const RevArgs &k, hipStream_t stream) {
    if (k.a.N == 16) return run_bwd<P, 16>(k, stream);
    if (k.a.N == 32) return run_bwd<P, 32>(k, stream);
    return run_bwd<P, 64>(k, stream);
}

}  // namespace

size_t ssm_bwd_workspace(int dtype, int B, int T, int D, int G, int N) {
    (void)dtype;
    if (static_cast<long long>(B) * T * D == 0) return 0;
    return sizes(B, T, D, G, N, bwd_segments(B, T, D, G, N)).total() * sizeof(float);
}

hipError_t launch_ssm_bwd(int dtype, const SsmBwdArgs &a, void *ws, hipStream_t stream) {
    if (static_cast<long long>(a.B) * a.T == 0) {
        const size_t n = static_cast<size_t>(a.B > 0 ? a.B : 1) * a.D * a.N;
        hipLaunchKernelGGL(ssm_bwd_empty_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    RevArgs k;
    k.a = a;
    k.Dg = a.D / a.G;
    k.nblk = (k.Dg + 63) / 64;
    k.seg = bwd_segments(a.B, a.T, a.D, a.G, a.N);
    const Sizes z = sizes(a.B, a.T, a.D, a.G, a.N, k.seg);
    float *w = static_cast<float *>(ws);
    SegBuf fwd{w, w + z.seg_h};
    w += z.seg_h + z.seg_s;
    k.rev = SegBuf{w, w + z.seg_h};
    w += z.seg_h + z.seg_s;
    k.keep = w;
    k.part_bc = k.keep + z.keep;
    k.part_a = k.part_bc + z.bc;
    k.part_d = k.part_a + z.pa;
    SsmArgs f{};
    f.u = a.u; f.dt = a.dt; f.Bm = a.Bm; f.Cm = a.Cm;
    f.A = a.A; f.dt_bias = a.dt_bias; f.S0 = a.S0;
    f.B = a.B; f.T = a.T; f.D = a.D; f.G = a.G; f.N = a.N;
    f.softplus = a.softplus;
    const hipError_t err = launch_ssm_states(dtype, f, k.seg, fwd, k.keep, stream);
    if (err != hipSuccess) return err;
    return dtype == 1 ? run_bwd_n<Bf16>(k, stream) : run_bwd_n<F32>(k, stream);
}

}  // namespace qd
