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
// is a channel, a wave some of its states, B and C in scalar registers, s1, s2 and y joined
// through LDS by the wave that staged the token.
//
// dB and dC sum over channels, which are lanes: two values a state, lane and token.  A wave
// puts 16 values a lane into its part of LDS, reads them back across the lanes four at a
// time, and joins the readers: about 1.8 instructions a value.  (Adding the lanes by fp32 MFMA
// products with ones, whose 36 cycles a value came on top of the vector instructions', took
// 266 of 897 us at 8 x 2048 tokens, 2048 channels, 16 states; exchanges in registers alone
// take 35 instructions a set against 28.)
//
// 8 x 2048 tokens, 2048 channels, 16 states, bf16, gated: 669 us a call among others; the least of
// 50 traced launches are 515 us for this kernel, 127 for the walk that keeps states and 16 for the
// sums over workgroups.
// Its bytes would take 95 us; two exponentials and sixteen multiply-adds a token, channel and state
// 225 us at the rate four waves a SIMD reach.  LDS (148 KB) holds one workgroup a compute unit, so
// two waves a SIMD; of this kernel's time the channel sums are 107 and the ends of tokens 71.
//
// Each 64-channel block leaves its sums in the workspace and a second kernel adds the blocks in
// order, so the result does not depend on the order of workgroups.
#include "qd_ssm.h"

namespace qd {
namespace {

struct RevArgs {
    SsmBwdArgs a;
    int Dg, nblk;
    Segments seg;
    float *keep;                     // [B][ceil(T / kTok)][N][D]
    RowBuf rows;                     // B and C in scalar order
    SegBuf rev;                      // segment p's local gradient (slot p) and sum of delta (slot p)
    float *part_bc;                  // [nblk][B][T][G][2][N]
    float *part_a;                   // [B][P][D][N]
    float *part_d;                   // [B][P][2][D]: dD, ddt_bias
};

// A segment's effect on the gradient that enters at its end: g_out = exp(A sum(delta)) g_in + g_local.
template <class P, int N>
__global__ __launch_bounds__(64 * N / states_per_wave<N>()) void seg_grad_kernel(const RevArgs k) {
    using R = typename P::R;
    constexpr int NS = states_per_wave<N>(), NW = N / NS, TPW = kTile / NW, GT = NS == 2 ? 8 : 4;
    __shared__ float2 s_in[2][kTile][64];
    const SsmBwdArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk, nseg = k.seg.P - 1;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = 1 + bp % nseg, b = bp / nseg;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const uint32_t ch = g * k.Dg + min(c_in, k.Dg - 1);
    const int n0 = wave * NS;
    const size_t D = a.D, row0 = static_cast<size_t>(b) * a.T;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int tb = p * k.seg.len, te = max(min(len, tb + k.seg.len), tb), ntile = (te - tb + kTile - 1) / kTile;
    float A2[NS], G[NS] = {}, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = decay_rate(a.A[static_cast<size_t>(ch) * N + n0 + i]);
    const R *dt = static_cast<const R *>(a.dt) + row0 * D;
    const R *d_o = static_cast<const R *>(a.d_o) + row0 * D;
    const bool gated = a.z != nullptr;
    const R *z = gated ? static_cast<const R *>(a.z) + row0 * D : d_o;
    const float *Cw = k.rows.c + ((static_cast<size_t>(b) * a.G + g) * NW + wave) * k.rows.Tp * NS;
    const float dt_bias = a.dt_bias ? a.dt_bias[ch] : 0.f;

    struct Raw {
        R dt[TPW], z[TPW], d_o[TPW];
    };
    auto fetch = [&](int tile, Raw &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const size_t t = max(min(tb + tile * kTile + wave + j * NW, te - 1), tb);
            r.dt[j] = (dt + t * D)[ch];
            r.d_o[j] = (d_o + t * D)[ch];
            r.z[j] = (z + t * D)[ch];
        }
    };
    auto stage = [&](int tile, const Raw &r) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const bool in = tb + tile * kTile + wave + j * NW < te;
            const float x = P::to_f32(r.dt[j]) + dt_bias, d = P::to_f32(r.d_o[j]), gate = siluf(P::to_f32(r.z[j]));
            const float delta = a.softplus ? softplusf(x) : x;
            s_in[tile & 1][wave + j * NW][lane] = in ? make_float2(delta, gated ? d * gate : d) : make_float2(0.f, 0.f);
        }
    };
    ScalarRows<GT, NS> rc;
    auto step = [&](int tile, Raw &r) {      // r: the rows of tile - 1, refilled with tile - 3
#pragma unroll
        for (int j = kTile - GT; j >= 0; j -= GT) {
            const int t0 = tb + tile * kTile + j;
            float2 in[GT];
#pragma unroll
            for (int t = 0; t < GT; ++t) in[t] = s_in[tile & 1][j + t][lane];
            const ScalarRows<GT, NS> c = rc;
#pragma unroll
            for (int t = 0; t < GT; ++t) asm volatile("" ::"v"(in[t].x), "v"(in[t].y), "s"(c.v[t][0]));
            __builtin_amdgcn_sched_barrier(0);
            rc.load(Cw + static_cast<size_t>(max(t0 - GT, 0)) * NS);
            __builtin_amdgcn_sched_barrier(0);
            float e[GT][NS], x[GT][NS];
#pragma unroll
            for (int t = 0; t < GT; ++t)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    e[t][i] = __builtin_amdgcn_exp2f(in[t].x * A2[i]);
                    x[t][i] = in[t].y * c.v[t][i];
                }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = GT - 1; t >= 0; --t) {
                sum += in[t].x;
#pragma unroll
                for (int i = 0; i < NS; ++i) G[i] = e[t][i] * (x[t][i] + G[i]);
            }
        }
        if (tile > 0) stage(tile - 1, r);
        fetch(tile - 3, r);
        __syncthreads();
    };
    Raw r0, r1;
    {
        Raw first;
        fetch(ntile - 1, first);
        fetch(ntile - 2, r0);
        fetch(ntile - 3, r1);
        rc.load(Cw + static_cast<size_t>(tb + (ntile - 1) * kTile + kTile - GT) * NS);
        stage(ntile - 1, first);
    }
    __syncthreads();
    int tile = ntile - 1;
    for (; tile > 0; tile -= 2) {
        step(tile, r0);
        step(tile - 1, r1);
    }
    if (tile == 0) step(0, r0);
    if (c_in >= k.Dg) return;
    float *out = k.rev.h + ((static_cast<size_t>(b) * k.seg.P + p) * N + n0) * D + ch;
#pragma unroll
    for (int i = 0; i < NS; ++i) out[i * D] = G[i];
    if (wave == 0) k.rev.s[(static_cast<size_t>(b) * k.seg.P + p) * D + ch] = sum;
}

// Eight waves a workgroup, one token of a tile each to stage and finish.
constexpr int kBwdWaves = kTok;
template <class P, int N>
__global__ __launch_bounds__(64 * kBwdWaves) void ssm_bwd_kernel(const RevArgs k) {
    using R = typename P::R;
    constexpr int NW = kBwdWaves, NS = N / NW;
    constexpr int NR = states_per_wave<N>(), SUB = NS / NR;          // states of a scalar row, rows a wave
    constexpr int RT = NS <= 4 ? kTok : kTok / 2;                    // tokens whose B and C are in scalar registers
    constexpr int VPT = 2 * NS, TPC = 16 / VPT, SETS = kTok / TPC;   // channel sums: values a token, tokens and sets of 16
    // Decays of a tile stay in registers; at eight states they do not fit, and also without them that
    // instance spills 63 of its 256 registers (252 bytes of scratch a lane).
    constexpr bool kHold = NS <= 4;
    constexpr int kPitch = 20;       // floats a lane in s_v: 16-byte accesses of eight lanes meet no bank twice
    __shared__ float2 s_in[2][kTok][64];
    __shared__ float s_dy[2][kTok][64];
    __shared__ float s_p[2][NW][3][kTok][64];
    __shared__ __attribute__((aligned(16))) float s_v[NW][64 * kPitch];
    const SsmBwdArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = bp % k.seg.P, b = bp / k.seg.P;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const bool live = c_in < k.Dg;
    const uint32_t ch = g * k.Dg + min(c_in, k.Dg - 1);
    const int n0 = wave * NS;
    const size_t D = a.D, row0 = static_cast<size_t>(b) * a.T;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int tb = p * k.seg.len, te = max(min(len, tb + k.seg.len), tb), ntile = (te - tb + kTok - 1) / kTok;
    const size_t st = (static_cast<size_t>(b) * D + ch) * N + n0;

    float A2[NS], G[NS], dA[NS] = {};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[static_cast<size_t>(ch) * N + n0 + i]);
        G[i] = a.dS_T && live ? a.dS_T[st + i] : 0.f;
    }
    for (int q0 = k.seg.P - 1; q0 > p; q0 -= kCompose) {
        float local[kCompose][NS], sum[kCompose];
#pragma unroll
        for (int j = 0; j < kCompose; ++j) {
            const size_t q = static_cast<size_t>(b) * k.seg.P + max(q0 - j, p + 1);
            sum[j] = k.rev.s[q * D + ch];
#pragma unroll
            for (int i = 0; i < NS; ++i) local[j][i] = k.rev.h[(q * N + n0 + i) * D + ch];
        }
#pragma unroll
        for (int j = 0; j < kCompose; ++j)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                G[i] = !live ? 0.f : q0 - j > p ? carry(A2[i], sum[j], G[i], local[j][i]) : G[i];
    }
    const R *u = static_cast<const R *>(a.u) + row0 * D;
    const R *dt = static_cast<const R *>(a.dt) + row0 * D;
    const R *d_o = static_cast<const R *>(a.d_o) + row0 * D;
    const bool gated = a.z != nullptr;
    const R *z = gated ? static_cast<const R *>(a.z) + row0 * D : u;
    // The gradients of padding, before the walk: behind it, where its registers live on, 690
    // instead of 679 us at the size above.
    for (int t = te + wave; live && t < min(a.T, tb + k.seg.len); t += NW) {     // padding
        const size_t at = (row0 + t) * D;
        (static_cast<R *>(a.du) + at)[ch] = P::from_f32(0.f);
        (static_cast<R *>(a.ddt) + at)[ch] = P::from_f32(0.f);
        if (gated) (static_cast<R *>(a.dz) + at)[ch] = P::from_f32(0.f);
    }
    const size_t row_step = static_cast<size_t>(k.rows.Tp) * NR;
    const size_t rows = ((static_cast<size_t>(b) * a.G + g) * (N / NR) + wave * SUB) * row_step;
    const float *Bw = k.rows.b + rows, *Cw = k.rows.c + rows;
    const float dt_bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.Dskip ? a.Dskip[ch] : 0.f;
    const size_t nc = (a.T + kTok - 1) / kTok;
    const float *keep = k.keep + ((static_cast<size_t>(b) * nc + tb / kTok) * N + n0) * D;
    float *part_bc = k.part_bc + (((static_cast<size_t>(cb % k.nblk) * a.B + b) * a.T) * a.G + g) * 2 * N + n0;
    float acc_d = 0.f, acc_b = 0.f;

    struct Raw {                     // as loaded: a conversion would wait for the load
        R u, x, z, d_o;
        float h[NS];                 // the tile's entry state
    };
    auto fetch = [&](int tile, Raw &r) {
        tile = max(tile, 0);
        const size_t t = min(tb + tile * kTok + wave, te - 1);
        r.u = (u + t * D)[ch];
        r.x = (dt + t * D)[ch];
        r.d_o = (d_o + t * D)[ch];
        r.z = (z + t * D)[ch];
#pragma unroll
        for (int i = 0; i < NS; ++i) r.h[i] = (keep + (static_cast<size_t>(tile) * N + i) * D)[ch];
    };
    struct Kept {                    // what the end of a token needs, and the tile's entry state
        float u, slope, dgate, delta, dy, h[NS];   // dgate: d_o silu'(z)
    };
    // Tokens past the end and lanes past the channels enter with delta, u, dy and state zero: the
    // state passes through them and they add nothing to any sum.
    auto stage = [&](int tile, const Raw &r, Kept &f) {
#pragma unroll
        for (int i = 0; i < NS; ++i) f.h[i] = live ? r.h[i] : 0.f;
        const bool in = live && tb + tile * kTok + wave < te;
        f.u = P::to_f32(r.u);
        const float z = P::to_f32(r.z), d = P::to_f32(r.d_o), x = P::to_f32(r.x) + dt_bias;
        const float s = sigmoidf(z);
        const Softplus sp = softplus_grad(x);
        f.delta = a.softplus ? sp.value : x;
        f.slope = a.softplus ? sp.slope : 1.f;
        f.dy = gated ? d * (z * s) : d;
        f.dgate = d * (s * fmaf(z, 1.f - s, 1.f));
        s_in[tile & 1][wave][lane] = in ? make_float2(f.delta, f.delta * f.u) : make_float2(0.f, 0.f);
        s_dy[tile & 1][wave][lane] = in ? f.dy : 0.f;
    };

    // Channel sums.  A set of 16 values a lane goes to LDS as it is; a lane reads four of them
    // from every sixteenth lane, adds those, and six exchanges join the 16 readers of a value.
    float *mine = s_v[wave];
    auto put = [&](const float (&v)[16]) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4 *>(mine + lane * kPitch + 4 * j) = f32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    struct Quads {
        f32x4 q[4];
    };
    auto take = [&](Quads &r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.q[j] = *reinterpret_cast<const f32x4 *>(mine + ((lane >> 2) + 16 * j) * kPitch + 4 * (lane & 3));
    };
    // Lane l gets the sum of value 4 (l % 4) + {0, 2, 1, 3}[l / 16].
    auto join = [&](const Quads &r) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (r.q[0][i] + r.q[1][i]) + (r.q[2][i] + r.q[3][i]);
        auto half = [](float x, float y) {       // lanes 0-31: x over both halves; 32-63: y
            const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
            return __uint_as_float(p[0]) + __uint_as_float(p[1]);
        };
        const float lo = half(v[0], v[1]), hi = half(v[2], v[3]);
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        float x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
        x += dpp_src<0x124, 0xf>(x);             // row_ror:4
        x += dpp_src<0x128, 0xf>(x);             // row_ror:8
        return x;
    };

    ScalarRows<RT, NR> rb[SUB], rc[SUB];         // B and C of RT tokens, loaded a part of a tile ahead
    auto load_rows = [&](int t0) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            rb[j].load(Bw + j * row_step + static_cast<size_t>(max(t0, 0)) * NR);
            rc[j].load(Cw + j * row_step + static_cast<size_t>(max(t0, 0)) * NR);
        }
    };
    // The sums of four sets (or all of a tile's) from token t0 on: set (l / 4) % 4 in lane l.
    auto emit = [&](int t0, float x) {
        const int set = (lane >> 2) & 3, row = lane >> 4;
        const int v = 4 * (lane & 3) + (row == 1 ? 2 : row == 2 ? 1 : row), t = t0 + set * TPC + v / VPT, e = v % VPT;
        if (set < SETS && t < te) part_bc[static_cast<size_t>(t) * a.G * 2 * N + (e / NS) * N + e % NS] = x;
    };
    auto walk = [&](int tile, const float (&h_in)[NS], auto between) {
        const int t0 = tb + tile * kTok, buf = tile & 1;
        float2 in[kTok];
        float dy[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            in[t] = s_in[buf][t][lane];
            dy[t] = s_dy[buf][t][lane];
        }
        float dec[kTok][NS], h[kTok][NS];
        auto advance = [&](int t) {
#pragma unroll
            for (int i = 0; i < NS; ++i) h[t][i] = fmaf(dec[t][i], t ? h[t - 1][i] : h_in[i], h[t][i]);
        };
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            if (RT < kTok && t % RT == 0) {
#pragma unroll
                for (int j = 0; j < SUB; ++j) rb[j].load(Bw + j * row_step + static_cast<size_t>(t0 + t) * NR);
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                dec[t][i] = __builtin_amdgcn_exp2f(in[t].x * A2[i]);
                h[t][i] = in[t].y * rb[i / NR].v[t % RT][i % NR];
            }
            if (!kHold) advance(t);
        }
        between();
        __builtin_amdgcn_s_setprio(1);           // as in the forward: the recurrence before staging
        __builtin_amdgcn_sched_barrier(0);
        if (kHold) {
#pragma unroll
            for (int t = 0; t < kTok; ++t) advance(t);
        } else {                     // the same decays again on the way back, not kept: A2 is made to look new
#pragma unroll
            for (int i = 0; i < NS; ++i) asm volatile("" : "+v"(A2[i]));
        }
        if (RT < kTok) {             // the upper half's C comes while the states are walked
#pragma unroll
            for (int j = 0; j < SUB; ++j) rc[j].load(Cw + j * row_step + static_cast<size_t>(t0 + kTok - RT) * NR);
        }
        float dAt[NS] = {};          // this tile's part of dA: fewer roundings against the long sum
        float val[16], out = 0.f;
        Quads due;
#pragma unroll
        for (int t = kTok - 1; t >= 0; --t) {
            if (RT < kTok && t == RT - 1) load_rows(t0);
            float y = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float b = rb[i / NR].v[t % RT][i % NR], c = rc[i / NR].v[t % RT][i % NR];
                const float gi = fmaf(c, dy[t], G[i]);
                val[(t % TPC) * VPT + i] = gi * in[t].y;
                val[(t % TPC) * VPT + NS + i] = dy[t] * h[t][i];
                y = i ? fmaf(c, h[t][i], y) : c * h[t][0];
                s1 = i ? fmaf(gi, b, s1) : gi * b;
                G[i] = (kHold ? dec[t][i] : __builtin_amdgcn_exp2f(in[t].x * A2[i])) * gi;
                const float q = G[i] * (t ? h[t - 1][i] : h_in[i]);
                s2 = i ? fmaf(A2[i], q, s2) : A2[0] * q;
                dAt[i] = fmaf(in[t].x, q, dAt[i]);
            }
            float *sp = &s_p[buf][wave][0][t][lane];
            sp[0] = y;
            sp[kTok * 64] = s1;
            sp[2 * kTok * 64] = s2;
            if (t % TPC == 0) {      // a set is whole: join the one before, whose values have arrived
                constexpr int last = SETS - 1;
                const int set = t / TPC;
                if (set < last) {
                    const float x = join(due);           // by every lane
                    out = ((lane >> 2) & 3) == ((set + 1) & 3) ? x : out;
                }
                if (SETS > 4 && set + 1 == 4) emit(t0 + 4 * TPC, out);
                put(val);
                take(due);
            }
        }
        if (RT == kTok) load_rows(t0 - kTok);
#pragma unroll
        for (int i = 0; i < NS; ++i) dA[i] += dAt[i];
        const float x = join(due);
        emit(t0, ((lane >> 2) & 3) == 0 ? x : out);
    };
    struct Sums {
        float v[3][NW];
    };
    auto gather = [&](int tile, Sums &s) {
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int v = 0; v < 3; ++v) s.v[v][w] = s_p[tile & 1][w][v][wave][lane];
    };
    auto finish = [&](int tile, const Sums &s, const Kept &r) {
        const int t = tb + tile * kTok + wave;
        float y = s.v[0][0], s1 = s.v[1][0], s2 = s.v[2][0];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            y += s.v[0][w];
            s1 += s.v[1][w];
            s2 += s.v[2][w];
        }
        const float dd = fmaf(r.u, s1, s2 * kLn2) * r.slope;
        const bool in = t < te;
        acc_d = in ? fmaf(r.dy, r.u, acc_d) : acc_d;
        acc_b += in ? dd : 0.f;
        const float du = fmaf(r.delta, s1, skip * r.dy);
        const float dz = r.dgate * fmaf(skip, r.u, y);
        if (live && in) {
            const size_t at = (row0 + t) * D;
            (static_cast<R *>(a.du) + at)[ch] = P::from_f32(du);
            (static_cast<R *>(a.ddt) + at)[ch] = P::from_f32(dd);
            if (gated) (static_cast<R *>(a.dz) + at)[ch] = P::from_f32(dz);
        }
    };

    // As in the forward: rows two tiles ahead in two sets by name, a tile's end among the next
    // tile's arithmetic.
    Kept cur, old;
    auto step = [&](int tile, Raw &r) {
        Sums s;
        gather(tile + 1, s);
        walk(tile, cur.h, [&] {
            if (tile + 1 < ntile) finish(tile + 1, s, old);
        });
        __builtin_amdgcn_s_setprio(0);
        old = cur;
        if (tile > 0) stage(tile - 1, r, cur);
        fetch(tile - 3, r);
        __syncthreads();
    };
    if (ntile > 0) {                 // none: the segment lies past the sequence's end
        Raw r0, r1;
        {
            Raw first;
            fetch(ntile - 1, first);
            fetch(ntile - 2, r0);
            fetch(ntile - 3, r1);
            if (RT == kTok) load_rows(tb + (ntile - 1) * kTok);
            stage(ntile - 1, first, cur);
        }
        old = cur;
        __syncthreads();
        int tile = ntile - 1;
        for (; tile > 0; tile -= 2) {
            step(tile, r0);
            step(tile - 1, r1);
        }
        if (tile == 0) step(0, r0);
        Sums s;
        gather(0, s);
        finish(0, s, old);
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

// The sums over workgroups, in one launch: dA's columns, those of dD and ddt_bias, and dB and
// dC from the channel blocks' sums, added in block order.
struct SumGrid {
    unsigned a, d, bc;               // workgroups of each
};
template <class P>
__global__ __launch_bounds__(kColThreads) void ssm_sums_kernel(const RevArgs k, const SumGrid grid) {
    using R = typename P::R;
    __shared__ ColShared sh;
    const int N = k.a.N, segs = k.a.B * k.seg.P;
    const unsigned blk = blockIdx.x;
    if (blk < grid.a) {
        column_sum_block(k.part_a, segs, static_cast<long long>(k.a.D) * N, blk, StoreA{k.a.dA}, sh);
        return;
    }
    if (blk < grid.a + grid.d) {
        column_sum_block(k.part_d, segs, 2LL * k.a.D, blk - grid.a, StoreD{k.a.dD, k.a.ddt_bias, k.a.D}, sh);
        return;
    }
    const long long rows = static_cast<long long>(k.a.B) * k.a.T * k.a.G;
    const long long i = (static_cast<long long>(blk - grid.a - grid.d) * kColThreads + threadIdx.x) * 4;   // four states of a row
    if (i >= rows * 2 * N) return;
    f32x4 s = zero4();
    const long long row = i / (2 * N);
    int b = 0;
    if (k.a.lens) {                  // rows of padding were not written: nothing to add
        const long long token = row / k.a.G;
        if (token % k.a.T >= k.a.lens[token / k.a.T]) b = k.nblk;
    }
    for (; b + 3 < k.nblk; b += 4) {
        f32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const f32x4 *>(k.part_bc + static_cast<size_t>(b + j) * rows * 2 * N + i);
        s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; b < k.nblk; ++b) s += *reinterpret_cast<const f32x4 *>(k.part_bc + static_cast<size_t>(b) * rows * 2 * N + i);
    const int e = static_cast<int>(i % (2 * N));
    R *out = static_cast<R *>(e < N ? k.a.dB : k.a.dC) + row * N + (e < N ? e : e - N);
    P::st4(out, s);
}

// With no tokens the gradients of what the tokens share are zero and dS0 is dS_T.
__global__ __launch_bounds__(256) void ssm_bwd_empty_kernel(const SsmBwdArgs a) {
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x, DN = static_cast<size_t>(a.D) * a.N;
    if (i < DN) a.dA[i] = 0.f;
    if (i < static_cast<size_t>(a.D)) {
        if (a.dD) a.dD[i] = 0.f;
        if (a.ddt_bias) a.ddt_bias[i] = 0.f;
    }
    for (size_t j = i; a.dS0 && j < a.B * DN; j += static_cast<size_t>(gridDim.x) * 256) a.dS0[j] = a.dS_T ? a.dS_T[j] : 0.f;
}

// Segments of the time axis: a workgroup (eight waves) for every compute unit, down to one tile
// a segment.  3 x 203 tokens, 142 channels in two groups, 32 states: 56 us; segments of at least
// 32 tokens 64, 64 tokens 85, 96 tokens 106.  The count is rounded up, so between half a card of
// workgroups and a whole one the cut brings the reverse walk nothing: 4096 tokens of 16 states take
// 1586 us with 150 workgroups, 1643 with 255 and, uncut, 1353 with 256.
Segments bwd_segments(int B, int T, int D, int G, int N) {
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    const long long waves = static_cast<long long>(B) * G * ((D / G + 63) / 64) * kBwdWaves;
    if (waves == 0) return cut_time(T, 1);
    const long long want = (8LL * cus + waves - 1) / waves;
    return cut_time(T, want);
}

struct Sizes {                       // floats of each part of the workspace, every one a multiple of four
    size_t rows, seg_h, seg_s, keep, bc, pa, pd;
    size_t total() const { return rows + 2 * (seg_h + seg_s) + keep + bc + pa + pd; }
};
size_t up4(size_t n) { return (n + 3) & ~static_cast<size_t>(3); }
Sizes sizes(int B, int T, int D, int G, int N, Segments s) {
    Sizes z;
    const size_t b = B, d = D, n = N, P = s.P, nc = (T + kTok - 1) / kTok, nblk = (D / G + 63) / 64;
    z.rows = row_floats(B, T, G, N);
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
    const unsigned per = static_cast<unsigned>(k.a.B) * k.a.G * k.nblk;
    if (k.seg.P > 1)
        hipLaunchKernelGGL((seg_grad_kernel<P, N>), dim3(per * (k.seg.P - 1)), dim3(64 * N / states_per_wave<N>()), 0, stream, k);
    hipLaunchKernelGGL((ssm_bwd_kernel<P, N>), dim3(per * k.seg.P), dim3(64 * kBwdWaves), 0, stream, k);
    const long long n4 = static_cast<long long>(k.a.B) * k.a.T * k.a.G * 2 * N / 4;
    SumGrid grid;
    grid.a = static_cast<unsigned>((static_cast<long long>(k.a.D) * N + 63) / 64);
    grid.d = k.a.dD || k.a.ddt_bias ? static_cast<unsigned>((2LL * k.a.D + 63) / 64) : 0;
    grid.bc = static_cast<unsigned>((n4 + kColThreads - 1) / kColThreads);
    hipLaunchKernelGGL((ssm_sums_kernel<P>), dim3(grid.a + grid.d + grid.bc), dim3(kColThreads), 0, stream, k, grid);
    return hipGetLastError();
}
template <class P>
hipError_t run_bwd_n(const RevArgs &k, hipStream_t stream) {
    if (k.a.N == 16) return run_bwd<P, 16>(k, stream);
    if (k.a.N == 32) return run_bwd<P, 32>(k, stream);
    return run_bwd<P, 64>(k, stream);
}

}  // namespace

size_t ssm_bwd_workspace(int B, int T, int D, int G, int N) {
    if (static_cast<long long>(B) * T * D == 0) return 0;
    return sizes(B, T, D, G, N, bwd_segments(B, T, D, G, N)).total() * sizeof(float);
}

hipError_t launch_ssm_bwd(int dtype, const SsmBwdArgs &a, void *ws, hipStream_t stream) {
    if (static_cast<long long>(a.B) * a.T == 0) {
        const size_t n = static_cast<size_t>(a.D) * a.N;
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
    k.rows = row_buf(w, a.B, a.T, a.G, a.N);
    w += z.rows;
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
    f.A = a.A; f.dt_bias = a.dt_bias; f.S0 = a.S0; f.lens = a.lens;
    f.B = a.B; f.T = a.T; f.D = a.D; f.G = a.G; f.N = a.N;
    f.softplus = a.softplus;
    launch_ssm_rows(dtype, f, k.rows, stream);
    const hipError_t err = launch_ssm_states(dtype, f, k.seg, fwd, k.rows, k.keep, stream);
    if (err != hipSuccess) return err;
    return dtype == 1 ? run_bwd_n<Bf16>(k, stream) : run_bwd_n<F32>(k, stream);
}

}  // namespace qd
