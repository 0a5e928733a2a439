// Selective state space scan for gfx950.  Per sequence, channel d and state n:
//
//   delta_t = softplus(dt_t + dt_bias)      (or dt_t + dt_bias itself)
//   h_t[n]  = exp(delta_t A[d, n]) h_{t-1}[n] + delta_t u_t B_t[n]
//   o_t     = (sum_n C_t[n] h_t[n] + D_d u_t) silu(z_t)
//
// with B and C shared by the channels of a group.  One exponential and four multiply-adds a
// token, channel and state against four to eight bytes a token and channel: instruction issue
// bounds it, not HBM.  The decay differs by channel and state, so there is no matrix product
// in it; the design keeps everything else off the vector units:
//   - a lane owns one channel and a wave NS of its N states, so the recurrence and the sum
//     over the wave's states need no exchange between lanes, and B_t and C_t are the same
//     for all lanes: they are scalar registers (RowBuf);
//   - the N / NS waves of a workgroup share 64 channels.  They stage delta_t and delta_t u_t
//     of a tile of kTile tokens once, each wave a part of the tokens, double-buffered in LDS;
//   - the waves' partial sums over their states meet in LDS, and the wave that staged a
//     token adds them up, applies D and the gate from the u and z it kept, and stores.
// One barrier a tile.  States and sums are fp32.  A wave in its recurrence goes before one that
// stages or waits (s_setprio): with two workgroups a compute unit 5 % (16 x 2048 tokens, 4096
// channels, 16 states 538 -> 522 us).
//
// 8 x 4096 tokens, 2048 channels, 16 states, bf16, gated: 340 us, 7 operations a token, channel
// and state at 25 TFLOP/s; one exponential and four multiply-adds alone would take 145 us at
// the rate that four waves a SIMD reach (21.2 cycles for 64 lanes), the 537 MB 105 us.  What is
// between: softplus, the gate and the sums over waves (a third of the vector instructions),
// and with one workgroup a compute unit two waves a SIMD do not cover each other's waits (at
// two workgroups the same work takes 258 us).
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
    RowBuf rows;
    float *keep;                     // kKeep: [B][ceil(T / kTok)][N][D]
};

// B and C in scalar order; one thread a token and wave.
template <class P, int NS>
__global__ __launch_bounds__(256) void ssm_rows_kernel(const ScanArgs k) {
    using R = typename P::R;
    const SsmArgs &a = k.a;
    const int NW = a.N / NS;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(a.B) * a.G * k.rows.Tp * NW) return;
    // threads next to each other take a row's waves, so that the reads are whole rows
    const int w = static_cast<int>(i % NW), t = static_cast<int>(i / NW % k.rows.Tp);
    const int bg = static_cast<int>(i / NW / k.rows.Tp), g = bg % a.G, b = bg / a.G;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    float vb[NS] = {}, vc[NS] = {};
    if (t < len) {
        const size_t at = ((static_cast<size_t>(b) * a.T + t) * a.G + g) * a.N + w * NS;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            vb[j] = P::to_f32(static_cast<const R *>(a.Bm)[at + j]);
            vc[j] = P::to_f32(static_cast<const R *>(a.Cm)[at + j]);
        }
    }
    const size_t to = ((static_cast<size_t>(bg) * NW + w) * k.rows.Tp + t) * NS;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        k.rows.b[to + j] = vb[j];
        k.rows.c[to + j] = vc[j];
    }
}

// PAIR: a lane stages two neighbouring channels of one token, the wave's halves two tokens: half
// the loads, stores and LDS accesses of one channel and token a lane.  It needs an even number
// of channels in a group and two tokens a wave (N = 16, 32).
// TILE tokens are staged at a time.  With 32 there are half the barriers, and each group's inputs
// come while the group before it is computed.
template <class P, int N, int MODE, bool PAIR, int TILE>
__global__ __launch_bounds__(64 * N / states_per_wave<N>()) void scan_kernel(const ScanArgs k) {
    using R = typename P::R;
    constexpr int NS = states_per_wave<N>(), NW = N / NS, TPW = TILE / NW;
    constexpr int CPL = PAIR ? 2 : 1, SLOTS = TPW / CPL;     // channels a lane stages, and how often
    static_assert(SLOTS >= 1, "pairs of tokens");
    struct __attribute__((aligned(CPL * P::kBytes))) Cell {
        R v[CPL];
    };
    constexpr int GT = NS == 2 ? 8 : 4;      // tokens whose B and C are in scalar registers
    constexpr bool kLong = TILE > kTile;
    static_assert(TPW >= 1 && TPW * NW == TILE, "each wave stages a whole number of tokens");
    __shared__ __attribute__((aligned(16))) float2 s_in[2][TILE][64];
    __shared__ __attribute__((aligned(16))) float s_y[MODE == kOut ? 2 : 1][MODE == kOut ? NW : 1][TILE][64];
    const SsmArgs &a = k.a;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int ncb = a.G * k.nblk, nseg = MODE == kSeg ? k.seg.P - 1 : k.seg.P;
    const int cb = blockIdx.x % ncb, bp = blockIdx.x / ncb, p = bp % nseg, b = bp / nseg;
    const int g = cb / k.nblk, c_in = (cb % k.nblk) * 64 + lane;
    const bool live = c_in < k.Dg;
    const uint32_t ch = g * k.Dg + min(c_in, k.Dg - 1);
    const int n0 = wave * NS;
    const size_t D = a.D;
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int tb = p * k.seg.len, te = min(len, tb + k.seg.len);

    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[static_cast<size_t>(ch) * N + n0 + i]);
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
        for (int q0 = 0; q0 < p; q0 += kCompose) {
            float local[kCompose][NS], sum[kCompose];
#pragma unroll
            for (int j = 0; j < kCompose; ++j) {
                const size_t q = min(q0 + j, p - 1);
                sum[j] = seg_s[q * D];
#pragma unroll
                for (int i = 0; i < NS; ++i) local[j][i] = seg_h[(q + 1) * N * D + i * D];
            }
#pragma unroll
            for (int j = 0; j < kCompose; ++j)
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = q0 + j < p ? carry(A2[i], sum[j], h[i], local[j][i]) : h[i];
        }
    }
    if (MODE == kSeg) {              // the local effect starts from zero
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = 0.f;
    }
    // A segment's sum of delta: pairs add what they stage, a sixteenth of the additions (16384 tokens
    // of one sequence 252 -> 248 us); one channel a lane, every wave adds as it walks (odd channel
    // counts, 2 x 4096 tokens: 130 us against 135).
    constexpr bool kStagedSum = MODE == kSeg && PAIR;
    float sum_delta = 0.f;

    if (tb < te) {
        const size_t row0 = static_cast<size_t>(b) * a.T;
        const R *u = static_cast<const R *>(a.u) + row0 * D;
        const R *dt = static_cast<const R *>(a.dt) + row0 * D;
        const bool gated = a.z != nullptr;
        const R *z = gated ? static_cast<const R *>(a.z) + row0 * D : u;
        R *o = MODE == kOut ? static_cast<R *>(a.o) + row0 * D : nullptr;
        const size_t rows = ((static_cast<size_t>(b) * a.G + g) * NW + wave) * k.rows.Tp * NS;
        const float *Bw = k.rows.b + rows, *Cw = k.rows.c + rows;
        const int ntile = (te - tb + TILE - 1) / TILE;

        // What this lane stages: channels sc, .. of the block, token `sub` of each slot's CPL.
        const int sc = PAIR ? 2 * (lane & 31) : lane, sub = PAIR ? lane >> 5 : 0;
        const int s_in_blk = (cb % k.nblk) * 64 + sc;
        const bool s_live = s_in_blk < k.Dg;
        const uint32_t s_ch = g * k.Dg + min(s_in_blk, k.Dg - CPL), s_off = sub * a.D + s_ch;
        float dt_bias[CPL], skip[CPL], staged[CPL] = {};
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            dt_bias[c] = a.dt_bias ? a.dt_bias[s_ch + c] : 0.f;
            skip[c] = a.Dskip ? a.Dskip[s_ch + c] : 0.f;
        }
        auto slot_token = [&](int j) { return CPL * (wave + j * NW); };     // the slot's first token in the tile

        // Loaded values stay as they came until they are used: a conversion would wait for the
        // load.  Rows at and past the end read the last row instead; what they give is not used.
        struct Raw {
            Cell u[SLOTS], dt[SLOTS], z[SLOTS];
            float line;
        };
        auto fetch = [&](int tile, Raw &r) {
            // The lines of the tile's scalar loads come to L2 with it: half the lanes for B, half for C.
            const int tl = min(tb + tile * TILE, (te - 1) / TILE * TILE);
            r.line = (lane < 32 ? Bw : Cw)[static_cast<size_t>(tl) * NS + (lane & 31) * (TILE * NS / 32)];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int t = min(tb + tile * TILE + slot_token(j), te - 1);
                const size_t row = static_cast<size_t>(t) * D;
                const uint32_t at = t + CPL <= te ? s_off : s_ch;
                r.u[j] = *reinterpret_cast<const Cell *>(u + row + at);
                r.dt[j] = *reinterpret_cast<const Cell *>(dt + row + at);
                if (MODE == kOut) r.z[j] = *reinterpret_cast<const Cell *>(z + row + at);
            }
        };
        struct Kept {                // what the end of a token needs of its rows
            float u[SLOTS][CPL], z[SLOTS][CPL];
        };
        // Tokens past the end enter with delta and delta u zero (and B, C are zero there): the
        // state passes through them.
        auto stage = [&](int tile, const Raw &r) {
            Kept f;
            asm volatile("" ::"v"(r.line));
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int i = slot_token(j) + sub;
                const bool in = tb + tile * TILE + i < te;
                float v[2 * CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const float x = P::to_f32(r.dt[j].v[c]) + dt_bias[c];
                    const float delta = a.softplus ? softplusf(x) : x;
                    f.u[j][c] = P::to_f32(r.u[j].v[c]);
                    f.z[j][c] = MODE == kOut ? P::to_f32(r.z[j].v[c]) : 0.f;
                    v[2 * c] = in ? delta : 0.f;
                    v[2 * c + 1] = in ? delta * f.u[j][c] : 0.f;
                    if constexpr (kStagedSum) staged[c] += v[2 * c];
                }
                if constexpr (PAIR) *reinterpret_cast<f32x4 *>(&s_in[tile & 1][i][sc]) = f32x4{v[0], v[1], v[2], v[3]};
                else s_in[tile & 1][i][sc] = make_float2(v[0], v[1]);
            }
            return f;
        };
        ScalarRows<GT, NS> rb, rc;           // the next group's B and C
        float2 ahead[kLong ? GT : 1];        // and, within a long tile, its inputs
        auto load_group = [&](int t0) {
            if constexpr (kLong) t0 = min(t0, k.rows.Tp - GT);     // past a long last tile there are no rows
            rb.load(Bw + static_cast<size_t>(t0) * NS);
            if constexpr (MODE == kOut) rc.load(Cw + static_cast<size_t>(t0) * NS);
        };
        auto keep_state = [&](int t0) {
            if (MODE == kKeep && live && t0 < te) {
                const size_t nc = (a.T + kTok - 1) / kTok;
                float *keep = k.keep + ((b * nc + t0 / kTok) * N + n0) * D;
#pragma unroll
                for (int i = 0; i < NS; ++i) (keep + i * D)[ch] = h[i];
            }
        };
        // GT tokens from t0 = tile start + j.  `between` is arithmetic of its own that the
        // compiler may place among the group's.
        auto group = [&](int tile, int j, auto between) {
            const int t0 = tb + tile * TILE + j;
            if (j % kTok == 0) keep_state(t0);
            float2 in[GT];
#pragma unroll
            for (int t = 0; t < GT; ++t) in[t] = kLong && j > 0 ? ahead[kLong ? t : 0] : s_in[tile & 1][j + t][lane];
            if constexpr (kLong) {
                if (j + GT < TILE) {
#pragma unroll
                    for (int t = 0; t < GT; ++t) ahead[t] = s_in[tile & 1][j + GT + t][lane];
                }
            }
            const ScalarRows<GT, NS> cb_ = rb, cc_ = rc;
            // Scalar and LDS loads count down together and out of order: the wait for this
            // group's is here, before the next group's scalar loads are issued, which then
            // have the whole group's arithmetic to arrive.
#pragma unroll
            for (int t = 0; t < GT; ++t) asm volatile("" ::"v"(in[t].x), "v"(in[t].y), "s"(cb_.v[t][0]));
            __builtin_amdgcn_sched_barrier(0);
            load_group(t0 + GT);
            __builtin_amdgcn_s_setprio(1);
            // The exponentials and inputs of the group first: independent, so their latency is hidden.
            float e[GT][NS], x[GT][NS];
#pragma unroll
            for (int t = 0; t < GT; ++t)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    e[t][i] = __builtin_amdgcn_exp2f(in[t].x * A2[i]);
                    x[t][i] = in[t].y * cb_.v[t][i];
                }
            between();
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = fmaf(e[t][i], h[i], x[t][i]);
                    if constexpr (MODE == kOut) y = i ? fmaf(cc_.v[t][i], h[i], y) : cc_.v[t][0] * h[0];
                }
                if constexpr (MODE == kOut) s_y[tile & 1][wave][j + t][lane] = y;
                else if constexpr (MODE == kSeg && !kStagedSum) sum_delta += in[t].x;
            }
        };
        // The tokens this wave staged: the waves' sums over their states, D, the gate, the store.
        struct Sums {
            float y[SLOTS][NW][CPL];
        };
        auto gather = [&](int tile, Sums &p) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float *from = &s_y[tile & 1][w][slot_token(j) + sub][sc];
                    if constexpr (PAIR) {
                        const float2 v = *reinterpret_cast<const float2 *>(from);
                        p.y[j][w][0] = v.x;
                        p.y[j][w][1] = v.y;
                    } else {
                        p.y[j][w][0] = *from;
                    }
                }
        };
        auto finish = [&](int tile, const Sums &p, const Kept &r) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int t0 = tb + tile * TILE + slot_token(j);
                Cell out;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    float y = skip[c] * r.u[j][c];
#pragma unroll
                    for (int w = 0; w < NW; ++w) y += p.y[j][w][c];
                    const float gate = siluf(r.z[j][c]);
                    y *= gated ? gate : 1.f;
                    out.v[c] = P::from_f32(y);
                }
                if (s_live && t0 + sub < te) *reinterpret_cast<Cell *>(o + static_cast<size_t>(t0) * D + s_off) = out;
            }
        };
        auto nothing = [] {};

        // Rows are on their way two tiles before they are staged, in two sets that take turns by
        // name (a copy would wait for its load): at tile i, `r` holds the rows of i + 1 and is
        // refilled with those of i + 3.  A tile's end runs among the next tile's arithmetic.
        Kept cur, old;
        auto step = [&](int i, Raw &r) {
            Sums p;
            if (MODE == kOut) gather(i - 1, p);
            group(i, 0, [&] {
                if (MODE == kOut && i > 0) finish(i - 1, p, old);
            });
#pragma unroll
            for (int j = GT; j < TILE; j += GT) group(i, j, nothing);
            __builtin_amdgcn_s_setprio(0);
            old = cur;
            cur = stage(i + 1, r);
            fetch(i + 3, r);
            __syncthreads();
        };
        Raw r0, r1;
        {
            Raw first;
            fetch(0, first);
            fetch(1, r0);
            fetch(2, r1);
            load_group(tb);
            cur = stage(0, first);
        }
        old = cur;
        __syncthreads();
        int i = 0;
        for (; i + 1 < ntile; i += 2) {
            step(i, r0);
            step(i + 1, r1);
        }
        if (i < ntile) step(i++, r0);
        if constexpr (MODE == kOut) {
            Sums p;
            gather(i - 1, p);
            finish(i - 1, p, old);
        }
        if constexpr (kStagedSum) {          // the sums meet where the inputs were
            float (*sums)[64] = reinterpret_cast<float (*)[64]>(&s_in[0][0][0]);
            static_assert(NW * CPL <= 2 * 2 * TILE, "rows of sums fit the tiles");
#pragma unroll
            for (int c = 0; c < CPL; ++c) sums[wave * CPL + sub][sc + c] = staged[c];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < NW * CPL; ++r) sum_delta += wave == 0 ? sums[r][lane] : 0.f;
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
// wave reads 1 KB in a row; kStepReps channels a lane are in flight.  256 sequences, 2048
// channels, 16 states: 14.5 us, 4.9 TB/s (one channel a lane 15.2 us, four 16.7).
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
            hp[i] = fmaf(__builtin_amdgcn_exp2f(delta * decay_rate(Ap[i])), hp[i], du * P::to_f32(Bm[i]));
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

// Segments of the time axis: where a call leaves a compute unit fewer than six waves, enough
// for sixteen, as long as a segment keeps at least 64 tokens (2 x 512 tokens, 1024 channels, 16
// states: 23 us; at least 128 tokens 30, 32 tokens 23, and 4 x 100 tokens then 23 against 21
// us).  With 2048 channels and 16 states, all of one build: 16384 tokens of one sequence 274 us
// (eight waves 343, twenty-four 280), 4 x 4096 tokens 272 us against 383 uncut; at 8 x 4096,
// eight waves a unit, the cut costs more than it gives (442 against 387 us).
Segments fwd_segments(int B, int T, int D, int G, int N) {
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    const long long waves = static_cast<long long>(B) * G * ((D / G + 63) / 64) * (N / states_per_wave_of(N));
    if (waves == 0 || waves >= 6LL * cus) return cut_time(T, 1);
    const long long want = (16LL * cus + waves - 1) / waves;
    return cut_time(T, want > T / 64 ? T / 64 : want);
}

// Tiles of 32 tokens, for 16 states and walks of at least 512 tokens in one piece.  The full walk's fill
// LDS, so they are for a compute unit with at most one workgroup: 8 x 4096 tokens, 2048 channels
// 362 -> 339 us, 8 x 2048 in fp32 201 -> 185, 6 x 2000 180 -> 170; 8 x 200 in fp32 26.7 -> 28.0.  With
// 32 or 64 states a wave has twice the independent work, and they bring nothing (32 states, 8 x 1024:
// 145 and 146 us).  The walk that keeps states (32 KB of LDS) takes them up to two workgroups a compute
// unit; gradients of 2048 channels with the short and the long tiles: 8 x 2048 tokens (256 workgroups)
// 699 and 688 us, 12 x 700 (384) 454 and 451, 16 x 1024 (512) 667 and 663; of 2112 channels, 8 x 2048
// (264) 1260 and 1244; of 4096, 16 x 512 (1024) 669 and 677; 16 x 100 (512) 95 and 98.
bool long_tiles(const ScanArgs &k, unsigned workgroups, int per_unit) {
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    return k.seg.P == 1 && k.a.T >= 512 && workgroups <= static_cast<unsigned>(per_unit * cus);
}

template <class P, int N, int MODE>
hipError_t run_scan(const ScanArgs &k, hipStream_t stream) {
    const dim3 blk(64 * N / states_per_wave<N>());
    const unsigned per = static_cast<unsigned>(k.a.B) * k.a.G * k.nblk;
    const dim3 first(per * (k.seg.P - 1)), all(per * k.seg.P);
    // Pairs: 369 against 386 us at 8 x 4096 tokens, 2048 channels, 16 states; the walk that keeps
    // states, with no output to finish, is 5 us slower with them.
    if constexpr (MODE != kKeep && kTile / (N / states_per_wave<N>()) >= 2) {
        if (k.Dg % 2 == 0) {         // with D = G Dg even every row starts on a pair
            if constexpr (MODE == kOut && N == 16) {
                if (long_tiles(k, per, 1)) {
                    hipLaunchKernelGGL((scan_kernel<P, N, kOut, true, 2 * kTile>), all, blk, 0, stream, k);
                    return hipGetLastError();
                }
            }
            if (k.seg.P > 1) hipLaunchKernelGGL((scan_kernel<P, N, kSeg, true, kTile>), first, blk, 0, stream, k);
            hipLaunchKernelGGL((scan_kernel<P, N, MODE, true, kTile>), all, blk, 0, stream, k);
            return hipGetLastError();
        }
    }
    if constexpr (MODE == kKeep && N == 16) {
        if (long_tiles(k, per, 2)) {
            hipLaunchKernelGGL((scan_kernel<P, N, kKeep, false, 2 * kTile>), all, blk, 0, stream, k);
            return hipGetLastError();
        }
    }
    if (k.seg.P > 1) hipLaunchKernelGGL((scan_kernel<P, N, kSeg, false, kTile>), first, blk, 0, stream, k);
    hipLaunchKernelGGL((scan_kernel<P, N, MODE, false, kTile>), all, blk, 0, stream, k);
    return hipGetLastError();
}

template <class P, int MODE>
hipError_t run_scan_n(const ScanArgs &k, hipStream_t stream) {
    if (k.a.N == 16) return run_scan<P, 16, MODE>(k, stream);
    if (k.a.N == 32) return run_scan<P, 32, MODE>(k, stream);
    return run_scan<P, 64, MODE>(k, stream);
}

ScanArgs scan_args(const SsmArgs &a, Segments seg, RowBuf rows) {
    ScanArgs k;
    k.a = a;
    k.Dg = a.D / a.G;
    k.nblk = (k.Dg + 63) / 64;
    k.seg = seg;
    k.buf = SegBuf{nullptr, nullptr};
    k.rows = rows;
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

// Every launch: up to 64 segments a channel block, 64 lanes for a wave's states; B and C in
// scalar order, a lane a token and wave; the sums over blocks, in one launch, take a lane for
// four values of dB and dC, and 16 for a value of dA.
bool ssm_fits(int B, int T, int D, int G, int N) {
    if (N != 16 && N != 32 && N != 64) return false;
    const long long blocks = static_cast<long long>(B) * G * ((D / G + 63) / 64), tiles = T / kTile + 1;
    const long long waves = N / states_per_wave_of(N), lim = (1LL << 32) - 1024;
    return blocks < (1LL << 31) && blocks * (tiles < 64 ? tiles : 64) * 64 * waves < lim &&
           static_cast<long long>(B) * T < (1LL << 31) && T < 0x7fffff00 &&
           static_cast<long long>(B) * G < (1LL << 31) && static_cast<long long>(B) * G * (T + 2LL * kTile) < lim / waves &&
           static_cast<long long>(B) * T * G < lim / N && static_cast<long long>(D) * N < (1LL << 26);
}

size_t row_floats(int B, int T, int G, int N) { return 2 * static_cast<size_t>(B) * G * N * padded_rows(T); }

RowBuf row_buf(float *ws, int B, int T, int G, int N) {
    return RowBuf{ws, ws + row_floats(B, T, G, N) / 2, padded_rows(T)};
}

void launch_ssm_rows(int dtype, const SsmArgs &a, RowBuf rows, hipStream_t stream) {
    const ScanArgs k = scan_args(a, Segments{1, a.T}, rows);
    const long long n = static_cast<long long>(a.B) * a.G * rows.Tp * (a.N / states_per_wave_of(a.N));
    const dim3 grid(static_cast<unsigned>((n + 255) / 256)), blk(256);
    if (a.N == 16) {
        constexpr int NS = states_per_wave<16>();
        if (dtype == 1) hipLaunchKernelGGL((ssm_rows_kernel<Bf16, NS>), grid, blk, 0, stream, k);
        else hipLaunchKernelGGL((ssm_rows_kernel<F32, NS>), grid, blk, 0, stream, k);
    } else {
        static_assert(states_per_wave<32>() == 4 && states_per_wave<64>() == 4, "one instance for both");
        if (dtype == 1) hipLaunchKernelGGL((ssm_rows_kernel<Bf16, 4>), grid, blk, 0, stream, k);
        else hipLaunchKernelGGL((ssm_rows_kernel<F32, 4>), grid, blk, 0, stream, k);
    }
}

size_t ssm_fwd_workspace(int B, int T, int D, int G, int N) {
    if (T == 0) return 0;
    const Segments s = fwd_segments(B, T, D, G, N);
    const size_t seg = s.P > 1 ? static_cast<size_t>(B) * s.P * D * (N + 1) : 0;
    return (row_floats(B, T, G, N) + seg) * sizeof(float);
}

hipError_t launch_ssm_fwd(int dtype, const SsmArgs &a, void *ws, hipStream_t stream) {
    float *w = static_cast<float *>(ws);
    ScanArgs k = scan_args(a, fwd_segments(a.B, a.T, a.D, a.G, a.N), row_buf(w, a.B, a.T, a.G, a.N));
    if (k.seg.P > 1) {
        k.buf.h = w + row_floats(a.B, a.T, a.G, a.N);
        k.buf.s = k.buf.h + static_cast<size_t>(a.B) * k.seg.P * a.N * a.D;
    }
    if (a.T > 0) launch_ssm_rows(dtype, a, k.rows, stream);
    return dtype == 1 ? run_scan_n<Bf16, kOut>(k, stream) : run_scan_n<F32, kOut>(k, stream);
}

hipError_t launch_ssm_states(int dtype, const SsmArgs &a, Segments seg, SegBuf buf, RowBuf rows, float *keep,
                             hipStream_t stream) {
    ScanArgs k = scan_args(a, seg, rows);
    k.buf = buf;
    k.keep = keep;
    return dtype == 1 ? run_scan_n<Bf16, kKeep>(k, stream) : run_scan_n<F32, kKeep>(k, stream);
}

hipError_t launch_ssm_step(int dtype, const SsmArgs &a, hipStream_t stream) {
    return dtype == 1 ? run_step<Bf16>(a, stream) : run_step<F32>(a, stream);
}

}  // namespace qd
