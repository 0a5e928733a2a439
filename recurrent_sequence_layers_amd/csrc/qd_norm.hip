// Group norm for gfx950, channels last, with an optional SiLU and an optional gate:
//
//   xhat = (x - mean) rstd  over a sample's group (L positions x E = C / G channels)
//   v = xhat w + bias,  f = v or silu(v),  y = f silu(gate)  (the gate's factor only if given)
//
// and, with gv = dy silu(gate) f'(v), a = sum(gv w), b = sum(gv w xhat) over the group's
// M = L E elements,
//
//   dx = rstd (gv w - (a + xhat b) / M),  dw = sum gv xhat,  dbias = sum gv,
//   dgate = dy f silu'(gate).
//
// Bound by HBM: every tensor is read once and written once where a group fits a workgroup's
// registers (L = 1: the norm of a token's heads).  Then the variance is that of the centred
// values held in registers.  Longer groups take two passes over x: partial statistics per
// channel and run of rows, their combination, and the elementwise pass, whose second read is
// served by the last-level cache while the tensors fit it.  Group sizes that 16 bytes do not divide go
// one element a lane, with one load of a row in flight: 32768 x 16 groups, bf16, SiLU, of 127 channels
// 145 us forward and 176 backward, of 128 channels 66 and 97.
#include "qd_internal.h"
#include "qd_mixer.h"

namespace qd {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- L = 1: a group in registers
// A unit is one (row, group), E contiguous elements at unit * E.  LG lanes share it, each
// with K vectors of V elements, interleaved.  LG is a power of two up to a wave, or the
// whole workgroup (one unit a workgroup, sums joined through LDS).
struct RowArgs {
    NormArgs a;
    int E, LG;
    long long units;
    float *part;                     // backward: [R][2][C], (sum gv, sum gv xhat)
    int R;
};

__device__ __forceinline__ float unit_sum(float x, int LG, float *red) {
    if (LG <= kWave) return group_sum(x, LG);
    x = group_sum(x, kWave);
    __syncthreads();
    if (lane_id() == 0) red[wave_id()] = x;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// A lane keeps its group and columns over all its units (the grid's step is a multiple of G
// units), so weight and bias are read once.
template <class P, int V, int K>
__global__ __launch_bounds__(kThreads) void norm_rows_kernel(const RowArgs k) {
    using R = typename P::R;
    __shared__ float red[kThreads / kWave];
    const NormArgs &a = k.a;
    const int sub = threadIdx.x & (k.LG - 1);
    const long long slot = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / k.LG;
    const long long step = static_cast<long long>(gridDim.x) * kThreads / k.LG;
    const int c0 = static_cast<int>(slot % a.G) * k.E;
    const bool gated = a.gate != nullptr;
    float w[K][V], bias[K][V];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = (sub + j * k.LG) * V + i;
            w[j][i] = a.w && e < k.E ? a.w[c0 + e] : 1.f;
            bias[j][i] = a.bias && e < k.E ? a.bias[c0 + e] : 0.f;
        }
    // every lane of a workgroup makes the same number of steps: the sums' barriers are met by all
    for (long long first = static_cast<long long>(blockIdx.x) * kThreads / k.LG; first < k.units; first += step) {
        const long long unit = first + threadIdx.x / k.LG;
        const bool live = unit < k.units;
        const long long un = live ? unit : k.units - 1;
        const size_t base = static_cast<size_t>(un) * k.E;
        const R *x = static_cast<const R *>(a.x) + base;
        const R *gate = gated ? static_cast<const R *>(a.gate) + base : x;
        float v[K][V], z[K][V];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e0 = (sub + j * k.LG) * V, e = e0 < k.E ? e0 : 0;
            load_vec<P, V>(x + e, v[j]);
            if (gated) load_vec<P, V>(gate + e, z[j]);
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool in = (sub + j * k.LG) * V < k.E;
#pragma unroll
            for (int i = 0; i < V; ++i) s += in ? v[j][i] : 0.f;
        }
        // divided, not multiplied by a rounded reciprocal: a constant group's mean is its value
        const float mean = unit_sum(s, k.LG, red) / static_cast<float>(k.E);
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool in = (sub + j * k.LG) * V < k.E;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[j][i] -= mean;
                q = in ? fmaf(v[j][i], v[j][i], q) : q;
            }
        }
        const float rstd = 1.f / sqrtf(unit_sum(q, k.LG, red) / static_cast<float>(k.E) + a.eps);
        if (!live) continue;
        if (a.stats && sub == 0) {
            a.stats[2 * un] = mean;
            a.stats[2 * un + 1] = rstd;
        }
        R *y = static_cast<R *>(a.y) + base;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e = (sub + j * k.LG) * V;
            if (e >= k.E) continue;
            float out[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f = fmaf(v[j][i] * rstd, w[j][i], bias[j][i]);
                if (a.silu) f = siluf(f);
                out[i] = gated ? f * siluf(z[j][i]) : f;
            }
            store_vec<P, V>(y + e, out);
        }
    }
}

// The gradient of the value v, and the gate's, at one element.
struct ElemGrad {
    float gv, dgate;
};
__device__ __forceinline__ ElemGrad elem_grad(float v, float dy, float z, bool has_gate, bool silu) {
    ElemGrad r;
    float f = v, df = 1.f;
    if (silu) {
        const float s = sigmoidf(v);
        f = v * s;
        df = s * fmaf(v, 1.f - s, 1.f);
    }
    r.gv = dy * df;
    r.dgate = 0.f;
    if (has_gate) {
        const float s = sigmoidf(z);
        r.dgate = dy * f * (s * fmaf(z, 1.f - s, 1.f));
        r.gv *= z * s;
    }
    return r;
}

// Persistent: a lane keeps its group and columns over all its units (the grid's step is a
// multiple of G units), so dw and dbias gather in its registers; each group slot of the grid
// writes one row of partial sums.
template <class P, int V, int K>
__global__ __launch_bounds__(kThreads) void norm_rows_bwd_kernel(const RowArgs k) {
    using R = typename P::R;
    __shared__ float red[kThreads / kWave];
    const NormArgs &a = k.a;
    const int sub = threadIdx.x & (k.LG - 1);
    const long long slot = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / k.LG;
    const long long step = static_cast<long long>(gridDim.x) * kThreads / k.LG;
    const int g = static_cast<int>(slot % a.G), c0 = g * k.E;
    const bool sums = a.dw || a.dbias;
    const float inv = 1.f / static_cast<float>(k.E);
    float w[K][V], bias[K][V], sw[K][V] = {}, sb[K][V] = {};
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = (sub + j * k.LG) * V + i;
            w[j][i] = a.w && e < k.E ? a.w[c0 + e] : 1.f;
            bias[j][i] = a.bias && e < k.E ? a.bias[c0 + e] : 0.f;
        }
    // every lane of a workgroup makes the same number of steps: the sums' barriers are met by all
    for (long long first = static_cast<long long>(blockIdx.x) * kThreads / k.LG; first < k.units; first += step) {
        const long long unit = first + threadIdx.x / k.LG;
        const bool live = unit < k.units;
        const long long un = live ? unit : k.units - 1;
        const size_t base = static_cast<size_t>(un) * k.E;
        const float mean = a.stats[2 * un], rstd = a.stats[2 * un + 1];
        float x[K][V], dy[K][V], z[K][V];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e0 = (sub + j * k.LG) * V, e = e0 < k.E ? e0 : 0;
            load_vec<P, V>(static_cast<const R *>(a.x) + base + e, x[j]);
            load_vec<P, V>(static_cast<const R *>(a.dy) + base + e, dy[j]);
            if (a.gate) load_vec<P, V>(static_cast<const R *>(a.gate) + base + e, z[j]);
        }
        float sa = 0.f, sx = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e = (sub + j * k.LG) * V;
            const bool in = live && e < k.E;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[j][i] = (x[j][i] - mean) * rstd;
                const ElemGrad r = elem_grad(fmaf(x[j][i], w[j][i], bias[j][i]), dy[j][i], z[j][i], a.gate != nullptr, a.silu);
                z[j][i] = r.dgate;
                const float gw = r.gv * w[j][i];
                dy[j][i] = gw;
                if (in) {
                    sa += gw;
                    sx = fmaf(gw, x[j][i], sx);
                    sb[j][i] += r.gv;
                    sw[j][i] = fmaf(r.gv, x[j][i], sw[j][i]);
                }
            }
            if (a.gate && in) store_vec<P, V>(static_cast<R *>(a.dgate) + base + e, z[j]);
        }
        sa = unit_sum(sa, k.LG, red) * inv;
        sx = unit_sum(sx, k.LG, red) * inv;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e = (sub + j * k.LG) * V;
            if (!live || e >= k.E) continue;
            float out[V];
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = rstd * (dy[j][i] - fmaf(x[j][i], sx, sa));
            store_vec<P, V>(static_cast<R *>(a.dx) + base + e, out);
        }
    }
    if (!sums) return;
    float *part = k.part + static_cast<size_t>(slot / a.G) * 2 * a.C + c0;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = (sub + j * k.LG) * V + i;
            if (e < k.E) {
                part[e] = sb[j][i];
                part[a.C + e] = sw[j][i];
            }
        }
}

// ---------------------------------------------------------------- groups over many rows
// Samples are cut into S runs of RL rows.  A thread owns a vector of channels over a run.
struct LongArgs {
    NormArgs a;
    int E, S, RL;
    float *part;                     // [N][S][2][C]: (mean, centred square sum), or (sum gv, sum gv xhat)
    float *group;                    // [N][G][2]: (mean, rstd), or (sum gv w, sum gv w xhat) / M
};

// The second pass reads again what the first one read; from this size of a tensor on its
// output, kept in the caches, would push out the rest of that.  With a reader of the output
// behind the call: 117 MiB, forward 149 -> 138 us and backward 184 -> 171; 29 MiB, 36 -> 37 and
// 52 -> 54 us.
constexpr size_t kAroundBytes = 64u << 20;

struct Where {
    int n, s, c, r0, r1;
    bool live;
};
template <int V>
__device__ __forceinline__ Where where(const LongArgs &k) {
    const int nvec = k.a.C / V;
    const long long idx = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    Where w;
    w.live = idx < static_cast<long long>(k.a.N) * k.S * nvec;
    w.c = static_cast<int>(idx % nvec) * V;
    const int ns = static_cast<int>(idx / nvec);
    w.n = ns / k.S;
    w.s = ns % k.S;
    w.r0 = w.s * k.RL;
    w.r1 = min(w.r0 + k.RL, k.a.L);
    return w;
}

// Mean and centred square sum of each channel's run.  Sums are taken of x - x0 with x0 the
// run's first value: that value is part of the run, so the square sum is at least
// (x0 - mean)^2 and what the shift can cancel is bounded by the run's length.
template <class P, int V>
__global__ __launch_bounds__(kThreads) void norm_partial_kernel(const LongArgs k) {
    using R = typename P::R;
    const Where at = where<V>(k);
    if (!at.live) return;
    const size_t C = k.a.C;
    const R *x = static_cast<const R *>(k.a.x) + static_cast<size_t>(at.n) * k.a.L * C + at.c;
    float x0[V], s[V] = {}, q[V] = {};
    load_vec<P, V>(x + at.r0 * C, x0);
    for (int r = at.r0 + 1; r < at.r1; r += 4) {
        float v[4][V];
#pragma unroll
        for (int j = 0; j < 4; ++j) load_vec<P, V>(x + static_cast<size_t>(min(r + j, at.r1 - 1)) * C, v[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = r + j < at.r1 ? v[j][i] - x0[i] : 0.f;
                s[i] += d;
                q[i] = fmaf(d, d, q[i]);
            }
    }
    const float inv = 1.f / static_cast<float>(at.r1 - at.r0);
    float *part = k.part + (static_cast<size_t>(at.n) * k.S + at.s) * 2 * C + at.c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float m = s[i] * inv;
        part[i] = x0[i] + m;
        part[C + i] = fmaxf(q[i] - s[i] * m, 0.f);
    }
}

// A group's runs: one workgroup, wide because its loads are what it waits for.  The grid is groups x
// samples; past these sizes a workgroup takes several, so that every launch fits.  32768 samples of
// 2 rows, 16 groups of 32 channels, fp32: 1.61 ms forward with 2048 samples a grid, 1.66 with 8192,
// 1.82 with all of them; gradients 1.54, 1.62 and 1.74.
constexpr int kGroupThreads = 1024, kGroupWaves = kGroupThreads / kWave;
constexpr int kGridGroups = 1 << 20, kGridSamples = 1 << 11;
__device__ __forceinline__ float block_sum(float x, float *red) {
    x = group_sum(x, kWave);
    __syncthreads();
    if (lane_id() == 0) red[wave_id()] = x;
    __syncthreads();
    return group_sum(red[lane_id() & (kGroupWaves - 1)], kGroupWaves);
}

// Statistics of a group from its channels' runs: the mean of the means, then the square sums
// moved to it.
__global__ __launch_bounds__(kGroupThreads) void norm_group_kernel(const LongArgs k) {
    __shared__ float red[kGroupWaves];
    const uint32_t items = static_cast<uint32_t>(k.S) * k.E, E = k.E;
    const float M = static_cast<float>(k.a.L) * static_cast<float>(k.E);
    auto one = [&](int n, int g) {
        const float *part = k.part + static_cast<size_t>(n) * k.S * 2 * k.a.C + g * k.E;
        float s = 0.f;
        for (uint32_t i = threadIdx.x; i < items; i += kGroupThreads) {
            const int run = i / E, e = i - run * E;
            s += part[static_cast<size_t>(run) * 2 * k.a.C + e] * static_cast<float>(min(k.RL, k.a.L - run * k.RL));
        }
        const float mean = block_sum(s, red) / M;
        float q = 0.f;
        for (uint32_t i = threadIdx.x; i < items; i += kGroupThreads) {
            const int run = i / E, e = i - run * E;
            const float *p = part + static_cast<size_t>(run) * 2 * k.a.C + e;
            const float d = p[0] - mean;
            q += fmaf(d * d, static_cast<float>(min(k.RL, k.a.L - run * k.RL)), p[k.a.C]);
        }
        q = block_sum(q, red);
        if (threadIdx.x == 0) {
            const float rstd = 1.f / sqrtf(q / M + k.a.eps);
            float *to = k.group + 2 * (static_cast<size_t>(n) * k.a.G + g);
            to[0] = mean;
            to[1] = rstd;
        }
    };
    for (int n = blockIdx.y; n < k.a.N; n += gridDim.y)
        for (int g = blockIdx.x; g < k.a.G; g += gridDim.x) one(n, g);
}

// A group's two sums for dx, over its channels' runs, divided by M.
__global__ __launch_bounds__(kGroupThreads) void norm_group_bwd_kernel(const LongArgs k) {
    __shared__ float red[kGroupWaves];
    const uint32_t items = static_cast<uint32_t>(k.S) * k.E, E = k.E;
    const float M = static_cast<float>(k.a.L) * static_cast<float>(k.E);
    auto one = [&](int n, int g) {
        const float *part = k.part + static_cast<size_t>(n) * k.S * 2 * k.a.C + g * k.E;
        float sa = 0.f, sx = 0.f;
        for (uint32_t i = threadIdx.x; i < items; i += kGroupThreads) {
            const int run = i / E, e = i - run * E;
            const float *p = part + static_cast<size_t>(run) * 2 * k.a.C + e;
            const float w = k.a.w ? k.a.w[g * k.E + e] : 1.f;
            sa = fmaf(w, p[0], sa);
            sx = fmaf(w, p[k.a.C], sx);
        }
        sa = block_sum(sa, red);
        sx = block_sum(sx, red);
        if (threadIdx.x == 0) {
            float *to = k.group + 2 * (static_cast<size_t>(n) * k.a.G + g);
            to[0] = sa / M;
            to[1] = sx / M;
        }
    };
    for (int n = blockIdx.y; n < k.a.N; n += gridDim.y)
        for (int g = blockIdx.x; g < k.a.G; g += gridDim.x) one(n, g);
}

// A lane's channels with what belongs to each: weight, bias and its group's two numbers.
template <int V>
struct Cols {
    float w[V], bias[V], m[V], r[V];
};
template <int V>
__device__ __forceinline__ Cols<V> columns(const LongArgs &k, const Where &at, const float *stats) {
    Cols<V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = at.c + i;
        const float *st = stats + 2 * (static_cast<size_t>(at.n) * k.a.G + c / k.E);
        o.w[i] = k.a.w ? k.a.w[c] : 1.f;
        o.bias[i] = k.a.bias ? k.a.bias[c] : 0.f;
        o.m[i] = st[0];
        o.r[i] = st[1];
    }
    return o;
}

template <class P, int V, bool AROUND>
__global__ __launch_bounds__(kThreads) void norm_apply_kernel(const LongArgs k) {
    using R = typename P::R;
    const Where at = where<V>(k);
    if (!at.live) return;
    const size_t C = k.a.C, base = static_cast<size_t>(at.n) * k.a.L * C + at.c;
    const R *x = static_cast<const R *>(k.a.x) + base, *gate = k.a.gate ? static_cast<const R *>(k.a.gate) + base : nullptr;
    R *y = static_cast<R *>(k.a.y) + base;
    const Cols<V> o = columns<V>(k, at, k.group);
    for (int r = at.r0; r < at.r1; r += 2) {
        float v[2][V], z[2][V];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t row = static_cast<size_t>(min(r + j, at.r1 - 1)) * C;
            load_vec<P, V>(x + row, v[j]);
            if (gate) load_vec<P, V>(gate + row, z[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f = fmaf((v[j][i] - o.m[i]) * o.r[i], o.w[i], o.bias[i]);
                if (k.a.silu) f = siluf(f);
                v[j][i] = gate ? f * siluf(z[j][i]) : f;
            }
            if (r + j < at.r1) store_vec<P, V, AROUND>(y + static_cast<size_t>(r + j) * C, v[j]);
        }
    }
}

// dgate, and each channel's run of sum gv and sum gv xhat.
template <class P, int V>
__global__ __launch_bounds__(kThreads) void norm_partial_bwd_kernel(const LongArgs k) {
    using R = typename P::R;
    const Where at = where<V>(k);
    if (!at.live) return;
    const size_t C = k.a.C, base = static_cast<size_t>(at.n) * k.a.L * C + at.c;
    const Cols<V> o = columns<V>(k, at, k.a.stats);
    float sb[V] = {}, sw[V] = {};
    for (int r = at.r0; r < at.r1; r += 2) {
        float x[2][V], dy[2][V], z[2][V];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t row = base + static_cast<size_t>(min(r + j, at.r1 - 1)) * C;
            load_vec<P, V>(static_cast<const R *>(k.a.x) + row, x[j]);
            load_vec<P, V>(static_cast<const R *>(k.a.dy) + row, dy[j]);
            if (k.a.gate) load_vec<P, V>(static_cast<const R *>(k.a.gate) + row, z[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (r + j >= at.r1) break;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (x[j][i] - o.m[i]) * o.r[i];
                const ElemGrad e = elem_grad(fmaf(xh, o.w[i], o.bias[i]), dy[j][i], z[j][i], k.a.gate != nullptr, k.a.silu);
                z[j][i] = e.dgate;
                sb[i] += e.gv;
                sw[i] = fmaf(e.gv, xh, sw[i]);
            }
            if (k.a.gate) store_vec<P, V>(static_cast<R *>(k.a.dgate) + base + static_cast<size_t>(r + j) * C, z[j]);
        }
    }
    float *part = k.part + (static_cast<size_t>(at.n) * k.S + at.s) * 2 * C + at.c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        part[i] = sb[i];
        part[C + i] = sw[i];
    }
}

template <class P, int V, bool AROUND>
__global__ __launch_bounds__(kThreads) void norm_apply_bwd_kernel(const LongArgs k) {
    using R = typename P::R;
    const Where at = where<V>(k);
    if (!at.live) return;
    const size_t C = k.a.C, base = static_cast<size_t>(at.n) * k.a.L * C + at.c;
    const Cols<V> o = columns<V>(k, at, k.a.stats), t = columns<V>(k, at, k.group);
    for (int r = at.r0; r < at.r1; r += 2) {
        float x[2][V], dy[2][V], z[2][V];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t row = base + static_cast<size_t>(min(r + j, at.r1 - 1)) * C;
            load_vec<P, V>(static_cast<const R *>(k.a.x) + row, x[j]);
            load_vec<P, V>(static_cast<const R *>(k.a.dy) + row, dy[j]);
            if (k.a.gate) load_vec<P, V>(static_cast<const R *>(k.a.gate) + row, z[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (x[j][i] - o.m[i]) * o.r[i];
                const ElemGrad e = elem_grad(fmaf(xh, o.w[i], o.bias[i]), dy[j][i], z[j][i], k.a.gate != nullptr, k.a.silu);
                x[j][i] = o.r[i] * (fmaf(e.gv, o.w[i], -t.m[i]) - xh * t.r[i]);
            }
            if (r + j < at.r1) store_vec<P, V, AROUND>(static_cast<R *>(k.a.dx) + base + static_cast<size_t>(r + j) * C, x[j]);
        }
    }
}

struct NormStore {
    float *dw, *dbias;
    int C;
    __device__ __forceinline__ void operator()(long long c, float v) const {
        if (c < C) {
            if (dbias) dbias[c] = v;
        } else if (dw) {
            dw[c - C] = v;
        }
    }
};

__global__ __launch_bounds__(kThreads) void norm_zero_kernel(float *dw, float *dbias, int C) {
    const size_t c = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= static_cast<size_t>(C)) return;
    if (dw) dw[c] = 0.f;
    if (dbias) dbias[c] = 0.f;
}

// ---------------------------------------------------------------- plans
struct RowPlan {
    bool use;
    int V, LG, K, grid, R;           // grid: workgroups of the backward; R: its rows of partial sums
};
// Forward: eight workgroups a compute unit, 90 us at 32768 rows of 16 x 128 bf16, gated, against
// 95 with four and 94 with sixteen.
constexpr int kGridFwd = 2048, kGridBwd = 1024;
// Workgroups of a persistent row kernel: at most `most`, and their slots a multiple of G, so
// that a slot's units are all of one group.
int row_grid(int N, int G, int LG, int most) {
    const int upb = kThreads / LG;
    int step = G;
    for (int d = upb; d > 1 && step % 2 == 0; d /= 2) step /= 2;
    const long long need = (static_cast<long long>(N) * G + upb - 1) / upb;
    const long long grid = need < most ? need : most;
    return static_cast<int>((grid + step - 1) / step * step);
}
int max_vec(int dtype) { return dtype == 1 ? 8 : 4; }
RowPlan row_plan(int dtype, int N, int L, int C, int G) {
    RowPlan p{};
    const int E = C / G;
    p.V = E % max_vec(dtype) == 0 ? max_vec(dtype) : 1;
    const int nv = E / p.V;
    // vectors a lane holds: the backward keeps three tensors and four sums of them in registers
    const int wave_k = p.V == 1 ? 8 : 2, block_k = p.V == 1 ? 8 : 4;
    p.use = L == 1 && nv <= kThreads * block_k;
    if (!p.use) return p;
    p.LG = 1;
    while (p.LG < kWave && p.LG < nv) p.LG *= 2;
    if (nv > p.LG * wave_k) p.LG = kThreads;
    p.K = 1;
    while (p.LG * p.K < nv) p.K *= 2;
    p.grid = row_grid(N, G, p.LG, kGridBwd);
    p.R = static_cast<int>(static_cast<long long>(p.grid) * (kThreads / p.LG) / G);
    return p;
}
struct LongPlan {
    int V, S, RL;
};
LongPlan long_plan(int dtype, int N, int L, int C) {
    LongPlan p;
    p.V = C % max_vec(dtype) == 0 ? max_vec(dtype) : 1;
    p.RL = 64;
    while (p.RL > 8 && static_cast<long long>(N) * ((L + p.RL - 1) / p.RL) * (C / p.V) < 131072) p.RL /= 2;
    p.S = (L + p.RL - 1) / p.RL;
    return p;
}

template <class P, int V>
void rows_k(const RowArgs &k, int K, int grid, bool back, hipStream_t stream) {
    const dim3 g(grid), b(kThreads);
    if (back) {
        if (K == 1) hipLaunchKernelGGL((norm_rows_bwd_kernel<P, V, 1>), g, b, 0, stream, k);
        else if (K == 2) hipLaunchKernelGGL((norm_rows_bwd_kernel<P, V, 2>), g, b, 0, stream, k);
        else if (K == 4) hipLaunchKernelGGL((norm_rows_bwd_kernel<P, V, 4>), g, b, 0, stream, k);
        else if constexpr (V == 1) hipLaunchKernelGGL((norm_rows_bwd_kernel<P, 1, 8>), g, b, 0, stream, k);
    } else {
        if (K == 1) hipLaunchKernelGGL((norm_rows_kernel<P, V, 1>), g, b, 0, stream, k);
        else if (K == 2) hipLaunchKernelGGL((norm_rows_kernel<P, V, 2>), g, b, 0, stream, k);
        else if (K == 4) hipLaunchKernelGGL((norm_rows_kernel<P, V, 4>), g, b, 0, stream, k);
        else if constexpr (V == 1) hipLaunchKernelGGL((norm_rows_kernel<P, 1, 8>), g, b, 0, stream, k);
    }
}
template <class P>
void rows(const RowArgs &k, const RowPlan &p, int grid, bool back, hipStream_t stream) {
    if (p.V == 1) rows_k<P, 1>(k, p.K, grid, back, stream);
    else rows_k<P, 16 / P::kBytes>(k, p.K, grid, back, stream);
}

dim3 group_grid(const LongArgs &k) {
    return dim3(static_cast<unsigned>(k.a.G < kGridGroups ? k.a.G : kGridGroups),
                static_cast<unsigned>(k.a.N < kGridSamples ? k.a.N : kGridSamples));
}
template <class P, int V>
void long_fwd(const LongArgs &k, hipStream_t stream) {
    const bool around = static_cast<size_t>(k.a.N) * k.a.L * k.a.C * P::kBytes >= kAroundBytes;
    const long long n = static_cast<long long>(k.a.N) * k.S * (k.a.C / V);
    const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads)), blk(kThreads);
    hipLaunchKernelGGL((norm_partial_kernel<P, V>), grid, blk, 0, stream, k);
    hipLaunchKernelGGL(norm_group_kernel, group_grid(k), dim3(kGroupThreads), 0, stream, k);
    if (around) hipLaunchKernelGGL((norm_apply_kernel<P, V, true>), grid, blk, 0, stream, k);
    else hipLaunchKernelGGL((norm_apply_kernel<P, V, false>), grid, blk, 0, stream, k);
}
template <class P, int V>
void long_bwd(const LongArgs &k, hipStream_t stream) {
    const bool around = static_cast<size_t>(k.a.N) * k.a.L * k.a.C * P::kBytes >= kAroundBytes;
    const long long n = static_cast<long long>(k.a.N) * k.S * (k.a.C / V);
    const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads)), blk(kThreads);
    hipLaunchKernelGGL((norm_partial_bwd_kernel<P, V>), grid, blk, 0, stream, k);
    hipLaunchKernelGGL(norm_group_bwd_kernel, group_grid(k), dim3(kGroupThreads), 0, stream, k);
    if (around) hipLaunchKernelGGL((norm_apply_bwd_kernel<P, V, true>), grid, blk, 0, stream, k);
    else hipLaunchKernelGGL((norm_apply_bwd_kernel<P, V, false>), grid, blk, 0, stream, k);
}

}  // namespace

bool norm_fits(int dtype, int N, int L, int C, int G) {
    const RowPlan r = row_plan(dtype, N, L, C, G);
    const long long lim = (1LL << 32) - 1024;
    if (static_cast<long long>(N) * L >= (1LL << 31) || C >= (1 << 26)) return false;
    if (r.use) return static_cast<long long>(N) * G * r.LG < lim && static_cast<long long>(row_grid(N, G, r.LG, kGridFwd)) * kThreads < lim;
    const LongPlan p = long_plan(dtype, N, L, C);
    return static_cast<long long>(N) * p.S * (C / p.V) < lim && static_cast<long long>(p.S) * (C / G) < lim;
}

size_t norm_fwd_workspace(int dtype, int N, int L, int C, int G) {
    if (static_cast<long long>(N) * L * C == 0 || row_plan(dtype, N, L, C, G).use) return 0;
    const LongPlan p = long_plan(dtype, N, L, C);
    return (static_cast<size_t>(N) * p.S * 2 * C + static_cast<size_t>(N) * G * 2) * sizeof(float);
}

size_t norm_bwd_workspace(int dtype, int N, int L, int C, int G) {
    if (static_cast<long long>(N) * L * C == 0) return 0;
    const RowPlan r = row_plan(dtype, N, L, C, G);
    if (r.use) return static_cast<size_t>(r.R) * 2 * C * sizeof(float);
    const LongPlan p = long_plan(dtype, N, L, C);
    return (static_cast<size_t>(N) * p.S * 2 * C + static_cast<size_t>(N) * G * 2) * sizeof(float);
}

hipError_t launch_norm_fwd(int dtype, const NormArgs &a, void *ws, hipStream_t stream) {
    const RowPlan r = row_plan(dtype, a.N, a.L, a.C, a.G);
    if (r.use) {
        RowArgs k{a, a.C / a.G, r.LG, static_cast<long long>(a.N) * a.G, nullptr, 0};
        const int grid = row_grid(a.N, a.G, r.LG, kGridFwd);
        if (dtype == 1) rows<Bf16>(k, r, grid, false, stream);
        else rows<F32>(k, r, grid, false, stream);
        return hipGetLastError();
    }
    const LongPlan p = long_plan(dtype, a.N, a.L, a.C);
    LongArgs k{a, a.C / a.G, p.S, p.RL, static_cast<float *>(ws), nullptr};
    k.group = a.stats ? a.stats : k.part + static_cast<size_t>(a.N) * p.S * 2 * a.C;
    if (dtype == 1) p.V == 8 ? long_fwd<Bf16, 8>(k, stream) : long_fwd<Bf16, 1>(k, stream);
    else p.V == 4 ? long_fwd<F32, 4>(k, stream) : long_fwd<F32, 1>(k, stream);
    return hipGetLastError();
}

hipError_t launch_norm_zero(float *dw, float *dbias, int C, hipStream_t stream) {
    hipLaunchKernelGGL(norm_zero_kernel, dim3(static_cast<unsigned>((C - 1) / kThreads + 1)), dim3(kThreads), 0, stream, dw, dbias, C);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(int dtype, const NormArgs &a, void *ws, hipStream_t stream) {
    const RowPlan r = row_plan(dtype, a.N, a.L, a.C, a.G);
    float *part = static_cast<float *>(ws);
    int R;
    if (r.use) {
        RowArgs k{a, a.C / a.G, r.LG, static_cast<long long>(a.N) * a.G, part, r.R};
        if (dtype == 1) rows<Bf16>(k, r, r.grid, true, stream);
        else rows<F32>(k, r, r.grid, true, stream);
        R = r.R;
    } else {
        const LongPlan p = long_plan(dtype, a.N, a.L, a.C);
        LongArgs k{a, a.C / a.G, p.S, p.RL, part, part + static_cast<size_t>(a.N) * p.S * 2 * a.C};
        if (dtype == 1) p.V == 8 ? long_bwd<Bf16, 8>(k, stream) : long_bwd<Bf16, 1>(k, stream);
        else p.V == 4 ? long_bwd<F32, 4>(k, stream) : long_bwd<F32, 1>(k, stream);
        R = a.N * p.S;
    }
    if (a.dw || a.dbias) column_sum(part, R, 2LL * a.C, NormStore{a.dw, a.dbias, a.C}, stream);
    return hipGetLastError();
}

}  // namespace qd
