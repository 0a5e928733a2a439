// RMS norms after and before a block, with the block's gate, its scale and the residual sum, for
// gfx950.  A row of C channels:
//
//   f = y r1 post, r1 = 1 / sqrt(mean y^2 + eps)       (y itself without post)
//   h = x + scale act(gate) f                          stored: the residual stream
//   n = h r2 pre,  r2 = 1 / sqrt(mean h^2 + eps)       of h as it is stored
//
// and its gradients, with yhat = y r1, hhat = h r2 and t the gradient that reaches h:
//
//   t = dh + r2 (pre dn - hhat mean(pre dn hhat)),     dx = t,  dpre = sum dn hhat
//   df = t scale act(gate),  dscale = sum t act(gate) f,  dgate = t scale f act'(gate)
//   dy = r1 (post df - yhat mean(post df yhat)),       dpost = sum df yhat
//
// Bound by HBM: every tensor is read once and written once.  A row sits in the registers of LG
// lanes, one or two 16-byte vectors each; the grid is persistent, so a lane keeps its columns'
// weights and gathers its columns' sums over all its rows; forwards the next row's vectors are on
// their way while this one is reduced.  A channel count that the vector does not divide ends in a vector
// that starts earlier and overlaps the one before it: what overlaps is the same in both, and
// counts once.  Rows that would not fit a workgroup's registers take the looping form, which reads
// a row again for each of its passes.  32768 rows of 2048 in bf16 with post norm, gate, scale, residual
// and pre norm: 133 us forward (671 MB, 5.05 TB/s), 220 backward (1074 MB, 4.9 TB/s, 7 us of it the
// sums over the rows' partial sums), as fast as a copy; 64 rows are a launch, 4.4 us.  Backwards rows
// above 2048 (fp32: 4096) take more registers than 1024 threads leave a lane, 8 (29) are spilled: 16384
// x 4096 bf16 284 us where its bytes take 218.  The looping form is far from its bytes: 4096 x 12288
// bf16 278 forward (102) and 1063 backward (163), where its sums go through memory for every row.
#include "qd_block_norm.h"
#include "qd_internal.h"
#include "qd_mixer.h"

namespace qd {
namespace {

constexpr int kMaxLanes = 1024;

// V elements from an address aligned to an element only: the hardware takes 16-byte accesses at
// any address.
template <class P, int V>
struct Vec {
    static constexpr int W = V * P::kBytes >= 4 ? V * P::kBytes / 4 : 1;
    uint32_t w[W];
    __device__ __forceinline__ void load(const typename P::R *p) {
        if constexpr (V == 1) {
            if constexpr (P::kBytes == 2) w[0] = *p;
            else w[0] = __float_as_uint(*p);
        } else {
            __builtin_memcpy(w, p, V * P::kBytes);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (P::kBytes == 4) return __uint_as_float(w[i]);
        else if constexpr (V == 1) return __uint_as_float(w[0] << 16);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void set(int i, float x) {
        if constexpr (P::kBytes == 4) {
            w[i] = __float_as_uint(x);
        } else {
            const uint32_t b = P::from_f32(x);
            if constexpr (V == 1) w[0] = b;
            else w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (b << 16) : b;
        }
    }
    __device__ __forceinline__ void store(typename P::R *p) const {
        if constexpr (V == 1) {
            if constexpr (P::kBytes == 2) *p = static_cast<uint16_t>(w[0]);
            else *p = __uint_as_float(w[0]);
        } else {
            __builtin_memcpy(p, w, V * P::kBytes);
        }
    }
};

// Sum over a row's LG lanes; all of a workgroup's waves call it equally often.  Two slots in turn:
// a slot is written again only after a barrier that its readers have passed.
struct RowSum {
    float *red;                      // [2][16]
    int LG, slot;
    __device__ __forceinline__ float operator()(float x) {
        if (LG <= kWave) return group_sum(x, LG);
        x = group_sum(x, kWave);
        float *r = red + 16 * slot;
        slot ^= 1;
        if (lane_id() == 0) r[wave_id()] = x;
        __syncthreads();
        const int per = LG / kWave, first = wave_id() / per * per;
        float s = 0.f;
        for (int i = 0; i < per; ++i) s += r[first + i];
        return s;
    }
};

struct Gate {
    float u, du;                     // the gate's factor and its derivative
};
__device__ __forceinline__ Gate gate_of(float z, int act) {
    if (act == 0) return Gate{z, 1.f};
    // 1 - p as e^-z p, which keeps its digits where p is near one
    const float e = __builtin_amdgcn_exp2f(-z * kLog2e), p = sigmoidf(z), q = p * (fminf(e, 3.0e38f) * p);
    return act == 1 ? Gate{p, q} : Gate{z * p, fmaf(z, q, p)};
}

// A lane's place: its row of the workgroup's, and its vectors' columns.
template <int V, int K>
struct Place {
    int sub, row, rpb;               // lane of the row, row of the block, rows a block
    int col[K], skip[K];             // first column, and how many of its elements the vector before has; V: nothing of its own
    __device__ __forceinline__ Place(const BlockNormArgs &a) {
        sub = threadIdx.x & (a.LG - 1);
        row = threadIdx.x / a.LG;
        rpb = blockDim.x / a.LG;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (sub + k * a.LG) * V, last = a.C - V;
            col[k] = e < last ? e : last;
            skip[k] = e >= a.C ? V : e - col[k];
        }
    }
};

template <class P, int V, int K>
__device__ __forceinline__ void columns(const float *w, const Place<V, K> &at, float (&out)[K][V]) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) out[k][i] = w ? w[at.col[k] + i] : 1.f;
}

template <class P, int V, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void block_norm_kernel(const BlockNormArgs a) {
    using R = typename P::R;
    __shared__ float red[32];
    RowSum row_sum{red, a.LG, 0};
    const Place<V, K> at(a);
    float post[K][V], scale[K][V], pre[K][V];
    columns<P, V, K>(a.post, at, post);
    columns<P, V, K>(a.scale, at, scale);
    columns<P, V, K>(a.pre, at, pre);
    Vec<P, V> y[K], x[K], z[K];
    auto load = [&](long long r) {
        const size_t base = static_cast<size_t>(r < a.N ? r : a.N - 1) * a.C;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            y[k].load(static_cast<const R *>(a.y) + base + at.col[k]);
            if (a.x) x[k].load(static_cast<const R *>(a.x) + base + at.col[k]);
            if (a.gate) z[k].load(static_cast<const R *>(a.gate) + base + at.col[k]);
        }
    };
    const float C = static_cast<float>(a.C);
    const long long step = static_cast<long long>(gridDim.x) * at.rpb;
    long long first = static_cast<long long>(blockIdx.x) * at.rpb;
    load(first + at.row);
    for (; first < a.N; first += step) {
        const long long r = first + at.row;
        const bool live = r < a.N;
        float f[K][V], u[K][V], q = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[k][i] = y[k].get(i);
                u[k][i] = scale[k][i];
                if (a.gate) u[k][i] *= gate_of(z[k].get(i), a.act).u;
                q = i >= at.skip[k] ? fmaf(f[k][i], f[k][i], q) : q;
            }
        Vec<P, V> old[K];
#pragma unroll
        for (int k = 0; k < K; ++k) old[k] = x[k];
        if (first + step < a.N) load(r + step);
        float r1 = 1.f;
        if (a.post) r1 = 1.f / sqrtf(row_sum(q) / C + a.eps);
        const size_t base = static_cast<size_t>(r) * a.C;
        float s = 0.f;
        Vec<P, V> h[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = f[k][i] * r1 * post[k][i] * u[k][i];
                h[k].set(i, a.x ? old[k].get(i) + v : v);
                const float w = h[k].get(i);         // as stored
                s = i >= at.skip[k] ? fmaf(w, w, s) : s;
            }
            if (live && at.skip[k] < V) h[k].store(static_cast<R *>(a.h) + base + at.col[k]);
        }
        float r2 = 0.f;
        if (a.pre) {
            r2 = 1.f / sqrtf(row_sum(s) / C + a.eps);
            if (live) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (at.skip[k] >= V) continue;
                    Vec<P, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.set(i, h[k].get(i) * r2 * pre[k][i]);
                    o.store(static_cast<R *>(a.n) + base + at.col[k]);
                }
            }
        }
        if (a.stats && live && at.sub == 0) {
            a.stats[2 * r] = a.post ? r1 : 0.f;
            a.stats[2 * r + 1] = r2;
        }
    }
}

template <class P, int V, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void block_norm_bwd_kernel(const BlockNormArgs a) {
    using R = typename P::R;
    __shared__ float red[32];
    extern __shared__ float sums[];              // [rows a block][3][C], where a block has several rows
    RowSum row_sum{red, a.LG, 0};
    const Place<V, K> at(a);
    float post[K][V], scale[K][V], pre[K][V];
    columns<P, V, K>(a.post, at, post);
    columns<P, V, K>(a.scale, at, scale);
    columns<P, V, K>(a.pre, at, pre);
    float spost[K][V] = {}, sscale[K][V] = {}, spre[K][V] = {};
    Vec<P, V> y[K], h[K], z[K], th[K], tn[K];
    auto load = [&](long long r) {
        const size_t base = static_cast<size_t>(r < a.N ? r : a.N - 1) * a.C;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            y[k].load(static_cast<const R *>(a.y) + base + at.col[k]);
            if (a.gate) z[k].load(static_cast<const R *>(a.gate) + base + at.col[k]);
            if (a.dh) th[k].load(static_cast<const R *>(a.dh) + base + at.col[k]);
            if (a.dn) {
                h[k].load(static_cast<const R *>(a.h) + base + at.col[k]);
                tn[k].load(static_cast<const R *>(a.dn) + base + at.col[k]);
            }
        }
    };
    const float inv = 1.f / static_cast<float>(a.C);
    const long long step = static_cast<long long>(gridDim.x) * at.rpb;
    for (long long first = static_cast<long long>(blockIdx.x) * at.rpb; first < a.N; first += step) {
        const long long r = first + at.row;
        const bool live = r < a.N;
        load(r);
        const float r1 = a.post ? a.stats[2 * (live ? r : a.N - 1)] : 1.f, r2 = a.dn ? a.stats[2 * (live ? r : a.N - 1) + 1] : 0.f;
        const size_t base = static_cast<size_t>(r) * a.C;
        float t[K][V];
        if (a.dn) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float e = h[k].get(i) * r2, d = tn[k].get(i);
                    t[k][i] = d * pre[k][i];
                    if (i >= at.skip[k]) {
                        m = fmaf(t[k][i], e, m);
                        if (live) spre[k][i] = fmaf(d, e, spre[k][i]);
                    }
                }
            m = row_sum(m) * inv;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    t[k][i] = r2 * (t[k][i] - h[k].get(i) * r2 * m);
                    if (a.dh) t[k][i] += th[k].get(i);
                }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) t[k][i] = a.dh ? th[k].get(i) : 0.f;
        }
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Vec<P, V> ot, og;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ot.set(i, t[k][i]);
                const float hat = y[k].get(i) * r1, f = hat * post[k][i];
                float u = 1.f;
                if (a.gate) {
                    const Gate g = gate_of(z[k].get(i), a.act);
                    og.set(i, t[k][i] * scale[k][i] * f * g.du);
                    u = g.u;
                }
                const float tu = t[k][i] * u, df = tu * scale[k][i];
                t[k][i] = df * post[k][i];
                if (i >= at.skip[k]) {
                    m = fmaf(t[k][i], hat, m);
                    if (live) {
                        sscale[k][i] = fmaf(tu, f, sscale[k][i]);
                        spost[k][i] = fmaf(df, hat, spost[k][i]);
                    }
                }
            }
            if (live && at.skip[k] < V) {
                if (a.dx) ot.store(static_cast<R *>(a.dx) + base + at.col[k]);
                if (a.gate) og.store(static_cast<R *>(a.dgate) + base + at.col[k]);
            }
        }
        if (a.post) m = row_sum(m) * inv;
        if (live) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (at.skip[k] >= V) continue;
                Vec<P, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.set(i, a.post ? r1 * (t[k][i] - y[k].get(i) * r1 * m) : t[k][i]);
                o.store(static_cast<R *>(a.dy) + base + at.col[k]);
            }
        }
    }
    if (!a.part) return;
    float *to = a.part + static_cast<size_t>(blockIdx.x) * 3 * a.C;
    float *mine = at.rpb > 1 ? sums + at.row * 3 * a.C : to;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i < at.skip[k]) continue;
            const int c = at.col[k] + i;
            mine[c] = spost[k][i];
            mine[a.C + c] = sscale[k][i];
            mine[2 * a.C + c] = spre[k][i];
        }
    if (at.rpb > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < 3 * a.C; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < at.rpb; ++i) s += sums[i * 3 * a.C + c];
            to[c] = s;
        }
    }
}

// ---------------------------------------------------------------- rows of any length
// A workgroup of 1024 a row; every pass reads the row again, one element a lane.
template <class P>
__global__ __launch_bounds__(kMaxLanes) void block_norm_long_kernel(const BlockNormArgs a) {
    using R = typename P::R;
    __shared__ float red[32];
    RowSum row_sum{red, kMaxLanes, 0};
    const float C = static_cast<float>(a.C);
    for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
        const size_t base = static_cast<size_t>(r) * a.C;
        const R *y = static_cast<const R *>(a.y) + base, *x = static_cast<const R *>(a.x) + (a.x ? base : 0);
        const R *z = static_cast<const R *>(a.gate) + (a.gate ? base : 0);
        R *h = static_cast<R *>(a.h) + base;
        float r1 = 1.f;
        if (a.post) {
            float q = 0.f;
            for (int c = threadIdx.x; c < a.C; c += kMaxLanes) {
                const float v = P::to_f32(y[c]);
                q = fmaf(v, v, q);
            }
            r1 = 1.f / sqrtf(row_sum(q) / C + a.eps);
        }
        float s = 0.f;
        for (int c = threadIdx.x; c < a.C; c += kMaxLanes) {
            float v = P::to_f32(y[c]) * r1 * (a.post ? a.post[c] : 1.f) * (a.scale ? a.scale[c] : 1.f);
            if (a.gate) v *= gate_of(P::to_f32(z[c]), a.act).u;
            if (a.x) v += P::to_f32(x[c]);
            const R w = P::from_f32(v);
            h[c] = w;
            s = fmaf(P::to_f32(w), P::to_f32(w), s);
        }
        float r2 = 0.f;
        if (a.pre) {
            r2 = 1.f / sqrtf(row_sum(s) / C + a.eps);
            R *n = static_cast<R *>(a.n) + base;
            for (int c = threadIdx.x; c < a.C; c += kMaxLanes) n[c] = P::from_f32(P::to_f32(h[c]) * r2 * a.pre[c]);
        }
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * r] = a.post ? r1 : 0.f;
            a.stats[2 * r + 1] = r2;
        }
    }
}
template <class P>
__global__ __launch_bounds__(kMaxLanes) void block_norm_bwd_long_kernel(const BlockNormArgs a) {
    using R = typename P::R;
    __shared__ float red[32];
    RowSum row_sum{red, kMaxLanes, 0};
    const float inv = 1.f / static_cast<float>(a.C);
    float *sum = a.part ? a.part + static_cast<size_t>(blockIdx.x) * 3 * a.C : nullptr;
    for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
        const bool fresh = r == blockIdx.x;          // a column's sums are its own thread's
        const size_t base = static_cast<size_t>(r) * a.C;
        auto at = [&](const void *p, int c) { return P::to_f32(static_cast<const R *>(p)[base + c]); };
        const float r1 = a.post ? a.stats[2 * r] : 1.f, r2 = a.dn ? a.stats[2 * r + 1] : 0.f;
        float m2 = 0.f;
        if (a.dn) {
            for (int c = threadIdx.x; c < a.C; c += kMaxLanes) {
                const float e = at(a.h, c) * r2, d = at(a.dn, c);
                m2 = fmaf(d * a.pre[c], e, m2);
                if (sum) sum[2 * static_cast<size_t>(a.C) + c] = fmaf(d, e, fresh ? 0.f : sum[2 * static_cast<size_t>(a.C) + c]);
            }
            m2 = row_sum(m2) * inv;
        } else if (sum && fresh) {
            for (int c = threadIdx.x; c < a.C; c += kMaxLanes) sum[2 * static_cast<size_t>(a.C) + c] = 0.f;
        }
        auto reach = [&](int c) {
            float t = a.dh ? at(a.dh, c) : 0.f;
            if (a.dn) t += r2 * (at(a.dn, c) * a.pre[c] - at(a.h, c) * r2 * m2);
            return t;
        };
        float m1 = 0.f;
        for (int c = threadIdx.x; c < a.C; c += kMaxLanes) {
            const float t = reach(c), w = a.post ? a.post[c] : 1.f, sc = a.scale ? a.scale[c] : 1.f;
            const float hat = at(a.y, c) * r1, f = hat * w;
            Gate g{1.f, 0.f};
            if (a.gate) {
                g = gate_of(at(a.gate, c), a.act);
                static_cast<R *>(a.dgate)[base + c] = P::from_f32(t * sc * f * g.du);
            }
            if (a.dx) static_cast<R *>(a.dx)[base + c] = P::from_f32(t);
            const float df = t * g.u * sc;
            m1 = fmaf(df * w, hat, m1);
            if (sum) {
                sum[c] = fmaf(df, hat, fresh ? 0.f : sum[c]);
                sum[a.C + c] = fmaf(t * g.u, f, fresh ? 0.f : sum[a.C + c]);
            }
            if (!a.post) static_cast<R *>(a.dy)[base + c] = P::from_f32(df);
        }
        if (!a.post) continue;
        m1 = row_sum(m1) * inv;
        for (int c = threadIdx.x; c < a.C; c += kMaxLanes) {
            float df = reach(c) * (a.scale ? a.scale[c] : 1.f);
            if (a.gate) df *= gate_of(at(a.gate, c), a.act).u;
            static_cast<R *>(a.dy)[base + c] = P::from_f32(r1 * (df * a.post[c] - at(a.y, c) * r1 * m1));
        }
    }
}

struct BlockNormStore {
    float *post, *scale, *pre;
    int C;
    __device__ __forceinline__ void operator()(long long c, float v) const {
        if (c < C) { if (post) post[c] = v; }
        else if (c < 2LL * C) { if (scale) scale[c - C] = v; }
        else if (pre) pre[c - 2LL * C] = v;
    }
};
__global__ __launch_bounds__(256) void block_norm_zero_kernel(BlockNormStore to) {
    const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (c < 3LL * to.C) to(c, 0.f);
}

// Lanes and vectors of a row
void plan(int dtype, BlockNormArgs &a) {
    a.V = dtype == 1 ? 8 : 4;
    if (a.C < a.V) a.V = 1;
    const int nvec = (a.C - 1) / a.V + 1, most = dtype == 1 ? 1 : 2;
    a.LG = 1;
    while (a.LG < kMaxLanes && a.LG < nvec) a.LG *= 2;
    a.K = (nvec + a.LG - 1) / a.LG;
    if (a.K > most) a.K = 0;
}
int threads(const BlockNormArgs &a) { return a.LG > 256 ? a.LG : 256; }
int grid_of(const BlockNormArgs &a, int most) {
    const long long rpb = a.K ? threads(a) / a.LG : 1, n = (a.N + rpb - 1) / rpb;
    return static_cast<int>(n < most ? n : most);
}
// Workgroups: twice what the card holds of the forward (32768 x 2048 bf16 131 us, half as many 137, four
// times 128; 4096 x 4096 27, 27, 28; 30000 x 256 15.7, 14.9, 15.8); for the backward, as many as are
// resident at once, each of which writes a row of partial sums (32768 x 2048 214 us, half 284, twice
// 232; 30000 x 256 30, 34, 36; 5000 x 1923 fp32 46, 53, 48).
int fwd_grid(const BlockNormArgs &a) { return grid_of(a, 4096 * 256 / threads(a)); }
int bwd_grid(const BlockNormArgs &a) { return grid_of(a, 768 * 256 / threads(a)); }

template <class P, int V, int K, int THREADS>
void run(const BlockNormArgs &a, bool back, hipStream_t stream) {
    const int n = threads(a);
    const unsigned lds = back && a.part && n > a.LG ? n / a.LG * 3u * a.C * sizeof(float) : 0;
    if (back) hipLaunchKernelGGL((block_norm_bwd_kernel<P, V, K, THREADS>), dim3(a.grid), dim3(n), lds, stream, a);
    else hipLaunchKernelGGL((block_norm_kernel<P, V, K, THREADS>), dim3(a.grid), dim3(n), 0, stream, a);
}
template <class P>
void dispatch(const BlockNormArgs &a, bool back, hipStream_t stream) {
    constexpr int V = 16 / P::kBytes;
    if (a.K == 0) {
        if (back) hipLaunchKernelGGL(block_norm_bwd_long_kernel<P>, dim3(a.grid), dim3(kMaxLanes), 0, stream, a);
        else hipLaunchKernelGGL(block_norm_long_kernel<P>, dim3(a.grid), dim3(kMaxLanes), 0, stream, a);
    } else if (a.V == 1) {
        run<P, 1, 1, 256>(a, back, stream);
    } else if (a.K == 1) {
        if (a.LG <= 256) run<P, V, 1, 256>(a, back, stream);
        else run<P, V, 1, 1024>(a, back, stream);
    } else if constexpr (P::kBytes == 4) {
        run<P, V, 2, 1024>(a, back, stream);
    }
}

}  // namespace

bool block_norm_fits(int dtype, int N, int C) { return C < (1 << 28); }

hipError_t launch_block_norm_fwd(int dtype, BlockNormArgs a, hipStream_t stream) {
    plan(dtype, a);
    a.grid = a.K ? fwd_grid(a) : grid_of(a, 1024);
    if (dtype == 1) dispatch<Bf16>(a, false, stream);
    else dispatch<F32>(a, false, stream);
    return hipGetLastError();
}

size_t block_norm_bwd_workspace(int dtype, int N, int C, bool sums) {
    if (!sums || N == 0 || C == 0) return 0;
    BlockNormArgs a{};
    a.N = N;
    a.C = C;
    plan(dtype, a);
    return static_cast<size_t>(a.K ? bwd_grid(a) : grid_of(a, 256)) * 3 * C * sizeof(float);
}

hipError_t launch_block_norm_bwd(int dtype, BlockNormArgs a, void *ws, hipStream_t stream) {
    const bool sums = a.dpost || a.dscale || a.dpre;
    const BlockNormStore store{a.dpost, a.dscale, a.dpre, a.C};
    if (a.N == 0) {
        if (sums) hipLaunchKernelGGL(block_norm_zero_kernel, dim3((3LL * a.C + 255) / 256), dim3(256), 0, stream, store);
        return hipGetLastError();
    }
    plan(dtype, a);
    a.grid = a.K ? bwd_grid(a) : grid_of(a, 256);
    a.part = sums ? static_cast<float *>(ws) : nullptr;
    if (dtype == 1) dispatch<Bf16>(a, true, stream);
    else dispatch<F32>(a, true, stream);
    if (sums) column_sum(a.part, a.grid, 3LL * a.C, store, stream);
    return hipGetLastError();
}

}  // namespace qd
