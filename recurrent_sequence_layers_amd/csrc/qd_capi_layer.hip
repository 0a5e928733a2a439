// C ABI of linear attention with a decay for each head and of the RMS norms around a block:
// host-side argument checks, then kernel dispatch.  Every check happens before anything is
// enqueued; nothing here allocates.
#include "qdelta.h"
#include "qd_block_norm.h"
#include "qd_checks.h"
#include "qd_linattn.h"

using qd::aligned16;
using qd::disjoint;

namespace {

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}
size_t elem(int dtype) { return dtype == QD_BF16 ? 2 : 4; }
size_t prod(size_t a, size_t b, size_t c = 1, size_t d = 1) { return a * b * c * d; }
int status(hipError_t e) { return e == hipSuccess ? QD_OK : QD_ERR_HIP; }
int decay_of(const float *g, int per_head) { return !g ? qd::kNoDecay : per_head ? qd::kHeadDecay : qd::kTokenDecay; }
size_t decay_bytes(int B, int T, int H, int per_head) { return per_head ? prod(H, 4) : prod(prod(B, T), H, 4); }

bool lin_ok(int B, int T, int H, int d_k, int d_v, int dtype, qd::LinCall call) {
    return qd::lin_supported(dtype, d_k, d_v) && qd::lin_fits(dtype, B, T, H, call);
}
bool norm_ok(int N, int C, int dtype) { return (dtype == QD_F32 || dtype == QD_BF16) && qd::block_norm_fits(dtype, N, C); }

}  // namespace

extern "C" {

size_t qdelta_linattn_fwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || !lin_ok(B, T, H, d_k, d_v, dtype, qd::kLinFwd)) return 0;
    return qd::lin_fwd_workspace(dtype, B, T, H, d_k, d_v);
}

int qdelta_linattn_fwd(const void *q, const void *k, const void *v, const float *g, const float *S0, const int *lens, void *o,
                       float *S_T, int B, int T, int H, int d_k, int d_v, int g_per_head, int dtype, void *workspace,
                       size_t ws_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0) return QD_ERR_INVALID_ARG;
    if (!lin_ok(B, T, H, d_k, d_v, dtype, qd::kLinFwd)) return QD_ERR_UNSUPPORTED;
    if (prod(B, H) == 0) return QD_OK;
    if (T > 0 && (!q || !k || !v || !o)) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_linattn_fwd_workspace_bytes(B, T, H, d_k, d_v, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({q, k, v, S0, o, S_T})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, H, elem(dtype)), st = prod(prod(B, H), d_k, d_v, 4);
    if (!disjoint({{q, n * d_k}, {k, n * d_k}, {v, n * d_v}, {g, decay_bytes(B, T, H, g_per_head)}, {S0, st}, {lens, prod(B, 4)}},
                  {{o, n * d_v}, {S_T, st}, {need ? workspace : nullptr, need}}, S0, S_T))
        return QD_ERR_INVALID_ARG;
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.lens = lens; a.o = o; a.S_T = S_T;
    a.B = B; a.T = T; a.H = H; a.DK = d_k; a.DV = d_v; a.decay = decay_of(g, g_per_head);
    return status(qd::launch_lin_fwd(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

int qdelta_linattn_step(const void *q, const void *k, const void *v, const float *g, float *S, void *o, int N, int H, int d_k,
                        int d_v, int g_per_head, int dtype, void *stream) {
    if (N < 0 || H < 0) return QD_ERR_INVALID_ARG;
    if (!lin_ok(N, 1, H, d_k, d_v, dtype, qd::kLinStep)) return QD_ERR_UNSUPPORTED;
    if (prod(N, H) == 0) return QD_OK;
    if (!q || !k || !v || !S || !o) return QD_ERR_INVALID_ARG;
    if (!all_aligned({q, k, v, S, o})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(N, H, elem(dtype)), st = prod(prod(N, H), d_k, d_v, 4);
    if (!disjoint({{q, n * d_k}, {k, n * d_k}, {v, n * d_v}, {g, decay_bytes(N, 1, H, g_per_head)}}, {{o, n * d_v}, {S, st}}))
        return QD_ERR_INVALID_ARG;
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.o = o;
    a.B = N; a.T = 1; a.H = H; a.DK = d_k; a.DV = d_v; a.decay = decay_of(g, g_per_head);
    return status(qd::launch_lin_step(dtype, a, S, static_cast<hipStream_t>(stream)));
}

size_t qdelta_linattn_bwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int want_dg, int dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || !lin_ok(B, T, H, d_k, d_v, dtype, qd::kLinBwd)) return 0;
    return qd::lin_bwd_workspace(dtype, B, T, H, d_k, d_v, want_dg != 0);
}

int qdelta_linattn_bwd(const void *q, const void *k, const void *v, const float *g, const float *S0, const int *lens,
                       const void *d_o, const float *dS_T, void *dq, void *dk, void *dv, float *dg, float *dS0, int B, int T,
                       int H, int d_k, int d_v, int g_per_head, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0) return QD_ERR_INVALID_ARG;
    if (!lin_ok(B, T, H, d_k, d_v, dtype, qd::kLinBwd)) return QD_ERR_UNSUPPORTED;
    if (H == 0) return QD_OK;
    if (!g && dg) return QD_ERR_INVALID_ARG;
    if (prod(B, T) > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_linattn_bwd_workspace_bytes(B, T, H, d_k, d_v, dg != nullptr, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({q, k, v, S0, d_o, dS_T, dq, dk, dv, dS0})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, H, elem(dtype)), st = prod(prod(B, H), d_k, d_v, 4), gn = decay_bytes(B, T, H, g_per_head);
    if (!disjoint({{q, n * d_k}, {k, n * d_k}, {v, n * d_v}, {g, gn}, {S0, st}, {lens, prod(B, 4)}, {d_o, n * d_v}, {dS_T, st}},
                  {{dq, n * d_k}, {dk, n * d_k}, {dv, n * d_v}, {dg, gn}, {dS0, st}, {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.lens = lens; a.d_o = d_o; a.dS_T = dS_T;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dS0 = dS0;
    a.B = B; a.T = T; a.H = H; a.DK = d_k; a.DV = d_v; a.decay = decay_of(g, g_per_head);
    return status(qd::launch_lin_bwd(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

int qdelta_block_norm_fwd(const void *y, const void *x, const float *post, const void *gate, const float *scale,
                          const float *pre, void *h, void *n, float *stats, int N, int C, float eps, int act, int dtype,
                          void *stream) {
    if (N < 0 || C < 0 || !(eps >= 0.f && eps <= 3.0e38f) || act < QD_GATE_LINEAR || act > QD_GATE_SILU) return QD_ERR_INVALID_ARG;
    if (!norm_ok(N, C, dtype)) return QD_ERR_UNSUPPORTED;
    if (prod(N, C) == 0) return QD_OK;
    if (!y || !h || (pre != nullptr) != (n != nullptr)) return QD_ERR_INVALID_ARG;
    if (!all_aligned({y, x, gate, h, n})) return QD_ERR_INVALID_ARG;
    const size_t t = prod(N, C, elem(dtype)), c = prod(C, 4);
    if (!disjoint({{y, t}, {x, t}, {gate, t}, {post, c}, {scale, c}, {pre, c}}, {{h, t}, {n, t}, {stats, prod(N, 8)}}))
        return QD_ERR_INVALID_ARG;
    qd::BlockNormArgs a{};
    a.y = y; a.x = x; a.gate = gate; a.post = post; a.scale = scale; a.pre = pre; a.h = h; a.n = n; a.stats = stats;
    a.N = N; a.C = C; a.eps = eps; a.act = act;
    return status(qd::launch_block_norm_fwd(dtype, a, static_cast<hipStream_t>(stream)));
}

size_t qdelta_block_norm_bwd_workspace_bytes(int N, int C, int want_sums, int dtype) {
    if (N <= 0 || C <= 0 || !norm_ok(N, C, dtype)) return 0;
    return qd::block_norm_bwd_workspace(dtype, N, C, want_sums != 0);
}

int qdelta_block_norm_bwd(const void *y, const void *h, const float *post, const void *gate, const float *scale,
                          const float *pre, const float *stats, const void *dh, const void *dn, void *dx, void *dy, void *dgate,
                          float *dpost, float *dscale, float *dpre, int N, int C, int act, int dtype, void *workspace,
                          size_t ws_bytes, void *stream) {
    if (N < 0 || C < 0 || act < QD_GATE_LINEAR || act > QD_GATE_SILU) return QD_ERR_INVALID_ARG;
    if (!norm_ok(N, C, dtype)) return QD_ERR_UNSUPPORTED;
    if (C == 0) return QD_OK;
    if ((dn && !pre) || (!post && dpost) || (!scale && dscale) || (!pre && dpre)) return QD_ERR_INVALID_ARG;
    const bool sums = dpost || dscale || dpre;
    if (N > 0) {
        if (!y || !dy || (!dh && !dn) || (dn && !h) || ((post || dn) && !stats) || (gate != nullptr) != (dgate != nullptr))
            return QD_ERR_INVALID_ARG;
    }
    const size_t need = qdelta_block_norm_bwd_workspace_bytes(N, C, sums, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({y, h, gate, dh, dn, dx, dy, dgate})) return QD_ERR_INVALID_ARG;
    const size_t t = prod(N, C, elem(dtype)), c = prod(C, 4);
    if (!disjoint({{y, t}, {h, t}, {gate, t}, {post, c}, {scale, c}, {pre, c}, {stats, prod(N, 8)}, {dh, t}, {dn, t}},
                  {{dx, t}, {dy, t}, {dgate, t}, {dpost, c}, {dscale, c}, {dpre, c}, {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    qd::BlockNormArgs a{};
    a.y = y; a.h = const_cast<void *>(h); a.gate = gate; a.post = post; a.scale = scale; a.pre = pre;
    a.stats = const_cast<float *>(stats); a.dh = dh; a.dn = dn; a.dx = dx; a.dy = dy; a.dgate = dgate;
    a.dpost = dpost; a.dscale = dscale; a.dpre = dpre;
    a.N = N; a.C = C; a.act = act;
    return status(qd::launch_block_norm_bwd(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
