// C ABI of the operators around the recurrence (short convolution, selective scan, group
// norm): host-side argument checks, then kernel dispatch.  Every check happens before
// anything is enqueued; nothing here allocates.
#include "qdelta.h"
#include "qd_checks.h"
#include "qd_mixer.h"

using qd::aligned16;
using qd::disjoint;

namespace {

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}
bool dtype_ok(int dtype) { return dtype == QD_F32 || dtype == QD_BF16; }
size_t elem(int dtype) { return dtype == QD_BF16 ? 2 : 4; }
size_t prod(size_t a, size_t b, size_t c = 1, size_t d = 1) { return a * b * c * d; }
int status(hipError_t e) { return e == hipSuccess ? QD_OK : QD_ERR_HIP; }

bool ssm_sizes(int B, int T, int D, int G, int N) { return B >= 0 && T >= 0 && D >= 0 && G >= 1 && N >= 0 && D % G == 0; }
bool norm_sizes(int N, int L, int C, int G) { return N >= 0 && L >= 0 && C >= 0 && G >= 1 && C % G == 0; }

}  // namespace

extern "C" {

int qdelta_conv_fwd(const void *x, const float *w, const float *bias, const void *S0, const int *lens, void *y, void *S_T,
                    int B, int T, int D, int W, int silu, int dtype, void *stream) {
    if (B < 0 || T < 0 || D < 0) return QD_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || W < 2 || W > 4 || (D > 0 && !qd::conv_fits(B, T, D))) return QD_ERR_UNSUPPORTED;
    if (B == 0 || D == 0) return QD_OK;
    if (!w || (T > 0 && (!x || !y))) return QD_ERR_INVALID_ARG;
    if (!all_aligned({x, y, S0, S_T})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, D, elem(dtype)), st = prod(B, W - 1, D, elem(dtype));
    if (!disjoint({{x, n}, {w, prod(D, W, 4)}, {bias, prod(D, 4)}, {S0, st}, {lens, prod(B, 4)}}, {{y, n}, {S_T, st}}, S0, S_T))
        return QD_ERR_INVALID_ARG;
    return status(qd::launch_conv_fwd(dtype, qd::ConvArgs{x, w, bias, S0, lens, y, S_T, B, T, D, W, silu != 0, 0},
                                      static_cast<hipStream_t>(stream)));
}

int qdelta_conv_step(const void *x, const float *w, const float *bias, void *S, void *y, int N, int D, int W, int silu,
                     int dtype, void *stream) {
    if (N < 0 || D < 0) return QD_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || W < 2 || W > 4 || (D > 0 && !qd::conv_fits(N, 1, D))) return QD_ERR_UNSUPPORTED;
    if (N == 0 || D == 0) return QD_OK;
    if (!x || !w || !S || !y) return QD_ERR_INVALID_ARG;
    if (!all_aligned({x, y, S})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(N, D, elem(dtype)), st = prod(N, W - 1, D, elem(dtype));
    if (!disjoint({{x, n}, {w, prod(D, W, 4)}, {bias, prod(D, 4)}}, {{y, n}, {S, st}})) return QD_ERR_INVALID_ARG;
    return status(qd::launch_conv_step(dtype, qd::ConvArgs{x, w, bias, S, nullptr, y, S, N, 1, D, W, silu != 0, 0},
                                       static_cast<hipStream_t>(stream)));
}

size_t qdelta_conv_bwd_workspace_bytes(int B, int T, int D, int W, int dtype) {
    if (B <= 0 || T <= 0 || D <= 0 || W < 2 || W > 4 || !dtype_ok(dtype) || !qd::conv_fits(B, T, D)) return 0;
    return qd::conv_bwd_workspace(B, T, D, W);
}

int qdelta_conv_bwd(const void *x, const float *w, const float *bias, const void *S0, const int *lens, const void *dy,
                    const void *dS_T, void *dx, float *dw, float *dbias, void *dS0, int B, int T, int D, int W, int silu,
                    int dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (B < 0 || T < 0 || D < 0) return QD_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || W < 2 || W > 4 || (D > 0 && !qd::conv_fits(B, T, D))) return QD_ERR_UNSUPPORTED;
    if (D == 0) return QD_OK;
    if (!w || !dw || (prod(B, T) > 0 && (!x || !dy || !dx))) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_conv_bwd_workspace_bytes(B, T, D, W, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({x, S0, dy, dS_T, dx, dS0})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, D, elem(dtype)), st = prod(B, W - 1, D, elem(dtype));
    if (!disjoint({{x, n}, {w, prod(D, W, 4)}, {bias, prod(D, 4)}, {S0, st}, {lens, prod(B, 4)}, {dy, n}, {dS_T, st}},
                  {{dx, n}, {dw, prod(D, W, 4)}, {dbias, prod(D, 4)}, {dS0, st}, {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    return status(qd::launch_conv_bwd(dtype, qd::ConvBwdArgs{x, w, bias, S0, lens, dy, dS_T, dx, dS0, dw, dbias,
                                                             static_cast<float *>(workspace), B, T, D, W, silu != 0, 0, 0, 0},
                                      static_cast<hipStream_t>(stream)));
}

size_t qdelta_ssm_fwd_workspace_bytes(int B, int T, int D, int G, int N, int dtype) {
    if (!ssm_sizes(B, T, D, G, N) || !qd::ssm_supported(dtype, N) || !qd::ssm_fits(B, T, D, G, N)) return 0;
    return prod(B, D) == 0 ? 0 : qd::ssm_fwd_workspace(B, T, D, G, N);
}

int qdelta_ssm_fwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                   const void *z, const float *dt_bias, const float *S0, const int *lens, void *o, float *S_T, int B, int T,
                   int D, int G, int N, int softplus, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (!ssm_sizes(B, T, D, G, N)) return QD_ERR_INVALID_ARG;
    if (!qd::ssm_supported(dtype, N) || !qd::ssm_fits(B, T, D, G, N)) return QD_ERR_UNSUPPORTED;
    if (B == 0 || D == 0) return QD_OK;
    if (!A || (T > 0 && (!u || !dt || !Bm || !Cm || !o))) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_ssm_fwd_workspace_bytes(B, T, D, G, N, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({u, dt, A, Bm, Cm, z, S0, o, S_T})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, D, elem(dtype)), bc = prod(prod(B, T, G), N, elem(dtype)), st = prod(B, D, N, 4);
    if (!disjoint({{u, n}, {dt, n}, {A, prod(D, N, 4)}, {Bm, bc}, {Cm, bc}, {Dskip, prod(D, 4)}, {z, n},
                   {dt_bias, prod(D, 4)}, {S0, st}, {lens, prod(B, 4)}},
                  {{o, n}, {S_T, st}, {need ? workspace : nullptr, need}}, S0, S_T))
        return QD_ERR_INVALID_ARG;
    return status(qd::launch_ssm_fwd(dtype, qd::SsmArgs{u, dt, Bm, Cm, A, Dskip, dt_bias, z, S0, lens, o, S_T, B, T, D, G, N,
                                                        softplus != 0},
                                     workspace, static_cast<hipStream_t>(stream)));
}

int qdelta_ssm_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                    const void *z, const float *dt_bias, float *S, void *o, int N_seq, int D, int G, int N, int softplus,
                    int dtype, void *stream) {
    if (!ssm_sizes(N_seq, 1, D, G, N)) return QD_ERR_INVALID_ARG;
    if (!qd::ssm_supported(dtype, N) || !qd::ssm_fits(N_seq, 1, D, G, N)) return QD_ERR_UNSUPPORTED;
    if (N_seq == 0 || D == 0) return QD_OK;
    if (!u || !dt || !A || !Bm || !Cm || !S || !o) return QD_ERR_INVALID_ARG;
    if (!all_aligned({u, dt, A, Bm, Cm, z, S, o})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(N_seq, D, elem(dtype)), bc = prod(N_seq, G, N, elem(dtype)), st = prod(N_seq, D, N, 4);
    if (!disjoint({{u, n}, {dt, n}, {A, prod(D, N, 4)}, {Bm, bc}, {Cm, bc}, {Dskip, prod(D, 4)}, {z, n}, {dt_bias, prod(D, 4)}},
                  {{o, n}, {S, st}}))
        return QD_ERR_INVALID_ARG;
    return status(qd::launch_ssm_step(dtype, qd::SsmArgs{u, dt, Bm, Cm, A, Dskip, dt_bias, z, S, nullptr, o, S, N_seq, 1, D, G,
                                                         N, softplus != 0},
                                      static_cast<hipStream_t>(stream)));
}

size_t qdelta_ssm_bwd_workspace_bytes(int B, int T, int D, int G, int N, int dtype) {
    if (!ssm_sizes(B, T, D, G, N) || !qd::ssm_supported(dtype, N) || !qd::ssm_fits(B, T, D, G, N)) return 0;
    return qd::ssm_bwd_workspace(B, T, D, G, N);
}

int qdelta_ssm_bwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                   const void *z, const float *dt_bias, const float *S0, const int *lens, const void *d_o, const float *dS_T,
                   void *du, void *ddt, float *dA, void *dB, void *dC, float *dDskip, void *dz, float *ddt_bias, float *dS0,
                   int B, int T, int D, int G, int N, int softplus, int dtype, void *workspace, size_t ws_bytes,
                   void *stream) {
    if (!ssm_sizes(B, T, D, G, N)) return QD_ERR_INVALID_ARG;
    if (!qd::ssm_supported(dtype, N) || !qd::ssm_fits(B, T, D, G, N)) return QD_ERR_UNSUPPORTED;
    if (D == 0) return QD_OK;
    if (!A || !dA || (prod(B, T) > 0 && (!u || !dt || !Bm || !Cm || !d_o || !du || !ddt || !dB || !dC)))
        return QD_ERR_INVALID_ARG;
    if (prod(B, T) > 0 && (z != nullptr) != (dz != nullptr)) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_ssm_bwd_workspace_bytes(B, T, D, G, N, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({u, dt, A, Bm, Cm, z, S0, d_o, dS_T, du, ddt, dA, dB, dC, dz, dS0})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(B, T, D, elem(dtype)), bc = prod(prod(B, T, G), N, elem(dtype)), st = prod(B, D, N, 4);
    const size_t an = prod(D, N, 4), dn = prod(D, 4);
    if (!disjoint({{u, n}, {dt, n}, {A, an}, {Bm, bc}, {Cm, bc}, {Dskip, dn}, {z, n}, {dt_bias, dn}, {S0, st}, {lens, prod(B, 4)},
                   {d_o, n}, {dS_T, st}},
                  {{du, n}, {ddt, n}, {dA, an}, {dB, bc}, {dC, bc}, {dDskip, dn}, {dz, n}, {ddt_bias, dn}, {dS0, st},
                   {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    return status(qd::launch_ssm_bwd(dtype, qd::SsmBwdArgs{u, dt, Bm, Cm, A, Dskip, dt_bias, z, S0, lens, d_o, dS_T, du, ddt, dB,
                                                           dC, dz, dA, dDskip, ddt_bias, dS0, B, T, D, G, N, softplus != 0},
                                     workspace, static_cast<hipStream_t>(stream)));
}

size_t qdelta_group_norm_fwd_workspace_bytes(int N, int L, int C, int G, int dtype) {
    if (!norm_sizes(N, L, C, G) || !dtype_ok(dtype) || C == 0 || !qd::norm_fits(dtype, N, L, C, G)) return 0;
    return qd::norm_fwd_workspace(dtype, N, L, C, G);
}

int qdelta_group_norm_fwd(const void *x, const float *weight, const float *bias, const void *gate, void *y, float *stats,
                          int N, int L, int C, int G, float eps, int silu, int dtype, void *workspace, size_t ws_bytes,
                          void *stream) {
    if (!norm_sizes(N, L, C, G) || !(eps >= 0.f && eps <= 3.0e38f)) return QD_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QD_ERR_UNSUPPORTED;
    if (prod(N, L, C) == 0) return QD_OK;
    if (!qd::norm_fits(dtype, N, L, C, G)) return QD_ERR_UNSUPPORTED;
    if (!x || !y) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_group_norm_fwd_workspace_bytes(N, L, C, G, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({x, gate, y})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(N, L, C, elem(dtype)), c = prod(C, 4);
    if (!disjoint({{x, n}, {weight, c}, {bias, c}, {gate, n}},
                  {{y, n}, {stats, prod(N, G, 8)}, {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    qd::NormArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.gate = gate; a.y = y; a.stats = stats;
    a.N = N; a.L = L; a.C = C; a.G = G; a.eps = eps; a.silu = silu != 0;
    return status(qd::launch_norm_fwd(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

size_t qdelta_group_norm_bwd_workspace_bytes(int N, int L, int C, int G, int dtype) {
    if (!norm_sizes(N, L, C, G) || !dtype_ok(dtype) || C == 0 || !qd::norm_fits(dtype, N, L, C, G)) return 0;
    return qd::norm_bwd_workspace(dtype, N, L, C, G);
}

int qdelta_group_norm_bwd(const void *x, const float *weight, const float *bias, const void *gate, const float *stats,
                          const void *dy, void *dx, float *dweight, float *dbias, void *dgate, int N, int L, int C, int G,
                          int silu, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (!norm_sizes(N, L, C, G)) return QD_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QD_ERR_UNSUPPORTED;
    if (C == 0) return QD_OK;
    if (prod(N, L) == 0) {
        // no rows: the sums over rows are zero
        return status(qd::launch_norm_zero(dweight, dbias, C, static_cast<hipStream_t>(stream)));
    }
    if (!qd::norm_fits(dtype, N, L, C, G)) return QD_ERR_UNSUPPORTED;
    if (!x || !stats || !dy || !dx || (gate != nullptr) != (dgate != nullptr)) return QD_ERR_INVALID_ARG;
    const size_t need = qdelta_group_norm_bwd_workspace_bytes(N, L, C, G, dtype);
    if (ws_bytes < need || (need > 0 && (!workspace || !aligned16(workspace)))) return QD_ERR_WORKSPACE;
    if (!all_aligned({x, gate, dy, dx, dgate})) return QD_ERR_INVALID_ARG;
    const size_t n = prod(N, L, C, elem(dtype)), c = prod(C, 4);
    if (!disjoint({{x, n}, {weight, c}, {bias, c}, {gate, n}, {stats, prod(N, G, 8)}, {dy, n}},
                  {{dx, n}, {dweight, c}, {dbias, c}, {dgate, n}, {need ? workspace : nullptr, need}}))
        return QD_ERR_INVALID_ARG;
    qd::NormArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.gate = gate; a.stats = const_cast<float *>(stats);
    a.dy = dy; a.dx = dx; a.dgate = dgate; a.dw = dweight; a.dbias = dbias;
    a.N = N; a.L = L; a.C = C; a.G = G; a.silu = silu != 0;
    return status(qd::launch_norm_bwd(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
