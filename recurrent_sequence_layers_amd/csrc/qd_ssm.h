// Device pieces shared by the selective scan's forward and backward kernels.
#pragma once

#include "qd_internal.h"
#include "qd_mixer.h"

namespace qd {

constexpr int kTok = 8;              // tokens per tile

// One token's B or C values for the wave's NS states, read through the scalar cache: the
// address is the same for every lane, so the values arrive in scalar registers and enter
// the vector instructions as they are.  The row start is a multiple of NS elements.
typedef const __attribute__((address_space(4))) uint32_t scalar_u32;
template <class P, int NS>
struct ScalarRow {
    static constexpr int kDw = NS * P::kBytes / 4;
    uint32_t q[kDw];
    __device__ __forceinline__ void load(const typename P::R *p) {
        scalar_u32 *s = (scalar_u32 *)(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int i = 0; i < kDw; ++i) q[i] = s[i];
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (P::kBytes == 4) return __uint_as_float(q[i]);
        else return __uint_as_float((i & 1) ? (q[i / 2] & 0xffff0000u) : (q[i / 2] << 16));
    }
};

// How the time axis is cut: P segments of `len` tokens (a multiple of kTok), walked at the
// same time; P = 1 needs no workspace for it.
struct Segments {
    int P, len;
};
inline Segments cut_time(int T, int want) {
    Segments s;
    const int tiles = (T + kTok - 1) / kTok;
    s.P = want < 1 ? 1 : want;
    if (s.P > tiles) s.P = tiles < 1 ? 1 : tiles;
    s.len = (tiles + s.P - 1) / s.P * kTok;
    if (s.len < kTok) s.len = kTok;
    s.P = (T + s.len - 1) / s.len;
    if (s.P < 1) s.P = 1;
    return s;
}

// Workspace of the segmented walk: each segment's effect on the state is
// h_out = exp(A2 sum(delta)) h_in + h_local (base-2 exponent, A2 = A log2 e).
struct SegBuf {
    float *h;                        // [B][P][N][D]: slot 0 the entry state, slot q + 1 segment q's h_local
    float *s;                        // [B][P][D]: segment q's sum of delta (slot q)
};

// The scan's launches (qd_ssm.hip) for the backward: the segments' effects, then the walk
// that keeps the state before every tile of kTok tokens, [B][ceil(T / kTok)][N][D].
hipError_t launch_ssm_states(int dtype, const SsmArgs &a, Segments seg, SegBuf buf, float *keep, hipStream_t stream);

}  // namespace qd
