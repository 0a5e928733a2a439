// Device pieces shared by the selective scan's forward and backward kernels.
#pragma once

#include "qd_internal.h"
#include "qd_mixer.h"

namespace qd {

constexpr int kTok = 8;              // tokens between two kept states (backward)
constexpr int kTile = 16;            // tokens a forward workgroup stages at a time

// States a wave of the scan owns: N / kStates waves share 64 channels.
template <int N>
constexpr int states_per_wave() {
    return N == 16 ? 2 : 4;
}
inline int states_per_wave_of(int N) { return N == 16 ? states_per_wave<16>() : 4; }

// B and C for the scalar cache.  A wave's B and C values are the same for all its lanes, so
// they enter the vector instructions as scalar registers; read from the inputs they would
// come four or eight bytes a token.  A first launch writes them as fp32 in the order a wave
// reads them, [B][G][wave][Tp][states per wave], so that one scalar load brings the values of
// several tokens.  Rows from a sequence's length up to Tp, the next multiple of kTile and one
// tile more, are zero: a token past the end then changes nothing.
struct RowBuf {
    float *b, *c;
    int Tp;
};
inline int padded_rows(int T) { return (T + kTile - 1) / kTile * kTile + kTile; }

// The decay exponent's factor A log2 e.  A decay without bound (A = -inf, or one that the
// product makes so) becomes the largest finite one: a token past the end has delta = 0 and has
// to leave the state as it is, where 0 times infinity would be NaN.
__device__ __forceinline__ float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -3.4028234e38f ? -3.4028234e38f : r;
}
// Segments whose effects are loaded before they are composed: one after the other each would wait
// for its own loads (gradients of 3 x 203 tokens, 142 channels, 32 states 52 -> 45 us, of 2 x 128
// tokens, 256 channels, 64 states 67 -> 57; one prompt of 16000 tokens, 512 channels 92 -> 89; eight
// or sixteen at a time differ by 2 % either way).
constexpr int kCompose = 4;

// A state through a segment, 2^r h + local with r = rate sum_delta.  The factor enters by its root,
// twice: where 2^r alone would overflow or vanish (a small state that grows, a large one that decays)
// the product need not, and the root does neither for any r that leaves a normal h a normal product.
// (r's whole part put into the exponent reaches subnormal h too, but costs the small calls: 2048 tokens,
// 512 channels forward 27.7 against 24.8 us; gradients of 2 x 128 tokens, 256 channels, 64 states 59.8
// against 55.8.)
// Nothing carried stays nothing also where the root overflows.
__device__ __forceinline__ float carry(float rate, float sum_delta, float h, float local) {
    const float root = __builtin_amdgcn_exp2f(0.5f * rate * sum_delta);
    const float through = fmaf(root, root * h, local);
    return h == 0.f ? local : through;
}

typedef const __attribute__((address_space(4))) float scalar_f32;
// COUNT tokens' values from row p on.
template <int COUNT, int NS>
struct ScalarRows {
    float v[COUNT][NS];
    __device__ __forceinline__ void load(const float *p) {
        scalar_f32 *s = (scalar_f32 *)(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int t = 0; t < COUNT; ++t)
#pragma unroll
            for (int i = 0; i < NS; ++i) v[t][i] = s[t * NS + i];
    }
};

// How the time axis is cut: P segments of `len` tokens (a multiple of kTile), walked at the
// same time; P = 1 needs no segment workspace.
struct Segments {
    int P, len;
};
inline Segments cut_time(int T, long long want) {
    Segments s;
    const int tiles = (T + kTile - 1) / kTile;
    s.P = static_cast<int>(want < 1 ? 1 : want > 64 ? 64 : want);
    if (s.P > tiles) s.P = tiles < 1 ? 1 : tiles;
    s.len = (tiles + s.P - 1) / s.P * kTile;
    if (s.len < kTile) s.len = kTile;
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

// The launches of qd_ssm.hip that the backward uses: B and C in scalar order, and the walk
// that keeps the state before every tile of kTok tokens, [B][ceil(T / kTok)][N][D].
size_t row_floats(int B, int T, int G, int N);      // of b and c together
RowBuf row_buf(float *ws, int B, int T, int G, int N);
void launch_ssm_rows(int dtype, const SsmArgs &a, RowBuf rows, hipStream_t stream);
hipError_t launch_ssm_states(int dtype, const SsmArgs &a, Segments seg, SegBuf buf, RowBuf rows, float *keep,
                             hipStream_t stream);

}  // namespace qd
