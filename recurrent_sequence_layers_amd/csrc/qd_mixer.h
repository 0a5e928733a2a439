// Launch interface of the operators around the recurrence (short convolution, selective
// scan, group norm), and the device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qd_device.h"

namespace qd {

// ---------------------------------------------------------------- short causal convolution
struct ConvArgs {
    const void *x;                  // [B][T][D] elements
    const float *w, *bias;          // [D][W]; [D] or null
    const void *S0;                 // [B][W-1][D] elements or null
    const int *lens;                // [B] or null
    void *y;                        // [B][T][D]
    void *S_T;                      // [B][W-1][D] or null
    int B, T, D, W;
    bool silu;
    int TL;                         // tokens per thread
};
struct ConvBwdArgs {
    const void *x;
    const float *w, *bias;
    const void *S0;
    const int *lens;                // [B] or null
    const void *dy, *dS_T;
    void *dx, *dS0;                 // dS0 null: not written
    float *dw, *dbias;              // dbias null: not written
    float *part;                    // workspace [R][W + 1][D]
    int B, T, D, W;
    bool silu;
    int TL, NX, R;                  // tokens per thread, channel vectors per block (power of two), partial rows
};
// *_fits: the sizes stay within the kernels' 32-bit launch and row counts.
bool conv_fits(int B, int T, int D);
hipError_t launch_conv_fwd(int dtype, const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_step(int dtype, const ConvArgs &a, hipStream_t stream);   // T = 1, S0 == S_T in place
size_t conv_bwd_workspace(int B, int T, int D, int W);
hipError_t launch_conv_bwd(int dtype, const ConvBwdArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- selective scan
struct SsmArgs {
    const void *u, *dt, *Bm, *Cm;   // [B][T][D], [B][T][D], [B][T][G][N], [B][T][G][N]
    const float *A, *Dskip, *dt_bias; // [D][N]; [D] or null; [D] or null
    const void *z;                  // [B][T][D] or null
    const float *S0;                // [B][D][N] or null
    const int *lens;                // [B] or null
    void *o;                        // [B][T][D]
    float *S_T;                     // [B][D][N] or null
    int B, T, D, G, N;
    bool softplus;
};
struct SsmBwdArgs {
    const void *u, *dt, *Bm, *Cm;
    const float *A, *Dskip, *dt_bias;
    const void *z;
    const float *S0;
    const int *lens;                // [B] or null
    const void *d_o;
    const float *dS_T;              // [B][D][N] or null
    void *du, *ddt, *dB, *dC, *dz;  // dz null when z is null
    float *dA, *dD, *ddt_bias, *dS0; // all but dA may be null
    int B, T, D, G, N;
    bool softplus;
};
bool ssm_supported(int dtype, int N);
bool ssm_fits(int B, int T, int D, int G, int N);
size_t ssm_fwd_workspace(int B, int T, int D, int G, int N);
hipError_t launch_ssm_fwd(int dtype, const SsmArgs &a, void *ws, hipStream_t stream);
hipError_t launch_ssm_step(int dtype, const SsmArgs &a, hipStream_t stream);      // T = 1, S0 == S_T in place
size_t ssm_bwd_workspace(int B, int T, int D, int G, int N);
hipError_t launch_ssm_bwd(int dtype, const SsmBwdArgs &a, void *ws, hipStream_t stream);

// ---------------------------------------------------------------- group norm
struct NormArgs {
    const void *x;                  // [N][L][C]
    const float *w, *bias;          // [C] or null (1, 0)
    const void *gate;               // [N][L][C] or null
    void *y;
    float *stats;                   // [N][G][2] mean, 1/std; may be null in the forward
    const void *dy;                 // backward only
    void *dx, *dgate;               // backward only; dgate null when gate is null
    float *dw, *dbias;              // backward only; may be null
    int N, L, C, G;
    float eps;
    bool silu;
};
bool norm_fits(int dtype, int N, int L, int C, int G);
size_t norm_fwd_workspace(int dtype, int N, int L, int C, int G);
hipError_t launch_norm_fwd(int dtype, const NormArgs &a, void *ws, hipStream_t stream);
size_t norm_bwd_workspace(int dtype, int N, int L, int C, int G);
hipError_t launch_norm_bwd(int dtype, const NormArgs &a, void *ws, hipStream_t stream);
hipError_t launch_norm_zero(float *dw, float *dbias, int C, hipStream_t stream);   // both may be null

// ---------------------------------------------------------------- device helpers
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// 1 / (1 + exp(-x)); exp(-x) may overflow to infinity, which gives 0.
__device__ __forceinline__ float sigmoidf(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}
__device__ __forceinline__ float siluf(float x) { return x * sigmoidf(x); }
// d/dx silu(x) = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ float dsiluf(float x) {
    const float s = sigmoidf(x);
    return s * fmaf(x, 1.f - s, 1.f);
}

// log(1 + exp(x)).  With e = exp(x) and r = fl(1 + e), log(1 + e) = log(r) + (e - (r - 1)) / r to
// rounding accuracy also where e is far below 1: the second term is what the sum r lost.
// The exponent's rounding, amplified by its size in a plain exp2(x log2 e), is put back as
// a first-order factor.  Above 20 the value is x to fp32 accuracy (exp(-20) = 2e-9); a NaN
// takes that branch too.  No branches: they would stop the tokens of a tile from overlapping.
struct Softplus {
    float value, slope;              // slope: the derivative, sigmoid(x) = e / (1 + e)
};
__device__ __forceinline__ Softplus softplus_grad(float x) {
    const float xc = fmaxf(x, -126.f);
    const float p = xc * kLog2e;
    const float q = fmaf(xc, 1.925963033500e-8f, fmaf(xc, kLog2e, -p));
    const float e = __builtin_amdgcn_exp2f(p) * fmaf(q, kLn2, 1.f);
    const float r = 1.f + e;
    const float inv = __builtin_amdgcn_rcpf(r);
    const float small = fmaf(__builtin_amdgcn_logf(r), kLn2, (e - (r - 1.f)) * inv);
    return Softplus{x <= 20.f ? small : x, x > 20.f ? 1.f : e * inv};
}
__device__ __forceinline__ float softplusf(float x) { return softplus_grad(x).value; }

// V consecutive elements as floats; V elements are 16 or 8 bytes (aligned to that) or one.
template <class P, int V>
__device__ __forceinline__ void load_vec(const typename P::R *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = P::to_f32(p[0]);
    } else {
        constexpr int W = V * P::kBytes / 4;
        static_assert(W == 4 || W == 2, "16 or 8 bytes");
        uint32_t q[W];
        if constexpr (W == 4) *reinterpret_cast<uint4 *>(q) = *reinterpret_cast<const uint4 *>(p);
        else *reinterpret_cast<uint2 *>(q) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (P::kBytes == 2) {
                v[2 * i] = __uint_as_float(q[i] << 16);
                v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(q[i]);
            }
        }
    }
}
// AROUND: past the caches, for an output that would push out what is still to be read.
template <class P, int V, bool AROUND = false>
__device__ __forceinline__ void store_vec(typename P::R *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        p[0] = P::from_f32(v[0]);
    } else {
        constexpr int W = V * P::kBytes / 4;
        uint32_t q[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (P::kBytes == 2)
                q[i] = static_cast<uint32_t>(P::from_f32(v[2 * i])) | (static_cast<uint32_t>(P::from_f32(v[2 * i + 1])) << 16);
            else
                q[i] = __float_as_uint(v[i]);
        }
        typedef __attribute__((ext_vector_type(W))) uint32_t vec;
        vec w;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = q[i];
        if constexpr (AROUND) __builtin_nontemporal_store(w, reinterpret_cast<vec *>(p));
        else *reinterpret_cast<vec *>(p) = w;
    }
}

// Sum over aligned groups of `lanes` (a power of two up to 64) lanes; every lane of a group
// gets its sum.  DPP moves up to 16 lanes; across the 16-lane rows, through LDS hardware
// permutes.
__device__ __forceinline__ float group_sum(float x, int lanes) {
    if (lanes > 1) x += dpp_src<0xB1, 0xf>(x);    // quad_perm 1,0,3,2
    if (lanes > 2) x += dpp_src<0x4E, 0xf>(x);    // quad_perm 2,3,0,1
    if (lanes > 4) x += dpp_src<0x141, 0xf>(x);   // row_half_mirror
    if (lanes > 8) x += dpp_src<0x140, 0xf>(x);   // row_mirror
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

// Column sums of a [rows][cols] fp32 matrix of partial results, always in the same order:
// 64 columns a block, 16 threads a column taking every 16th row, four rows in flight, then
// the 16 sums through LDS.  The row loop's sum is kept in four parts, so no addend meets a
// sum of more than rows / 64 others.
constexpr int kColThreads = 1024, kColLanes = 16;
typedef float ColShared[kColLanes][64];
template <class Store>
__device__ __forceinline__ void column_sum_block(const float *__restrict__ m, int rows, long long cols, long long block,
                                                 Store store, ColShared &s) {
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
    const long long c = block * 64 + lane;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < cols) {
        const float *p = m + c;
        int r = part;
        for (; r + 3 * kColLanes < rows; r += 4 * kColLanes) {
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += p[static_cast<size_t>(r + k * kColLanes) * cols];
        }
        for (; r < rows; r += kColLanes) acc[0] += p[static_cast<size_t>(r) * cols];
    }
    s[part][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    if (part == 0 && c < cols) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kColLanes; ++k) t += s[k][lane];
        store(c, t);
    }
}
template <class Store>
__global__ __launch_bounds__(kColThreads) void column_sum_kernel(const float *__restrict__ m, int rows, long long cols,
                                                                 Store store) {
    __shared__ ColShared s;
    for (long long block = blockIdx.x; block * 64 < cols; block += gridDim.x) {
        column_sum_block(m, rows, cols, block, store, s);
        __syncthreads();                         // s is written again
    }
}
// A launch has fewer than 2^32 threads; one of more is cut short without an error.
constexpr long long kColBlocks = 1LL << 21;
template <class Store>
void column_sum(const float *m, int rows, long long cols, Store store, hipStream_t stream) {
    const long long blocks = (cols + 63) / 64;
    hipLaunchKernelGGL((column_sum_kernel<Store>), dim3(static_cast<unsigned>(blocks < kColBlocks ? blocks : kColBlocks)),
                       dim3(kColThreads), 0, stream, m, rows, cols, store);
}

}  // namespace qd
