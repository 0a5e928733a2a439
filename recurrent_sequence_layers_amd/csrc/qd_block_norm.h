// Launch interface of the RMS norms after and before a block with its gate, scale and residual sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace qd {

struct BlockNormArgs {
    const void *y, *x, *gate;        // [N][C]; x null: zeros; gate null: no factor
    const float *post, *scale, *pre; // [C] or null (no norm; 1; no norm)
    void *h, *n;                     // [N][C]; n null when pre is null
    float *stats;                    // [N][2] or null in the forward
    const void *dh, *dn;             // backward: [N][C], each may be null (zero)
    void *dx, *dy, *dgate;           // backward; dx may be null
    float *dpost, *dscale, *dpre;    // backward: [C] or null
    float *part;                     // backward: [rows][3][C] partial sums
    int N, C;
    float eps;
    int act;                         // of the gate: 0 itself, 1 sigmoid, 2 silu
    int LG, V, K;                    // lanes a row, elements a vector, vectors a lane; K == 0: the looping form
    int grid;
};

bool block_norm_fits(int dtype, int N, int C);
hipError_t launch_block_norm_fwd(int dtype, BlockNormArgs a, hipStream_t stream);
size_t block_norm_bwd_workspace(int dtype, int N, int C, bool sums);
hipError_t launch_block_norm_bwd(int dtype, BlockNormArgs a, void *ws, hipStream_t stream);

}  // namespace qd
