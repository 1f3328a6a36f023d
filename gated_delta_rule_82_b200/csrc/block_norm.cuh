// block_norm.cuh -- arguments of the fused block norms (block_norm.cu has the formulas).
#pragma once

#include "common.cuh"

namespace ckda {

constexpr int kBlockNormMaxD = 8192;     // 1024 threads of 8 channels

struct BlockNormArgs {
    const void *y, *gate, *x;            // [rows][D]; gate and x nullable
    const float *w_post, *w_pre, *r;     // [W], [D], [D]; nullable (ones)
    void *h, *n;                         // [rows][D]; n nullable (no second norm)
    long long rows;
    int D, W;                            // W: group of the first norm (0: none, D: the row)
    int act;                             // 1 sigmoid, 2 silu (with a gate)
    float scale, eps;
};

struct BlockNormGrads {
    const void *dh, *dn;                 // nullable (zero)
    void *dx, *dy, *dgate;               // dx nullable
    float *dw_post, *dw_pre, *dr;        // nullable
    float* partial;
};

int block_norm_bwd_grid(long long rows, int D);
// floats of scratch for the CTAs' sums of the three weight gradients
size_t block_norm_bwd_partial_floats(long long rows, int D, int W);
cudaError_t launch_block_norm(const BlockNormArgs& p, ckda_dtype dtype, cudaStream_t s);
cudaError_t launch_block_norm_bwd(const BlockNormArgs& p, const BlockNormGrads& g,
                                  ckda_dtype dtype, cudaStream_t s);

}  // namespace ckda
