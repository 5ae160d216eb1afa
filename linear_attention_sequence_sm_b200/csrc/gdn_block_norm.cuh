// gdn_block_norm.cuh -- the block norms' arguments as the kernels see them.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

struct BlockNormArgs {
    int64_t rows;
    int32_t width;
    uint32_t flags;
    const void *x, *residual, *gate;
    const float *post_weight, *scale, *pre_weight;
    float eps, residual_scale, branch_scale;
    void *h, *y;                                  // forward
    const void *d_h, *d_y;                        // backward
    void *dx, *d_residual, *d_gate;
    float *d_post_weight, *d_scale, *d_pre_weight;
    float *partial;                               // [lines][3][width]
};

// Lines of column sums the backward keeps (its workspace: 12 * lines * width bytes).
int block_norm_lines(int64_t rows, int32_t width);
constexpr int kBlockNormMaxWidth = 16384;

cudaError_t launch_block_norm_forward(const BlockNormArgs &a, int32_t dtype, int32_t residual_dtype,
                                      cudaStream_t stream);
cudaError_t launch_block_norm_backward(const BlockNormArgs &a, int32_t dtype, int32_t residual_dtype,
                                       cudaStream_t stream);

}  // namespace gdn
