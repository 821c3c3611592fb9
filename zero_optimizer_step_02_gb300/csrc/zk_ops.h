// zk_ops.h -- host-side launch interface of the training operators beside the
// optimizer step (zk_norm.cu, zk_ortho.cu).
#pragma once

#include <cuda_runtime.h>

#include "zero.h"

namespace zk {

inline int dtype_bytes(int dt) { return dt == ZERO_FP32 ? 4 : 2; }

// ------------------------------------------------------------- layer norm
constexpr int kLnMaxParts = 304;   // partial weight-gradient rows kept in the workspace

struct LnArgs {
    const void* x;
    const void* dy;      // backward
    const void* gain;    // may be null (ones)
    const void* bias;    // forward; may be null
    const float* mean;   // backward
    const float* rstd;
    void* out;           // y or dx
    float* mean_out;     // forward; may be null
    float* rstd_out;
    void* dgain;         // backward; may be null
    void* dbias;
    float* parts;        // backward: [parts][2][cols] partial column sums
    float* rowsums;      // backward: [rows][2]
    long long rows;
    long long x_stride, dy_stride, out_stride;
    int cols;
    int dtype, w_dtype;
    float eps;
};

cudaError_t launch_ln_forward(const LnArgs& a, cudaStream_t st);
cudaError_t launch_ln_backward(const LnArgs& a, cudaStream_t st);

}  // namespace zk
