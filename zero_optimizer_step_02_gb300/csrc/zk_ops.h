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
    float* parts;        // backward: [parts][2][pitch] partial column sums
    int pitch;           // ln_pitch(cols)
    float* rowsums;      // backward: [rows][2]
    long long rows;
    long long x_stride, dy_stride, out_stride;
    int cols;
    int dtype, w_dtype;
    float eps;
};

// columns and what a row may begin with, in whole words
inline int ln_pitch(int cols) { return (cols + 7) / 8 * 8 + 8; }
// widths from which a row may be too wide for one CTA's registers (the row
// means then go through the workspace)
constexpr int kLnWide = 8176;
cudaError_t launch_ln_forward(const LnArgs& a, cudaStream_t st);
cudaError_t launch_ln_backward(const LnArgs& a, cudaStream_t st);

// ------------------------------------------- orthogonalised matrix updates
constexpr int kNsMaxSteps = 32;

// A batch of equal matrices and what becomes of them.
struct NsArgs {
    int rows, cols, batch;
    int steps;
    float coef[kNsMaxSteps][3];   // a, b, c of x <- a x + (b G + c G G) x, G the Gram matrix
    float eps;
    int products;                 // 1: fp16 operands; 3: pairs of fp16 (see zk_ortho.cu)
    // input: a matrix of `in_dtype`, or (Muon) the rank gradients
    const void* in;
    int in_dtype;
    long long in_ld, in_stride;
    // output
    void* out;
    int out_dtype;
    long long out_ld, out_stride;
    // Muon: out is null
    const void* const* ranks;     // host array
    int n_d;
    float divisor, mu;
    int nesterov;
    int loss_scaling, clipping;   // from the scalars block
    float* momentum;
    float* master;
    void* lp;
    int lp_dtype;
    float decay, step;
    long long flat_stride;
    void* ws;
    zero_dev_scalars* sc;
};

size_t ns_workspace_bytes(int rows, int cols, int batch, int products, bool muon);
cudaError_t launch_ns(const NsArgs& a, cudaStream_t st);
// how a call is cut up on a device of `sms` SMs (zero_matrix_plan)
void ns_plan(int rows, int cols, int batch, int products, int sms, zero_matrix_plan* out);
// one matrix product whose copies are never issued (tests the timeout path);
// scratch: 16 KB
cudaError_t launch_mm_starved(void* scratch, zero_dev_scalars* sc, unsigned long long timeout_ns, cudaStream_t st);

}  // namespace zk
