// zk_norm.cu -- layer norm, forward and backward with the weight gradients.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y = (x - mean) * rstd * gain + bias
//   h = dy * gain,  xhat = (x - mean) * rstd
//   dx = rstd * (h - mean_C(h) - xhat * mean_C(h * xhat))
//   dgain = sum over rows of dy * xhat,  dbias = sum over rows of dy
//
// Every sum is fp32 (the last stage of the column sums fp64); the results are
// rounded once, to the tensor's type.  The sum of squares is taken about the
// mean in a second pass over the row, so an offset in x costs no digits.
#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"

namespace zk {
namespace {

template <int DT>
struct El;
template <>
struct El<ZERO_BF16> {
    using T = uint16_t;
    __device__ static __forceinline__ float up(T v) { return Lp<ZERO_BF16>::widen(v); }
    __device__ static __forceinline__ T down(float v) { return Lp<ZERO_BF16>::narrow(v); }
};
template <>
struct El<ZERO_FP16> {
    using T = uint16_t;
    __device__ static __forceinline__ float up(T v) { return Lp<ZERO_FP16>::widen(v); }
    __device__ static __forceinline__ T down(float v) { return Lp<ZERO_FP16>::narrow(v); }
};
template <>
struct El<ZERO_FP32> {
    using T = float;
    __device__ static __forceinline__ float up(T v) { return v; }
    __device__ static __forceinline__ T down(float v) { return v; }
};

// a weight vector's element in whichever type it has
__device__ __forceinline__ float weight_at(const void* w, int dt, long long i)
{
    if (dt == ZERO_FP32) return static_cast<const float*>(w)[i];
    const uint16_t h = static_cast<const uint16_t*>(w)[i];
    return dt == ZERO_BF16 ? Lp<ZERO_BF16>::widen(h) : Lp<ZERO_FP16>::widen(h);
}
__device__ __forceinline__ void put_weight(void* w, int dt, long long i, float v)
{
    if (dt == ZERO_FP32)
        static_cast<float*>(w)[i] = v;
    else
        static_cast<uint16_t*>(w)[i] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::narrow(v) : Lp<ZERO_FP16>::narrow(v);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// sum over the block, the same value in every thread; red: 32 floats
__device__ __forceinline__ float block_sum(float v, float* red)
{
    v = warp_sum(v);
    const int w = threadIdx.x >> 5, n = (blockDim.x + 31) >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += red[i];
    return s;
}

// ------------------------------------------------------ any width, any stride
// One CTA a row; the row is read three times, the last two from cache.
template <int DT>
__global__ void __launch_bounds__(256) ln_forward_any(const __grid_constant__ LnArgs a)
{
    using E = El<DT>;
    __shared__ float red[32];
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const typename E::T* x = static_cast<const typename E::T*>(a.x) + r * a.x_stride;
        typename E::T* y = static_cast<typename E::T*>(a.out) + r * a.out_stride;
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += E::up(x[c]);
        const float mean = block_sum(s, red) * inv_c;
        float q = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = E::up(x[c]) - mean;
            q = fmaf(d, d, q);
        }
        const float rstd = 1.0f / sqrtf(block_sum(q, red) * inv_c + a.eps);
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float g = a.gain != nullptr ? weight_at(a.gain, a.w_dtype, c) : 1.0f;
            const float b = a.bias != nullptr ? weight_at(a.bias, a.w_dtype, c) : 0.0f;
            y[c] = E::down(fmaf((E::up(x[c]) - mean) * rstd, g, b));
        }
        if (threadIdx.x == 0) {
            if (a.mean_out != nullptr) a.mean_out[r] = mean;
            if (a.rstd_out != nullptr) a.rstd_out[r] = rstd;
        }
    }
}

// the two row means of the backward pass
template <int DT>
__global__ void __launch_bounds__(256) ln_backward_rows(const __grid_constant__ LnArgs a)
{
    using E = El<DT>;
    __shared__ float red[32];
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const typename E::T* x = static_cast<const typename E::T*>(a.x) + r * a.x_stride;
        const typename E::T* dy = static_cast<const typename E::T*>(a.dy) + r * a.dy_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float h = E::up(dy[c]) * (a.gain != nullptr ? weight_at(a.gain, a.w_dtype, c) : 1.0f);
            s1 += h;
            s2 = fmaf(h, (E::up(x[c]) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, red) * inv_c;
        s2 = block_sum(s2, red) * inv_c;
        if (threadIdx.x == 0) {
            a.rowsums[2 * r] = s1;
            a.rowsums[2 * r + 1] = s2;
        }
    }
}

// dx and the partial column sums: blockIdx.x takes 256 columns, blockIdx.y
// every gridDim.y-th row
template <int DT>
__global__ void __launch_bounds__(256) ln_backward_cols(const __grid_constant__ LnArgs a)
{
    using E = El<DT>;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    const float gain = a.gain != nullptr ? weight_at(a.gain, a.w_dtype, c) : 1.0f;
    float dg = 0.0f, db = 0.0f;
    for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float rstd = a.rstd[r];
        const float xhat = (E::up(static_cast<const typename E::T*>(a.x)[r * a.x_stride + c]) - a.mean[r]) * rstd;
        const float dy = E::up(static_cast<const typename E::T*>(a.dy)[r * a.dy_stride + c]);
        dg = fmaf(dy, xhat, dg);
        db += dy;
        const float dx = rstd * (dy * gain - a.rowsums[2 * r] - xhat * a.rowsums[2 * r + 1]);
        static_cast<typename E::T*>(a.out)[r * a.out_stride + c] = E::down(dx);
    }
    float* p = a.parts + static_cast<long long>(blockIdx.y) * 2 * a.cols;
    p[c] = dg;
    p[a.cols + c] = db;
}

// the partial column sums in order, one thread a column
__global__ void __launch_bounds__(128) ln_backward_finish(const __grid_constant__ LnArgs a, int parts)
{
    const int i = blockIdx.x * 128 + threadIdx.x;
    if (i >= 2 * a.cols) return;
    const bool bias = i >= a.cols;
    void* out = bias ? a.dbias : a.dgain;
    if (out == nullptr) return;
    double s = 0.0;
    for (int p = 0; p < parts; ++p) s += static_cast<double>(a.parts[static_cast<long long>(p) * 2 * a.cols + i]);
    put_weight(out, a.w_dtype, bias ? i - a.cols : i, static_cast<float>(s));
}

template <int DT>
cudaError_t forward_of(const LnArgs& a, cudaStream_t st)
{
    const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
    ln_forward_any<DT><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <int DT>
cudaError_t backward_of(const LnArgs& a, cudaStream_t st)
{
    const int parts = static_cast<int>(a.rows < kLnMaxParts ? a.rows : kLnMaxParts);
    if (a.rows > 0) {
        const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
        ln_backward_rows<DT><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
        count_launch();
        ln_backward_cols<DT><<<dim3((a.cols + 255) / 256, parts), 256, 0, st>>>(a);
        count_launch();
    }
    if (a.dgain != nullptr || a.dbias != nullptr) {
        ln_backward_finish<<<(2 * a.cols + 127) / 128, 128, 0, st>>>(a, parts);
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ln_forward(const LnArgs& a, cudaStream_t st)
{
    if (a.rows == 0) return cudaSuccess;
    if (a.dtype == ZERO_FP32) return forward_of<ZERO_FP32>(a, st);
    return a.dtype == ZERO_BF16 ? forward_of<ZERO_BF16>(a, st) : forward_of<ZERO_FP16>(a, st);
}

cudaError_t launch_ln_backward(const LnArgs& a, cudaStream_t st)
{
    if (a.dtype == ZERO_FP32) return backward_of<ZERO_FP32>(a, st);
    return a.dtype == ZERO_BF16 ? backward_of<ZERO_BF16>(a, st) : backward_of<ZERO_FP16>(a, st);
}

}  // namespace zk
