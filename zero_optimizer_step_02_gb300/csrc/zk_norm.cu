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
#include "zk_tc.cuh"

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
// For rows too wide for the kernels below.  One CTA a row; the row is read
// three times, the last two from cache.
template <int DT>
__global__ void __launch_bounds__(256) ln_forward_any(const __grid_constant__ LnArgs a)
{
    using E = El<DT>;
    __shared__ float red[32];
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    pdl_wait();
    pdl_launch();
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
    pdl_wait();
    pdl_launch();
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
    pdl_wait();
    pdl_launch();
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

// ---------------------------------------------------------- wide-load kernels
// VEC consecutive elements: 16 bytes where bases, strides and the width are
// multiples of 16 bytes, else one element.  Held as they came from memory and
// widened at each use, so that a row costs half the registers in 16 bits
// (keep() makes the compiler forget the widened values it has).
template <int DT, int VEC>
struct Chunk;
template <int DT>
struct Chunk<DT, 8> {
    uint4 w;
    __device__ __forceinline__ void keep() { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p) { w = __ldcs(static_cast<const uint4*>(p)); }
    __device__ __forceinline__ void up(float (&v)[8]) const
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = Lp<DT>::lo(a[i]), v[2 * i + 1] = Lp<DT>::hi(a[i]);
    }
    __device__ static __forceinline__ void store(void* p, const float (&v)[8])
    {
        __stcs(static_cast<uint4*>(p), make_uint4(Lp<DT>::narrow2(v[0], v[1]), Lp<DT>::narrow2(v[2], v[3]),
                                                  Lp<DT>::narrow2(v[4], v[5]), Lp<DT>::narrow2(v[6], v[7])));
    }
};
template <>
struct Chunk<ZERO_FP32, 4> {
    float4 w;
    __device__ __forceinline__ void keep() {}
    __device__ __forceinline__ void zero() { w = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void load(const void* p) { w = __ldcs(static_cast<const float4*>(p)); }
    __device__ __forceinline__ void up(float (&v)[4]) const { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
    __device__ static __forceinline__ void store(void* p, const float (&v)[4])
    {
        __stcs(static_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <int DT>
struct Chunk<DT, 1> {
    typename El<DT>::T w;
    __device__ __forceinline__ void keep() {}
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const typename El<DT>::T*>(p); }
    __device__ __forceinline__ void up(float (&v)[1]) const { v[0] = El<DT>::up(w); }
    __device__ static __forceinline__ void store(void* p, const float (&v)[1])
    {
        *static_cast<typename El<DT>::T*>(p) = El<DT>::down(v[0]);
    }
};

// VEC weights from column c on, in whichever type they have
template <int VEC>
__device__ __forceinline__ void weights_at(const void* w, int dt, int c, float none, float (&v)[VEC])
{
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = none;
    } else if (VEC == 1) {
        v[0] = weight_at(w, dt, c);
    } else if (dt == ZERO_FP32) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + e);
            v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
        }
    } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(w) + c);
        uint32_t a[VEC / 2 > 0 ? VEC / 2 : 1];
        if (VEC == 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            a[0] = x.x, a[1] = x.y, a[VEC / 2 - 2] = x.z, a[VEC / 2 - 1] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            a[0] = x.x, a[VEC / 2 - 1] = x.y;
        }
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            v[2 * e] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::lo(a[e]) : Lp<ZERO_FP16>::lo(a[e]);
            v[2 * e + 1] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::hi(a[e]) : Lp<ZERO_FP16>::hi(a[e]);
        }
    }
}

// Forward, the row in registers: NCH chunks a lane, a warp (BLOCK false) or a
// whole CTA a row.  One read of x, one write of y.
template <int DT, int VEC, int NCH, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256, BLOCK ? 1 : 2) ln_forward_row(const __grid_constant__ LnArgs a)
{
    using T = typename El<DT>::T;
    __shared__ float red[32];
    pdl_wait();
    pdl_launch();
    const long long r = BLOCK ? blockIdx.x : blockIdx.x * static_cast<long long>(blockDim.x / 32) + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const int t = BLOCK ? threadIdx.x : threadIdx.x & 31, width = BLOCK ? blockDim.x : 32;
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    T* y = static_cast<T*>(a.out) + r * a.out_stride;
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    Chunk<DT, VEC> v[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (t + i * width) * VEC;
        if (c < a.cols)
            v[i].load(x + c);
        else
            v[i].zero();
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        float f[VEC];
        v[i].up(f);
        float p = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) p += f[e];
        s += p;
    }
    const float mean = (BLOCK ? block_sum(s, red) : warp_sum(s)) * inv_c;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        if ((t + i * width) * VEC >= a.cols) break;
        float f[VEC];
        v[i].keep();
        v[i].up(f);
        float p = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) p = fmaf(f[e] - mean, f[e] - mean, p);
        q += p;
    }
    const float rstd = 1.0f / sqrtf((BLOCK ? block_sum(q, red) : warp_sum(q)) * inv_c + a.eps);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (t + i * width) * VEC;
        if (c >= a.cols) break;
        float f[VEC], g[VEC], b[VEC];
        v[i].keep();
        v[i].up(f);
        weights_at<VEC>(a.gain, a.w_dtype, c, 1.0f, g);
        weights_at<VEC>(a.bias, a.w_dtype, c, 0.0f, b);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mean) * rstd, g[e], b[e]);
        Chunk<DT, VEC>::store(y + c, f);
    }
    if (t == 0) {
        if (a.mean_out != nullptr) a.mean_out[r] = mean;
        if (a.rstd_out != nullptr) a.rstd_out[r] = rstd;
    }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Backward: a persistent CTA of `groups` row groups of `warps` warps.  A thread
// keeps the same NCH * VEC columns for all its rows, so the column sums (and
// the gain) stay in its registers; the rows to come are on their way into a
// ring that each thread fills and empties alone (16-byte copies, DEPTH rows;
// without them the next row waits in registers).  One exchange between the
// warps of a group for the two row sums, double-buffered.
template <int DT, int VEC, int NCH, int DEPTH>
__global__ void __launch_bounds__(512) ln_backward_fused(const __grid_constant__ LnArgs a, int warps, int groups)
{
    using T = typename El<DT>::T;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[2][16][2];
    const int width = warps * 32;
    const int grp = threadIdx.x / width, t = threadIdx.x % width, lane = threadIdx.x & 31, wg = t >> 5;
    const long long step = static_cast<long long>(gridDim.x) * groups;
    const T* xb = static_cast<const T*>(a.x);
    const T* db = static_cast<const T*>(a.dy);
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    pdl_wait();
    pdl_launch();
    float gain[NCH][VEC], dg[NCH][VEC], dbias[NCH][VEC];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (t + i * width) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) gain[i][e] = 0.0f, dg[i][e] = 0.0f, dbias[i][e] = 0.0f;
        if (c < a.cols) weights_at<VEC>(a.gain, a.w_dtype, c, 1.0f, gain[i]);
    }
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;   // [DEPTH][2][NCH][blockDim.x]
    const int slot = 2 * NCH * blockDim.x;
    Chunk<DT, VEC> nx[NCH], nd[NCH];
    const long long r0 = static_cast<long long>(blockIdx.x) * groups + grp;
    auto fetch = [&](long long r, int s) {
        if (r < a.rows) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = (t + i * width) * VEC;
                if (c >= a.cols) break;
                if (DEPTH > 0) {
                    cp_async16(ring + s * slot + i * blockDim.x, xb + r * a.x_stride + c);
                    cp_async16(ring + s * slot + (NCH + i) * blockDim.x, db + r * a.dy_stride + c);
                } else {
                    nx[i].load(xb + r * a.x_stride + c);
                    nd[i].load(db + r * a.dy_stride + c);
                }
            }
        }
        if (DEPTH > 0) cp_async_commit();
    };
    if (DEPTH > 0) {
        for (int s = 0; s < DEPTH - 1; ++s) fetch(r0 + s * step, s);
    } else {
#pragma unroll
        for (int i = 0; i < NCH; ++i) nx[i].zero(), nd[i].zero();
        fetch(r0, 0);
    }
    int s = 0, buf = 0;
    float mean = 0.0f, rstd = 0.0f;
    if (r0 < a.rows) mean = a.mean[r0], rstd = a.rstd[r0];
    for (long long r = r0; r < a.rows; r += step) {
        Chunk<DT, VEC> cx[NCH], cd[NCH];
        float mean_n = 0.0f, rstd_n = 0.0f;
        if (r + step < a.rows) mean_n = a.mean[r + step], rstd_n = a.rstd[r + step];
        if (DEPTH > 0) {
            cp_async_wait<DEPTH - 2 >= 0 ? DEPTH - 2 : 0>();
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                cx[i].zero(), cd[i].zero();
                if ((t + i * width) * VEC < a.cols) {
                    *reinterpret_cast<uint4*>(&cx[i]) = ring[s * slot + i * blockDim.x];
                    *reinterpret_cast<uint4*>(&cd[i]) = ring[s * slot + (NCH + i) * blockDim.x];
                }
            }
            fetch(r + (DEPTH - 1) * step, s == 0 ? DEPTH - 1 : s - 1);
            s = s + 1 == DEPTH ? 0 : s + 1;
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) cx[i] = nx[i], cd[i] = nd[i];
            fetch(r + step, 0);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if ((t + i * width) * VEC >= a.cols) break;
            float x[VEC], d[VEC];
            cx[i].up(x);
            cd[i].up(d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xhat = (x[e] - mean) * rstd, h = d[e] * gain[i][e];
                dg[i][e] = fmaf(d[e], xhat, dg[i][e]);
                dbias[i][e] += d[e];
                s1 += h;
                s2 = fmaf(h, xhat, s2);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (warps > 1) {
            if (lane == 0) red[buf][threadIdx.x >> 5][0] = s1, red[buf][threadIdx.x >> 5][1] = s2;
            named_bar_sync(1 + grp, width);
            s1 = s2 = 0.0f;
            for (int w = 0; w < warps; ++w) s1 += red[buf][grp * warps + w][0], s2 += red[buf][grp * warps + w][1];
            buf ^= 1;
        }
        s1 *= inv_c;
        s2 *= inv_c;
        T* out = static_cast<T*>(a.out) + r * a.out_stride;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (t + i * width) * VEC;
            if (c >= a.cols) break;
            float x[VEC], d[VEC];
            cx[i].keep();
            cd[i].keep();
            cx[i].up(x);
            cd[i].up(d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = rstd * (fmaf(d[e], gain[i][e], -s1) - (x[e] - mean) * rstd * s2);
            Chunk<DT, VEC>::store(out + c, x);
        }
        mean = mean_n, rstd = rstd_n;
    }
    // the CTA's column sums: its row groups add up one after the other (the
    // ring's memory is free by then), then one row of partial sums leaves
    float* p = a.parts + static_cast<long long>(blockIdx.x) * 2 * a.cols;
    float* acc = reinterpret_cast<float*>(smem);
    if (groups > 1) {
        cp_async_wait<0>();
        __syncthreads();
        for (int g = groups - 1; g > 0; --g) {
            if (grp == g) {
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int k = (i * VEC + e) * 2 * width + t;
                        acc[k] = dg[i][e] + (g < groups - 1 ? acc[k] : 0.0f);
                        acc[k + width] = dbias[i][e] + (g < groups - 1 ? acc[k + width] : 0.0f);
                    }
            }
            __syncthreads();
        }
    }
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (t + i * width) * VEC;
            if (c >= a.cols) break;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = (i * VEC + e) * 2 * width + t;
                p[c + e] = dg[i][e] + (groups > 1 ? acc[k] : 0.0f);
                p[a.cols + c + e] = dbias[i][e] + (groups > 1 ? acc[k + width] : 0.0f);
            }
        }
    }
}

// The partial column sums, in a fixed order: 32 columns a CTA, sixteen slices
// of the parts side by side, fp64.
__global__ void __launch_bounds__(512) ln_backward_finish(const __grid_constant__ LnArgs a, int parts)
{
    __shared__ double red[16][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    double s = 0.0;
    if (i < 2 * a.cols) {
#pragma unroll 8
        for (int p = slice; p < parts; p += 16) s += static_cast<double>(a.parts[static_cast<long long>(p) * 2 * a.cols + i]);
    }
    red[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || i >= 2 * a.cols) return;
    const bool bias = i >= a.cols;
    void* out = bias ? a.dbias : a.dgain;
    if (out == nullptr) return;
    for (int k = 1; k < 16; ++k) s += red[k][lane];
    put_weight(out, a.w_dtype, bias ? i - a.cols : i, static_cast<float>(s));
}

// ------------------------------------------------------------------- host
int sms_of_device()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

bool wide(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int DT, int VEC, int NCH>
cudaError_t forward_row(const LnArgs& a, int sms, cudaStream_t st)
{
    // a warp a row; as few rows a CTA as spreads them over the SMs
    const long long per = (a.rows + sms - 1) / sms;
    const int warps = per < 8 ? static_cast<int>(per) : 8;
    return launch_after(ln_forward_row<DT, VEC, NCH, false>, dim3(static_cast<unsigned>((a.rows + warps - 1) / warps)),
                        dim3(32 * warps), 0, st, a);
}

template <int DT, int VEC, int NCH>
cudaError_t forward_block(const LnArgs& a, int chunks, cudaStream_t st)
{
    const int threads = ((chunks + NCH - 1) / NCH + 31) / 32 * 32;
    return launch_after(ln_forward_row<DT, VEC, NCH, true>, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0, st, a);
}

// A row stays in a warp's registers up to kWarpChunks chunks a lane (16 x 16
// bytes: 4096 columns in 16 bits; 64 single elements), in a CTA's up to four
// (16 single) a thread; wider rows are read again for each pass.
template <int DT, int VEC>
cudaError_t forward_vec(const LnArgs& a, int sms, cudaStream_t st, bool& done)
{
    done = true;
    const int chunks = (a.cols + VEC - 1) / VEC;
    if (a.rows < (1LL << 31)) {
        if constexpr (VEC > 1) {
            if (chunks <= 32) return forward_row<DT, VEC, 1>(a, sms, st);
            if (chunks <= 64) return forward_row<DT, VEC, 2>(a, sms, st);
            if (chunks <= 96) return forward_row<DT, VEC, 3>(a, sms, st);
            if (chunks <= 128) return forward_row<DT, VEC, 4>(a, sms, st);
            if (chunks <= 256) return forward_row<DT, VEC, 8>(a, sms, st);
            if (chunks <= 512) return forward_row<DT, VEC, 16>(a, sms, st);
            if (chunks <= 4096) return forward_block<DT, VEC, 4>(a, chunks, st);
        } else {
            if (chunks <= 256) return forward_row<DT, VEC, 8>(a, sms, st);
            if (chunks <= 1024) return forward_row<DT, VEC, 32>(a, sms, st);
            if (chunks <= 2048) return forward_row<DT, VEC, 64>(a, sms, st);
            if (chunks <= 16384) return forward_block<DT, VEC, 16>(a, chunks, st);
        }
    }
    done = false;
    return cudaSuccess;
}

template <int DT>
cudaError_t forward_of(const LnArgs& a, cudaStream_t st)
{
    constexpr int V = DT == ZERO_FP32 ? 4 : 8;
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    bool done;
    const bool vec = a.cols % V == 0 && a.x_stride % V == 0 && a.out_stride % V == 0 && wide(a.x) && wide(a.out) &&
                     wide(a.gain) && wide(a.bias);
    const cudaError_t e = vec ? forward_vec<DT, V>(a, sms, st, done) : forward_vec<DT, 1>(a, sms, st, done);
    if (done) return e;
    const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
    return launch_after(ln_forward_any<DT>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, a);
}

template <int DT, int VEC, int NCH, int DEPTH>
cudaError_t backward_fused(const LnArgs& a, int warps, int sms, cudaStream_t st, int& parts)
{
    // about 512 threads an SM in CTAs of up to 512 (256 where a row needs no
    // more); small problems in as many CTAs as they have row groups
    int groups = warps > 8 ? 1 : 8 / warps;
    long long spread = (a.rows + sms - 1) / sms;
    if (groups > spread) groups = static_cast<int>(spread);
    const int threads = 32 * warps * groups;
    long long grid = (a.rows + groups - 1) / groups;
    const long long most = static_cast<long long>(sms) * (threads <= 256 ? 2 : 1);
    if (grid > most) grid = most;
    if (grid > kLnMaxParts) grid = kLnMaxParts;
    parts = static_cast<int>(grid);
    size_t smem = static_cast<size_t>(DEPTH) * 2 * NCH * 16 * threads;
    const size_t sums = groups > 1 ? static_cast<size_t>(2) * NCH * VEC * 32 * warps * sizeof(float) : 0;
    if (smem < sums) smem = sums;
    const auto k = ln_backward_fused<DT, VEC, NCH, DEPTH>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_after(k, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, st, a, warps, groups);
}

template <int DT>
cudaError_t backward_of(const LnArgs& a, cudaStream_t st)
{
    constexpr int V = DT == ZERO_FP32 ? 4 : 8;
    constexpr int N = DT == ZERO_FP32 ? 4 : 2;    // chunks a thread when a row takes several warps: 16 columns
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    int parts = static_cast<int>(a.rows < kLnMaxParts ? a.rows : kLnMaxParts);
    if (a.rows > 0) {
        const bool vec = a.cols % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 && a.out_stride % V == 0 &&
                         wide(a.x) && wide(a.dy) && wide(a.out) && wide(a.gain);
        const int chunks = a.cols / V;
        cudaError_t e = cudaSuccess;
        if (vec && chunks <= 32) {
            e = backward_fused<DT, V, 1, 4>(a, 1, sms, st, parts);
        } else if (vec && chunks <= 64) {
            e = backward_fused<DT, V, 2, 4>(a, 1, sms, st, parts);
        } else if (vec && chunks <= 96) {
            e = backward_fused<DT, V, 3, 4>(a, 1, sms, st, parts);
        } else if (vec && chunks <= 512 * N) {
            e = backward_fused<DT, V, N, N == 4 ? 3 : 4>(a, (chunks + 32 * N - 1) / (32 * N), sms, st, parts);
        } else if (!vec && a.cols <= 16 * 32 * 8) {
            e = backward_fused<DT, 1, 8, 0>(a, (a.cols + 255) / 256, sms, st, parts);
        } else if (!vec && a.cols <= 16 * 32 * 16) {
            e = backward_fused<DT, 1, 16, 0>(a, (a.cols + 511) / 512, sms, st, parts);
        } else {
            const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
            e = launch_after(ln_backward_rows<DT>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, a);
            if (e == cudaSuccess) e = launch_after(ln_backward_cols<DT>, dim3((a.cols + 255) / 256, parts), dim3(256), 0, st, a);
        }
        if (e != cudaSuccess) return e;
    }
    if (a.dgain == nullptr && a.dbias == nullptr) return cudaSuccess;
    return launch_after(ln_backward_finish, dim3((2 * a.cols + 31) / 32), dim3(512), 0, st, a, parts);
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
