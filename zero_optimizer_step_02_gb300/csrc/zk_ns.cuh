// zk_ns.cuh -- what the two forms of the Newton-Schulz iteration share: the
// scaling, element types, the rank mean and momentum of a Muon step.
#pragma once

#include <cuda_fp16.h>

#include "zk_common.cuh"
#include "zk_ops.h"
#include "zk_tc.cuh"

namespace zk {

constexpr float kScale = 4096.0f;
constexpr float kInvScale = 1.0f / 4096.0f;

__device__ __forceinline__ float2 half2_up(uint32_t w)
{
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
}

__device__ __forceinline__ uint16_t narrow16(int dt, float v)
{
    return dt == ZERO_BF16 ? Lp<ZERO_BF16>::narrow(v) : Lp<ZERO_FP16>::narrow(v);
}
__device__ __forceinline__ uint32_t narrow16x2(int dt, float v, float w)
{
    return dt == ZERO_BF16 ? Lp<ZERO_BF16>::narrow2(v, w) : Lp<ZERO_FP16>::narrow2(v, w);
}

// eight consecutive values of a row of `dt`; n: how many of them exist
__device__ __forceinline__ void put_row8(void* base, int dt, long long i, const float* v, int n, bool vec)
{
    if (dt == ZERO_FP32) {
        float* p = static_cast<float*>(base) + i;
        if (vec && n >= 8) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = v[e];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if (vec && n >= 8) {
            *reinterpret_cast<uint4*>(p) = make_uint4(narrow16x2(dt, v[0], v[1]), narrow16x2(dt, v[2], v[3]),
                                                      narrow16x2(dt, v[4], v[5]), narrow16x2(dt, v[6], v[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = narrow16(dt, v[e]);
        }
    }
}

// eight consecutive elements from column 8 * ch of a row, zeros past its end
__device__ __forceinline__ void load_row8(const void* in, int dtype, bool vec, long long row_at, int cols, int ch, float (&v)[8])
{
    const long long i = row_at + 8 * ch;
    const int n = cols - 8 * ch;
    if (dtype == ZERO_FP32) {
        const float* p = static_cast<const float*>(in) + i;
        if (vec && n >= 8) {
            const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
        }
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(in) + i;
    uint32_t w[4];
    if (vec && n >= 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (2 * e < n ? p[2 * e] : 0u) | ((2 * e + 1 < n ? static_cast<uint32_t>(p[2 * e + 1]) : 0u) << 16);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = dtype == ZERO_BF16 ? Lp<ZERO_BF16>::lo(w[e]) : Lp<ZERO_FP16>::lo(w[e]);
        v[2 * e + 1] = dtype == ZERO_BF16 ? Lp<ZERO_BF16>::hi(w[e]) : Lp<ZERO_FP16>::hi(w[e]);
    }
}

// A sum of squares in fp32, whatever the values' size: eight squares at a time
// go to one of three sums, as they are (compensated), times 2^-180 if they pass
// 2^90, times 2^180 if they are under 2^-90.  No sum over a matrix (2^28 eights
// at most) passes 2^118 then, and no square that counts falls under fp32's
// normal range: 2^-149 squared is 2^-118 in `tiny`, and what a square loses to
// subnormals in `sum` is under 2^-50 of it.  NaN and infinity go to `big`.
// (fp64 would cost more than all else here: it runs at a small fraction of
// fp32's rate.)
constexpr float kTo90 = 1.2379400392853803e27f;   // 2^90
struct SquareSum {
    float sum = 0.0f, lost = 0.0f, big = 0.0f, tiny = 0.0f;
    __device__ __forceinline__ void add8(const float (&v)[8])
    {
        float q = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
        if (q >= 1.0f / kTo90 && q <= kTo90) {
            const float a = fmaxf(sum, q), b = fminf(sum, q), t = a + b;
            lost += b - (t - a);
            sum = t;
            return;
        }
        const bool small = q < kTo90;
        const float f = small ? kTo90 : 1.0f / kTo90;
        q = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[e] * f, v[e] * f, q);
        if (small)
            tiny += q;
        else
            big += q;
    }
    // {sum, big, tiny, 0}
    __device__ __forceinline__ float4 value() const { return make_float4(sum + lost, big, tiny, 0.0f); }
};
__device__ __forceinline__ void add_sums(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z; }

// sums over a block, in thread 0; red: a float4 for each warp
__device__ __forceinline__ float4 block_sums(float4 v, float4* red)
{
    const auto warp_sums = [](float4& x) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add_sums(x, make_float4(__shfl_xor_sync(0xFFFFFFFFu, x.x, o), __shfl_xor_sync(0xFFFFFFFFu, x.y, o),
                                    __shfl_xor_sync(0xFFFFFFFFu, x.z, o), 0.0f));
    };
    warp_sums(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        warp_sums(v);
    }
    return v;
}

// kScale / (|g| + eps) from the sums of squares (thread 0's), in every thread; a
// NaN or an infinity in g makes it NaN.  eps >= 1e-30 keeps it finite.
__device__ __forceinline__ float block_scale(float4 sums, float eps, float* shared)
{
    if (threadIdx.x == 0) {
        constexpr float kDown = 1.0f / kTo90;
        float f;
        if (sums.y != 0.0f) {
            // all of it times 2^-90; what is in `tiny` is nothing beside it
            const float s = sums.y + sums.x * kDown * kDown;
            f = is_finite_f32(s) ? kScale * kDown / (sqrtf(s) + eps * kDown) : s - s;
        } else if (sums.x != 0.0f) {
            f = kScale / (sqrtf(sums.x + sums.z * kDown * kDown) + eps);
        } else {
            f = kScale / (sqrtf(sums.z) * kDown + eps);
        }
        *shared = f;
    }
    __syncthreads();
    return *shared;
}

struct MuonArgs {
    const void* rank[ZERO_MAX_RANKS];
    int n_d, dtype, nesterov;
    int loss_scaling, clipping;  // the divisor's scale and the coefficient are the scalars block's
    zero_dev_scalars* sc;
    float divisor, mu;
    float* momentum;
    float* u;
    long long stride, u_stride;
    uint32_t elems;              // of one matrix
    float4* parts;
    unsigned* counters;
    int n_counters;
};

// What the rank sums are divided and multiplied by (without clipping: 1, exact).
struct MuonMean {
    float divisor, coef;
    __device__ __forceinline__ explicit MuonMean(const MuonArgs& a)
    {
        divisor = a.loss_scaling ? __fmul_rn(static_cast<float>(a.n_d), a.sc->loss_scale) : a.divisor;
        coef = a.clipping ? a.sc->clip_coef : 1.0f;
    }
    __device__ __forceinline__ float of(float sum) const { return __fmul_rn(__fdiv_rn(sum, divisor), coef); }
};

// whether this step is one to skip (set by muon_check, or before the call)
__device__ __forceinline__ bool muon_skips(const MuonArgs& a)
{
    return a.loss_scaling && *reinterpret_cast<volatile int*>(&a.sc->nonfinite) != 0;
}

// the ranks' sums (rank order, fp32) of elements `at` .. of which n <= 8 exist
__device__ __forceinline__ void rank_sums8(const MuonArgs& a, long long at, int n, float (&g)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0.0f;
    if (n == 8) {
#pragma unroll 4
        for (int q = 0; q < a.n_d; ++q) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.rank[q]) + at);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[2 * e] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::lo(w[e]) : Lp<ZERO_FP16>::lo(w[e]);
                g[2 * e + 1] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::hi(w[e]) : Lp<ZERO_FP16>::hi(w[e]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e >= n) continue;
            for (int q = 0; q < a.n_d; ++q) {
                const uint16_t h = static_cast<const uint16_t*>(a.rank[q])[at + e];
                g[e] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::widen(h) : Lp<ZERO_FP16>::widen(h);
            }
        }
    }
}

// Momentum and the update direction u of elements 8 i .. of matrix b:
// m <- mu m + g, u = g + mu m (Nesterov) or m; zeros past the matrix.
__device__ __forceinline__ void muon_direction8(const MuonArgs& a, const MuonMean& mean_of, int b, uint32_t i, float (&u)[8])
{
    const int n = a.elems - 8 * i < 8 ? static_cast<int>(a.elems - 8 * i) : 8;
    const long long at = b * a.stride + 8ll * i;
    float g[8], m[8];
    float* mp = a.momentum + at;
    if (n == 8) {
        const float4 x = *reinterpret_cast<const float4*>(mp), y = *reinterpret_cast<const float4*>(mp + 4);
        m[0] = x.x, m[1] = x.y, m[2] = x.z, m[3] = x.w, m[4] = y.x, m[5] = y.y, m[6] = y.z, m[7] = y.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = e < n ? mp[e] : 0.0f;
    }
    rank_sums8(a, at, n, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float mean = mean_of.of(g[e]);
        m[e] = __fadd_rn(__fmul_rn(a.mu, m[e]), mean);
        u[e] = e >= n ? 0.0f : a.nesterov ? __fadd_rn(mean, __fmul_rn(a.mu, m[e])) : m[e];
    }
    put_row8(a.momentum, ZERO_FP32, at, m, n, true);
    put_row8(a.u, ZERO_FP32, b * a.u_stride + 8ll * i, u, 8, true);
}

// w <- w * (1 - lr wd) - step * o for n of eight consecutive weights, and
// their 16-bit cast (lp may be null)
__device__ __forceinline__ void put_weights8(float* master, void* lp, int lp_dtype, long long at, float (&o)[8], int n, bool vec,
                                             float decay, float step)
{
    float w[8];
    if (vec && n >= 8) {
        const float4 p = *reinterpret_cast<const float4*>(master + at), q = *reinterpret_cast<const float4*>(master + at + 4);
        w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w, w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < n ? master[at + e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(-step, o[e], w[e] * decay);
    put_row8(master, ZERO_FP32, at, o, n, vec);
    if (lp != nullptr) put_row8(lp, lp_dtype, at, o, n, vec);
}

// whether rows of dt from p on may be read and written 16 bytes at a time
inline bool wide_rows(const void* p, int dt, long long ld, long long stride)
{
    const int v = 16 / dtype_bytes(dt);
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % v == 0 && stride % v == 0;
}

// the form for matrices that one SM holds (zk_ortho_small.cu); mu: the Muon
// step's, or null
bool small_ns_fits(int rows, int cols, int products);
cudaError_t launch_small_ns(const NsArgs& a, const MuonArgs* mu, cudaStream_t st);

}  // namespace zk
