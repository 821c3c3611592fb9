// zk_ortho_small.cu -- the Newton-Schulz iteration for matrices that one SM
// holds: a short side of up to 128, a long side of up to 256, three products.
//
// Every operand stays in shared memory for the whole iteration and every sum
// in tensor memory, so a step costs its MMAs, two tensor-memory reads and
// three block barriers, not three trips through L2.  One CTA a matrix, one
// launch a call.  96 x 160 takes 37 us (the general form 100), 140 matrices of
// 128 x 256 58 us side by side.  Its floor is nothing (under 0.1 us of work at
// the whole chip's rate); what it takes is the latency of fifteen dependent
// products: about 2.4 us each for the barrier, a short chain of MMAs, the sums
// out of tensor memory and the pairs back into shared memory (by counters: issue
// slots 39% busy, tensor cores 34%, waits for tensor memory on top of the
// stalls).  Larger matrices do not fit: both planes of x, twice 128 x 256, and
// of one square matrix are 192 KB.
//
// Shared memory: planes of panels, a panel 128 lines of 64 fp16 values (128
// bytes, 128-byte swizzle).  Line i of panel p of x holds x[i][64 p ..], the
// short side first (a tall matrix is transposed on its way in and out).  That
// one image is K-major for G = x x^T and MN-major for P x.  G and P = b G +
// c G G share one square image: P replaces G once its product is complete, as
// the new x replaces the old.  Lines and columns past the matrix are zeros and
// stay zeros.
#include <cstring>

#include "zk_launch.h"
#include "zk_ns.cuh"
#include "zk_ops.h"
#include "zk_tc.cuh"

namespace zk {
namespace {

constexpr int kSmallThreads = 512;
constexpr int kLines = 128;
constexpr int kPanelBytes = kLines * 128;
constexpr int kMaxPanels = 4;
constexpr int kSquarePanels = 2;
// tensor memory columns: the large product's sums, the small products' sums
constexpr int kTmemCols = 512, kTmemSmall = 256;

struct SmallNsArgs {
    int rows, cols, m, n, wide, panels;
    int steps;
    float coef[kNsMaxSteps][3];
    float eps;
    const void* in;
    int in_dtype, in_vec;
    long long in_ld, in_stride;
    void* out;                   // null: Muon
    int out_dtype, out_vec;
    long long out_ld, out_stride;
    float* master;
    void* lp;
    float decay, step;
    zero_dev_scalars* sc;
    unsigned long long timeout_ns;
};

// byte of element (i, j) in a plane
__device__ __forceinline__ int at_of(int i, int j)
{
    return j / 64 * kPanelBytes + i * 128 + ((j % 64 / 8) ^ (i & 7)) * 16 + j % 8 * 2;
}

__device__ __forceinline__ void split_half(float v, __half& hi, __half& lo)
{
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

// eight values to both planes (16 bytes each); `lo` bytes further on
__device__ __forceinline__ void put_pair8(unsigned char* p, int lo, const float (&v)[8])
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2 x = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
        const float2 f = __half22float2(x);
        const __half2 y = __floats2half2_rn(v[2 * e] - f.x, v[2 * e + 1] - f.y);
        h[e] = *reinterpret_cast<const uint32_t*>(&x);
        l[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p + lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// v = alpha * v + beta * (hi + lo)
__device__ __forceinline__ void combine8(const unsigned char* p, int lo, float (&v)[8], float alpha, float beta)
{
    const uint4 h = *reinterpret_cast<const uint4*>(p), l = *reinterpret_cast<const uint4*>(p + lo);
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = half2_up(hw[e]), y = half2_up(lw[e]);
        v[2 * e] = fmaf(beta, x.x + y.x, alpha * v[2 * e]);
        v[2 * e + 1] = fmaf(beta, x.y + y.y, alpha * v[2 * e + 1]);
    }
}

// The MMAs of one phase: 128 x n sums over `steps` slices of sixteen values of
// depth.  a: the K-major image's hi plane, b: the other operand's; `mn`: b is
// read MN-major.  lo planes follow at the given distances.
__device__ __forceinline__ void issue(uint32_t tmem, uint32_t a, int a_lo, uint32_t b, int b_lo, int n, int steps, bool mn)
{
    const uint32_t idesc = instr_desc(128, n, false, mn);
    for (int k = 0; k < steps; ++k) {
        const uint32_t along = k / 4 * kPanelBytes + k % 4 * 32;
        const uint32_t da = smem_desc_lo(a + along, kPanelBytes);
        const uint32_t db = smem_desc_lo(b + (mn ? k * 2048u : along), kPanelBytes);
        const uint32_t la = static_cast<uint32_t>(a_lo) >> 4, lb = static_cast<uint32_t>(b_lo) >> 4;
        mma_f16<1>(tmem + kTmemSmall, da + la, db, idesc, k > 0);
        mma_f16<1>(tmem + kTmemSmall, da, db + lb, idesc, 1);
        mma_f16<1>(tmem, da, db, idesc, k > 0);
    }
}

template <bool MUON>
__device__ __forceinline__ void ns_small_body(const SmallNsArgs& a, const MuonArgs* mu)
{
    if (MUON && mu->loss_scaling) {
        pdl_wait();
        if (muon_skips(*mu)) return;   // the same for every thread
    }
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t bar, drain;
    __shared__ uint32_t tmem_base;
    __shared__ float4 red[kSmallThreads / 32];
    __shared__ float shared_scale;
    unsigned char* x = smem_raw + (1024 - (smem_u32(smem_raw) & 1023u)) % 1024;
    const int x_lo = a.panels * kPanelBytes, g_lo = kSquarePanels * kPanelBytes;
    unsigned char* g = x + 2 * x_lo;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, b = blockIdx.x;

    if (t == 0) {
        mbar_init(&bar, 1);
        mbar_init(&drain, 1);
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<1>(&tmem_base, kTmemCols);
    for (int i = t; i < (2 * x_lo + 2 * g_lo) / 16; i += kSmallThreads) reinterpret_cast<uint4*>(x)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_launch();

    // |g|, then x = g / (|g| + eps), scaled
    const int chunks = (a.cols + 7) / 8, total = a.rows * chunks;
    SquareSum q;
    if (MUON) {
        const MuonMean mean(*mu);
        for (uint32_t i = t; 8 * i < mu->elems; i += kSmallThreads) {
            float u[8];
            muon_direction8(*mu, mean, b, i, u);
            q.add8(u);
        }
    } else {
        for (int i = t; i < total; i += kSmallThreads) {
            const int row = i / chunks;
            float v[8];
            load_row8(a.in, a.in_dtype, a.in_vec, b * a.in_stride + row * a.in_ld, a.cols, i - row * chunks, v);
            q.add8(v);
        }
    }
    const float f = block_scale(block_sums(q.value(), red), a.eps, &shared_scale);
    for (int i = t; i < total; i += kSmallThreads) {
        const int row = i / chunks, col = (i - row * chunks) * 8;
        float v[8];
        load_row8(a.in, a.in_dtype, a.in_vec, b * a.in_stride + row * a.in_ld, a.cols, col / 8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = col + e < a.cols ? v[e] * f : 0.0f;
        if (a.wide) {
            put_pair8(x + at_of(row, col), x_lo, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (col + e >= a.cols) break;
                unsigned char* p = x + at_of(col + e, row);
                split_half(v[e], *reinterpret_cast<__half*>(p), *reinterpret_cast<__half*>(p + x_lo));
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base, xs = smem_u32(x), gs = smem_u32(g);
    const int row = (warp & 3) * 32 + lane;   // this thread's line: its warp's quarter of TMEM
    const int fourth = warp >> 2;             // its warp's part of the columns
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int width = (a.m + 15) / 16 * 16, length = (a.n + 15) / 16 * 16;   // what the products cover
    uint32_t parity = 0;
    int failed = 0;
    for (int phase = 0; phase < 3 * a.steps; ++phase) {
        const int s = phase / 3, kind = phase % 3;
        fence_proxy_async_smem();
        tc_fence_before();
        if (__syncthreads_or(failed)) break;
        if (warp == 0) {
            tc_fence_after();
            if (elect_one()) {
                if (kind == 0)
                    issue(tmem, xs, x_lo, xs, x_lo, width, length / 16, false);
                else if (kind == 1)
                    issue(tmem, gs, g_lo, gs, g_lo, width, width / 16, false);
                else
                    issue(tmem, gs, g_lo, xs, x_lo, length, width / 16, true);
                mma_commit<1>(&bar);
            }
            __syncwarp();
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar, parity, nullptr, a.timeout_ns))) {
            failed = 1;
            continue;
        }
        parity ^= 1;
        tc_fence_after();
        const bool last = phase + 1 == 3 * a.steps;
        unsigned char* image = kind == 2 ? x : g;
        const int lo = kind == 2 ? x_lo : g_lo;
        const float alpha = (kind == 1 ? a.coef[s][2] : 1.0f) * (last ? kInvScale * kInvScale : kInvScale);
        const float beta = kind == 0 ? 0.0f : (kind == 1 ? a.coef[s][1] : a.coef[s][0]) * (last ? kInvScale : 1.0f);
        const int cols = kind == 2 ? length : width;
        for (int c = fourth * 16; c < cols; c += 64) {
            float v[16];
            tmem_sum16(mine + c, mine + kTmemSmall + c, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = v[8 * h + e];
                const int j = c + 8 * h;
                unsigned char* p = image + at_of(row, j);
                if (kind == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] *= alpha;
                } else {
                    combine8(p, lo, u, alpha, beta);
                }
                if (!last) {
                    put_pair8(p, lo, u);
                } else if (row < a.m && j < a.n) {
                    const int n = a.n - j;
                    if (a.wide) {
                        const long long o = b * a.out_stride + row * a.out_ld + j;
                        if (MUON)
                            put_weights8(a.master, a.lp, a.out_dtype, o, u, n, a.out_vec, a.decay, a.step);
                        else
                            put_row8(a.out, a.out_dtype, o, u, n, a.out_vec);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (e >= n) break;
                            const long long o = b * a.out_stride + (j + e) * a.out_ld + row;
                            float one[8] = {u[e], 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                            if (MUON)
                                put_weights8(a.master, a.lp, a.out_dtype, o, one, 1, false, a.decay, a.step);
                            else
                                put_row8(a.out, a.out_dtype, o, one, 1, false);
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    failed = __syncthreads_or(failed);
    if (warp == 0) {
        if (elect_one()) mma_commit<1>(&drain);   // TMEM is given back only after the last MMA
        __syncwarp();
        mbar_wait_bounded(&drain, 0, nullptr, 1000000000ull);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<1>(tmem, kTmemCols);
    if (t == 0 && failed && a.sc != nullptr) atomicOr(&a.sc->status, ZERO_DEV_TIMEOUT);
}

__global__ void __launch_bounds__(kSmallThreads, 1) ns_small(const __grid_constant__ SmallNsArgs a)
{
    ns_small_body<false>(a, nullptr);
}
__global__ void __launch_bounds__(kSmallThreads, 1) muon_small(const __grid_constant__ SmallNsArgs a, const __grid_constant__ MuonArgs mu)
{
    ns_small_body<true>(a, &mu);
}

}  // namespace

bool small_ns_fits(int rows, int cols, int products)
{
    const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    return products == 3 && m <= kLines && n <= 64 * kMaxPanels;
}

cudaError_t launch_small_ns(const NsArgs& a, const MuonArgs* mu, cudaStream_t st)
{
    SmallNsArgs k;
    std::memset(&k, 0, sizeof(k));
    k.rows = a.rows;
    k.cols = a.cols;
    k.wide = a.rows <= a.cols;
    k.m = k.wide ? a.rows : a.cols;
    k.n = k.wide ? a.cols : a.rows;
    k.panels = (k.n + 63) / 64;
    k.steps = a.steps;
    std::memcpy(k.coef, a.coef, sizeof(k.coef));
    k.eps = a.eps;
    k.sc = a.sc;
    k.timeout_ns = kDefaultTimeoutNs;
    if (mu != nullptr) {
        k.in = mu->u;
        k.in_dtype = ZERO_FP32;
        k.in_ld = a.cols;
        k.in_stride = mu->u_stride;
        k.in_vec = a.cols % 4 == 0;
        k.master = a.master;
        k.lp = a.lp;
        k.out_dtype = a.lp_dtype;
        k.out_ld = a.cols;
        k.out_stride = a.flat_stride;
        k.out_vec = a.cols % 8 == 0;
        k.decay = a.decay;
        k.step = a.step;
    } else {
        k.in = a.in;
        k.in_dtype = a.in_dtype;
        k.in_ld = a.in_ld;
        k.in_stride = a.in_stride;
        k.in_vec = wide_rows(a.in, a.in_dtype, a.in_ld, a.in_stride);
        k.out = a.out;
        k.out_dtype = a.out_dtype;
        k.out_ld = a.out_ld;
        k.out_stride = a.out_stride;
        k.out_vec = wide_rows(a.out, a.out_dtype, a.out_ld, a.out_stride);
    }
    const int smem = 2 * (k.panels + kSquarePanels) * kPanelBytes + 1024;
    constexpr int most = 2 * (kMaxPanels + kSquarePanels) * kPanelBytes + 1024;
    const cudaError_t e = mu != nullptr ? cudaFuncSetAttribute(muon_small, cudaFuncAttributeMaxDynamicSharedMemorySize, most)
                                        : cudaFuncSetAttribute(ns_small, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (mu != nullptr) return launch_after(muon_small, dim3(a.batch), dim3(kSmallThreads), smem, st, k, *mu);
    return launch_after(ns_small, dim3(a.batch), dim3(kSmallThreads), smem, st, k);
}

}  // namespace zk
