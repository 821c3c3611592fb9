// zk_ortho.cu -- the orthogonalised update: Newton-Schulz products on the
// tensor cores, and the Muon step built on them.
//
// With x_0 = g / (|g|_F + eps) and the Gram matrix on the short side
// (G = x x^T for rows <= cols, x^T x for tall matrices) every step is
//     G = x x^T,   P = b G + c G G,   x <- a x + P x      (tall: a x + x P)
// which moves each singular value s of x to a s + b s^3 + c s^5 and leaves the
// singular vectors alone.
//
// Numbers.  The products run on fp16 operands with fp32 accumulation (the
// tensor cores' full rate).  x, G and P are bounded (|x_ij| <= its largest
// singular value; the host checks the bounds for the given coefficients), so
// all three are stored times 2^12: entries of typical size 2^-12 and less
// then lie in fp16's normal range.  x is always carried as a pair hi + lo of
// fp16 values (22 bits): the term a x takes both, so the rounding of x to one
// fp16 does not feed back into its weak directions (with a single fp16 x, a
// gradient of a few strong directions came out 2e-2 off; as a pair 7e-4).
// products = 1 multiplies the hi parts only: the result is 2e-4 to 1.7e-3 off
// (relative, 2-norm), about the rounding of a bf16 result (1.7e-3).
// products = 3 also carries G and P as pairs and multiplies
// lo*hi + hi*lo + hi*hi: 3e-7 to 4e-6 off, for results kept in more than bf16.
#include <cuda_fp16.h>

#include <climits>
#include <cstring>

#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"
#include "zk_tc.cuh"

namespace zk {
namespace {

constexpr float kScale = 4096.0f;
constexpr float kInvScale = 1.0f / 4096.0f;
constexpr int kBM = 128;       // output rows of a CTA's tile (TMEM lanes)
constexpr int kBK = 64;        // depth of a pipeline stage: 128 bytes, one swizzle line
constexpr int kBox = 64;       // TMA boxes are 64 x 64 values, 8 KB, whichever side is the depth
constexpr int kBoxBytes = kBox * kBK * 2;
constexpr int kMmThreads = 320;   // producer, MMA, eight epilogue warps
constexpr int kMaxNsParts = 1024;
constexpr int kStrip = 16;

// how an operand lies in memory: its depth contiguous (K-major), its rows
// contiguous (MN-major), or a symmetric matrix of which only the blocks of
// `sb` x `sb` on and under the diagonal are stored
enum { kMajorK = 0, kMajorMN = 1, kSymLower = 2 };
enum { EPI_PLANES = 0, EPI_ADD = 1, EPI_OUT = 2, EPI_MUON = 3 };

struct MmArgs {
    CUtensorMap a[2], b[2];       // hi and lo planes
    int a_mode, b_mode;
    int m, n, k;
    int sb;
    int products;
    int lower;                    // only blocks on and under the diagonal
    int tiles_m, tiles_n, tiles_per_matrix, tiles;
    // result: alpha * sum + beta * addend
    float alpha, beta;
    const __half* add_hi;
    const __half* add_lo;         // may be null
    __half* out_hi;
    __half* out_lo;               // may be null
    long long add_ld, add_stride, out_ld, out_stride;   // elements
    void* out;                    // EPI_OUT
    int out_dtype, out_vec;
    float* master;                // EPI_MUON
    void* lp;
    float decay, step;
    zero_dev_scalars* sc;
    int starve;                   // issue no copy, so that every wait runs out
    unsigned long long timeout_ns;
};

struct Tile {
    int b, m0, n0;
};

// Tile t of the launch.  Lower-triangle launches number the tiles of block row
// I (sb rows, (I + 1) * sb columns) after those of the rows above.
template <int BN>
__device__ __forceinline__ Tile tile_of(const MmArgs& a, int t)
{
    Tile r;
    r.b = t / a.tiles_per_matrix;
    t -= r.b * a.tiles_per_matrix;
    if (!a.lower) {
        // strips of kStrip row tiles, column by column: the tiles in flight at a
        // time form a near-square block, whose operands stay in L2
        const int strip = t / (kStrip * a.tiles_n), first = strip * kStrip;
        const int rows = a.tiles_m - first < kStrip ? a.tiles_m - first : kStrip;
        t -= first * a.tiles_n;
        r.m0 = (first + t % rows) * kBM;
        r.n0 = t / rows * BN;
        return r;
    }
    constexpr int SB = BN > kBM ? BN : kBM;
    constexpr int kRows = SB / kBM, kCols = SB / BN;
    int i = static_cast<int>((sqrtf(1.0f + 8.0f * static_cast<float>(t / (kRows * kCols))) - 1.0f) * 0.5f);
    while (kRows * kCols * ((i + 1) * (i + 2) / 2) <= t) ++i;
    while (i > 0 && kRows * kCols * (i * (i + 1) / 2) > t) --i;
    t -= kRows * kCols * (i * (i + 1) / 2);
    const int width = (i + 1) * kCols;
    r.m0 = (i * kRows + t / width) * kBM;
    r.n0 = t % width * BN;
    return r;
}

// the depth from which an operand's tile at mn0 is read MN-major
__device__ __forceinline__ int mn_from(int mode, int sb, int mn0)
{
    return mode == kMajorK ? INT_MAX : mode == kMajorMN ? 0 : (mn0 & -sb) + sb;
}

template <int BOXES>
__device__ __forceinline__ void load_operand(unsigned char* dst, const CUtensorMap* map, bool mn, int mn0, int k0, int b,
                                             uint64_t* bar)
{
#pragma unroll
    for (int h = 0; h < BOXES; ++h)
        tma_load_3d(dst + h * kBoxBytes, map, mn ? mn0 + h * kBox : k0, mn ? k0 : mn0 + h * kBox, b, bar);
}

// a place in the ring of stages: the slot, and the parity of its current use
template <int N>
struct Slot {
    uint32_t i = 0, parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++i == N) i = 0, parity ^= 1;
    }
};

// ------------------------------------------------------------- epilogues
__device__ __forceinline__ float2 half2_up(uint32_t w)
{
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
}

// 32 consecutive values of a row of a pair of planes (lo may be null: zeros),
// all loads issued together, from L2 (another SM wrote them)
struct Addend {
    uint4 h[4], l[4];
    __device__ __forceinline__ void load(const __half* hi, const __half* lo, int n)
    {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            h[c] = l[c] = make_uint4(0, 0, 0, 0);
            if (8 * c < n) h[c] = __ldcg(reinterpret_cast<const uint4*>(hi) + c);
            if (8 * c < n && lo != nullptr) l[c] = __ldcg(reinterpret_cast<const uint4*>(lo) + c);
        }
    }
    // v = alpha * v + beta * (hi + lo)
    __device__ __forceinline__ void into(float (&v)[32], float alpha, float beta) const
    {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t hw[4] = {h[c].x, h[c].y, h[c].z, h[c].w}, lw[4] = {l[c].x, l[c].y, l[c].z, l[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = half2_up(hw[i]), q = half2_up(lw[i]);
                float* o = v + 8 * c + 2 * i;
                o[0] = fmaf(beta, p.x + q.x, alpha * o[0]);
                o[1] = fmaf(beta, p.y + q.y, alpha * o[1]);
            }
        }
    }
};

__device__ __forceinline__ void put_planes8(const float* v, __half* hi, __half* lo)
{
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
        hw[i] = *reinterpret_cast<const uint32_t*>(&h);
        lw[i] = *reinterpret_cast<const uint32_t*>(&l);
    }
    *reinterpret_cast<uint4*>(hi) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    if (lo != nullptr) *reinterpret_cast<uint4*>(lo) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
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

// 32 consecutive sums of one output row, from column `col`; what the result
// needs besides them is loaded before the sums arrive
template <int EPI>
__device__ __forceinline__ void epilogue(const MmArgs& a, int b, int row, int col, uint32_t tmem)
{
    const int n = a.n - col;
    const bool in = row < a.m;
    Addend x;
    if (EPI != EPI_PLANES && in) {
        const long long at = b * a.add_stride + row * a.add_ld + col;
        x.load(a.add_hi + at, a.add_lo != nullptr ? a.add_lo + at : nullptr, n);
    }
    float v[32];
    tmem_load32(tmem, v);
    if (!in) return;
    if (EPI == EPI_PLANES) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= a.alpha;
    } else {
        x.into(v, a.alpha, a.beta);
    }
    const long long o = b * a.out_stride + row * a.out_ld + col;
    if (EPI == EPI_PLANES || EPI == EPI_ADD) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (8 * c < n) put_planes8(v + 8 * c, a.out_hi + o + 8 * c, a.out_lo != nullptr ? a.out_lo + o + 8 * c : nullptr);
    } else if (EPI == EPI_OUT) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (8 * c < n) put_row8(a.out, a.out_dtype, o + 8 * c, v + 8 * c, n - 8 * c, a.out_vec);
    } else {
        // w <- w * (1 - lr wd) - step * o, rounded to the master's fp32, then its 16-bit cast
        float w[32];
        if (a.out_vec && n >= 32) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float4 p = *reinterpret_cast<const float4*>(a.master + o + 4 * c);
                w[4 * c] = p.x, w[4 * c + 1] = p.y, w[4 * c + 2] = p.z, w[4 * c + 3] = p.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = e < n ? a.master[o + e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(-a.step, v[e], w[e] * a.decay);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (8 * c >= n) break;
            put_row8(a.master, ZERO_FP32, o + 8 * c, v + 8 * c, n - 8 * c, a.out_vec);
            if (a.lp != nullptr) put_row8(a.lp, a.out_dtype, o + 8 * c, v + 8 * c, n - 8 * c, a.out_vec);
        }
    }
}

template <int BN>
struct MmShape {
    static constexpr int kStageBytes = (kBM + BN) * kBK * 2;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int kSmem = kStages * kStageBytes + 1024;   // + alignment of the ring
};

// One persistent CTA per SM walks the tiles: a producer thread keeps a ring of
// 64-deep operand tiles full by TMA, one thread issues the MMAs into one of
// two TMEM accumulators, and eight warps turn the other one into results.
template <int BN, int EPI>
__global__ void __launch_bounds__(kMmThreads, 1) mm_kernel(const __grid_constant__ MmArgs a)
{
    using S = MmShape<BN>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;
    unsigned char* ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023u)) % 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 8);
        }
        mbar_init(&drain, 1);
        abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&a.a[0]);
        prefetch_tmap(&a.b[0]);
    }
    if (warp == 1) tmem_alloc(&tmem_base, 2 * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_launch();

    if (warp == 0) {
      if (lane == 0) {
        fence_proxy_async_global();   // the previous kernel's plain stores, before our TMA loads
        Slot<S::kStages> s;
        uint32_t issued = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < a.tiles; t += gridDim.x) {
            const Tile tl = tile_of<BN>(a, t);
            const int am = mn_from(a.a_mode, a.sb, tl.m0), bm = mn_from(a.b_mode, a.sb, tl.n0);
            // small products first: lo*hi, hi*lo, then hi*hi
            for (int pass = 3 - a.products; ok && pass < 3; ++pass) {
                const CUtensorMap* ma = &a.a[pass == 0];
                const CUtensorMap* mb = &a.b[pass == 1];
                for (int k0 = 0; k0 < a.k; k0 += kBK) {
                    if (issued >= S::kStages && !mbar_wait_bounded(&empty[s.i], s.parity ^ 1, &abort_flag, a.timeout_ns)) {
                        abort_flag = 1;
                        ok = false;
                        break;
                    }
                    if (!a.starve) {
                        unsigned char* p = ring + s.i * S::kStageBytes;
                        mbar_arrive_expect_tx(&full[s.i], S::kStageBytes);
                        load_operand<kBM / kBox>(p, ma, k0 >= am, tl.m0, k0, tl.b, &full[s.i]);
                        load_operand<BN / kBox>(p + kBM * kBK * 2, mb, k0 >= bm, tl.n0, k0, tl.b, &full[s.i]);
                    }
                    s.next();
                    ++issued;
                }
            }
        }
        if (!ok && !a.starve) {
            // nothing of ours may still be landing when the CTA's memory goes away
            for (uint32_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
                mbar_wait_bounded(&full[i % S::kStages], (i / S::kStages) & 1, nullptr, 1000000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        Slot<S::kStages> s;
        Slot<2> acc;
        uint32_t n_tile = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < a.tiles; t += gridDim.x, ++n_tile) {
            const Tile tl = tile_of<BN>(a, t);
            const int am = mn_from(a.a_mode, a.sb, tl.m0), bm = mn_from(a.b_mode, a.sb, tl.n0);
            if (n_tile >= 2 && !mbar_wait_bounded(&acc_empty[acc.i], acc.parity ^ 1, &abort_flag, a.timeout_ns)) {
                abort_flag = 1;
                break;
            }
            tc_fence_after();
            bool more = false;   // false: the accumulator starts anew
            for (int pass = 3 - a.products; ok && pass < 3; ++pass) {
                for (int k0 = 0; k0 < a.k; k0 += kBK) {
                    if (!mbar_wait_bounded(&full[s.i], s.parity, &abort_flag, a.timeout_ns)) {
                        abort_flag = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool a_mn = k0 >= am, b_mn = k0 >= bm;
                    const uint32_t idesc = instr_desc(kBM, BN, a_mn, b_mn);
                    const uint32_t p = smem_u32(ring + s.i * S::kStageBytes);
                    const uint64_t da = smem_desc(p), db = smem_desc(p + kBM * kBK * 2);
                    // sixteen values of depth: 32 bytes along a line, or sixteen lines
                    const uint32_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sbb = b_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        mma_f16(tmem + acc.i * BN, da + k * sa, db + k * sbb, idesc, more || k > 0);
                    more = true;
                    mma_commit(&empty[s.i]);
                    s.next();
                }
            }
            if (ok) mma_commit(&acc_full[acc.i]);
            acc.next();
        }
        mma_commit(&drain);   // TMEM is given back only after the last MMA
        mbar_wait_bounded(&drain, 0, nullptr, 1000000000ull);
      }
      __syncwarp();
    } else {
        const int quarter = warp & 3;         // the TMEM lanes this warp may read
        const int half = (warp - 2) >> 2;     // its half of the columns
        uint32_t n_tile = 0;
        for (int t = blockIdx.x; t < a.tiles; t += gridDim.x, ++n_tile) {
            const Tile tl = tile_of<BN>(a, t);
            const int acc = n_tile & 1;
            if (!mbar_wait_bounded(&acc_full[acc], (n_tile >> 1) & 1, &abort_flag, a.timeout_ns)) {
                abort_flag = 1;
                break;
            }
            tc_fence_after();
            const int row = tl.m0 + quarter * 32 + lane;
#pragma unroll 1
            for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
                if (tl.n0 + c >= a.n) break;
                epilogue<EPI>(a, tl.b, row, tl.n0 + c, tmem + acc * BN + c + (static_cast<uint32_t>(quarter * 32) << 16));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem, 2 * BN);
    if (threadIdx.x == 0 && abort_flag && a.sc != nullptr) atomicOr(&a.sc->status, ZERO_DEV_TIMEOUT);
}

// ------------------------------------------------- norms and first operands
struct PrepArgs {
    const void* in;
    int dtype, vec;
    long long ld, stride;
    int rows, cols, chunks;      // chunks: groups of eight columns in a row
    float eps;
    double* parts;               // [batch][gridDim.x]
    __half* hi;
    __half* lo;
    long long out_ld, out_stride;
};

// eight consecutive elements from column 8 * ch of a row, zeros past its end
__device__ __forceinline__ void load_row8(const PrepArgs& a, long long base, int row, int ch, float (&v)[8])
{
    const long long i = base + row * a.ld + 8 * ch;
    const int n = a.cols - 8 * ch;
    if (a.dtype == ZERO_FP32) {
        const float* p = static_cast<const float*>(a.in) + i;
        if (a.vec && n >= 8) {
            const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
        }
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(a.in) + i;
    uint32_t w[4];
    if (a.vec && n >= 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (2 * e < n ? p[2 * e] : 0u) | ((2 * e + 1 < n ? static_cast<uint32_t>(p[2 * e + 1]) : 0u) << 16);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::lo(w[e]) : Lp<ZERO_FP16>::lo(w[e]);
        v[2 * e + 1] = a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::hi(w[e]) : Lp<ZERO_FP16>::hi(w[e]);
    }
}

// the squares of eight values; in fp32 unless that overflows
__device__ __forceinline__ double squares8(const float (&v)[8])
{
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
    if (is_finite_f32(s)) return static_cast<double>(s);
    double d = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) d += static_cast<double>(v[e]) * static_cast<double>(v[e]);
    return d;
}

// sum over a block of 256 threads, in every thread; red: 8 doubles
__device__ __forceinline__ double block_sum_f64(double v, double* red)
{
    v = warp_sum_f64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < 8; ++i) s += red[i];
    return s;
}

__global__ void __launch_bounds__(256) ns_sqnorm(const __grid_constant__ PrepArgs a)
{
    __shared__ double red[8];
    pdl_wait();
    pdl_launch();
    const uint32_t total = static_cast<uint32_t>(a.rows) * a.chunks;
    const long long base = blockIdx.y * a.stride;
    double s = 0.0;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
        const uint32_t row = i / static_cast<uint32_t>(a.chunks);
        float v[8];
        load_row8(a, base, row, i - row * a.chunks, v);
        s += squares8(v);
    }
    s = block_sum_f64(s, red);
    if (threadIdx.x == 0) a.parts[blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x] = s;
}

// x_0 = g / (|g| + eps) as a scaled hi/lo pair; parts_n partial sums a matrix
__global__ void __launch_bounds__(256) ns_scale(const __grid_constant__ PrepArgs a, int parts_n)
{
    __shared__ double red[8];
    pdl_wait();
    pdl_launch();
    double s = 0.0;
    for (int i = threadIdx.x; i < parts_n; i += 256) s += a.parts[blockIdx.y * static_cast<long long>(parts_n) + i];
    s = block_sum_f64(s, red);
    const float f = static_cast<float>(static_cast<double>(kScale) / (sqrt(s) + static_cast<double>(a.eps)));
    const uint32_t total = static_cast<uint32_t>(a.rows) * a.chunks;
    const long long base = blockIdx.y * a.stride;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
        const uint32_t row = i / static_cast<uint32_t>(a.chunks);
        const int ch = i - row * a.chunks;
        float v[8];
        load_row8(a, base, row, ch, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 8 * ch + e < a.cols ? v[e] * f : 0.0f;
        const long long o = blockIdx.y * a.out_stride + row * a.out_ld + 8 * ch;
        put_planes8(v, a.hi + o, a.lo + o);
    }
}

struct MuonArgs {
    const void* rank[ZERO_MAX_RANKS];
    int n_d, dtype, nesterov;
    float divisor, mu;
    float* momentum;
    float* u;
    long long stride, u_stride;
    uint32_t elems;              // of one matrix
    double* parts;
};

// Rank mean (rank order, fp32), momentum, and the update direction u with its
// squared norm: m <- mu m + g, u = g + mu m (Nesterov) or m.
__global__ void __launch_bounds__(256) muon_direction(const __grid_constant__ MuonArgs a)
{
    __shared__ double red[8];
    pdl_wait();
    pdl_launch();
    double s = 0.0;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i * 8u < a.elems; i += gridDim.x * 256) {
        const int n = a.elems - 8 * i < 8 ? static_cast<int>(a.elems - 8 * i) : 8;
        const long long at = blockIdx.y * a.stride + 8ll * i;
        float g[8], m[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.0f;
        if (n == 8) {
#pragma unroll 4
            for (int q = 0; q < a.n_d; ++q) {
                const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.rank[q]) + at);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[2 * e] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::lo(w[e]) : Lp<ZERO_FP16>::lo(w[e]);
                    g[2 * e + 1] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::hi(w[e]) : Lp<ZERO_FP16>::hi(w[e]);
                }
            }
        } else {
            for (int q = 0; q < a.n_d; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) {
                        const uint16_t h = static_cast<const uint16_t*>(a.rank[q])[at + e];
                        g[e] += a.dtype == ZERO_BF16 ? Lp<ZERO_BF16>::widen(h) : Lp<ZERO_FP16>::widen(h);
                    }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = 0.0f;
        float* mp = a.momentum + at;
        if (n == 8) {
            const float4 x = *reinterpret_cast<const float4*>(mp), y = *reinterpret_cast<const float4*>(mp + 4);
            m[0] = x.x, m[1] = x.y, m[2] = x.z, m[3] = x.w, m[4] = y.x, m[5] = y.y, m[6] = y.z, m[7] = y.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) m[e] = mp[e];
        }
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float mean = __fdiv_rn(g[e], a.divisor);
            m[e] = __fadd_rn(__fmul_rn(a.mu, m[e]), mean);
            u[e] = e >= n ? 0.0f : a.nesterov ? __fadd_rn(mean, __fmul_rn(a.mu, m[e])) : m[e];
        }
        put_row8(a.momentum, ZERO_FP32, at, m, n, true);
        put_row8(a.u, ZERO_FP32, blockIdx.y * a.u_stride + 8ll * i, u, 8, true);
        s += squares8(u);
    }
    s = block_sum_f64(s, red);
    if (threadIdx.x == 0) a.parts[blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x] = s;
}

// ------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
long long up64(long long n) { return (n + 63) / 64 * 64; }

// An fp16 matrix batch of the workspace: rows of ld (a multiple of 64, so that
// the epilogue's 32-wide pieces stay inside a row) elements.
struct Planes {
    __half* hi = nullptr;
    __half* lo = nullptr;
    int rows = 0, cols = 0;
    long long ld = 0, stride = 0;
};

bool encode(CUtensorMap* map, const Planes& p, const __half* plane, int batch)
{
    const EncodeFn fn = encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.cols), static_cast<cuuint64_t>(p.rows), static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.ld) * 2, static_cast<cuuint64_t>(p.stride) * 2};
    const cuuint32_t box[3] = {kBox, kBox, 1}, unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(plane), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
    size_t parts, u, x[2], g, p, end;
    long long x_plane, s_plane;   // elements of one plane
    int planes;
};

Layout layout_of(int rows, int cols, int batch, int products, bool muon)
{
    Layout l;
    const long long m = rows < cols ? rows : cols;
    l.planes = products == 3 ? 2 : 1;
    l.x_plane = static_cast<long long>(batch) * rows * up64(cols);
    l.s_plane = static_cast<long long>(batch) * m * up64(m);
    size_t at = 0;
    l.parts = at;
    at += up256(static_cast<size_t>(batch) * kMaxNsParts * sizeof(double));
    l.u = at;
    if (muon) at += up256(static_cast<size_t>(batch) * ((static_cast<size_t>(rows) * cols + 7) / 8 * 8) * sizeof(float));
    for (int i = 0; i < 2; ++i) {
        l.x[i] = at;
        at += 2 * up256(static_cast<size_t>(l.x_plane) * 2);
    }
    l.g = at;
    at += l.planes * up256(static_cast<size_t>(l.s_plane) * 2);
    l.p = at;
    at += l.planes * up256(static_cast<size_t>(l.s_plane) * 2);
    l.end = at;
    return l;
}

Planes planes_at(void* ws, size_t at, long long elems, int rows, int cols, bool two)
{
    Planes p;
    p.hi = reinterpret_cast<__half*>(static_cast<char*>(ws) + at);
    p.lo = two ? reinterpret_cast<__half*>(static_cast<char*>(ws) + at + up256(static_cast<size_t>(elems) * 2)) : nullptr;
    p.rows = rows;
    p.cols = cols;
    p.ld = up64(cols);
    p.stride = static_cast<long long>(rows) * p.ld;
    return p;
}

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

template <int BN, int EPI>
cudaError_t launch_mm_as(const MmArgs& a, int sms, cudaStream_t st)
{
    const cudaError_t e = cudaFuncSetAttribute(mm_kernel<BN, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmShape<BN>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_after(mm_kernel<BN, EPI>, dim3(a.tiles < sms ? a.tiles : sms), dim3(kMmThreads), MmShape<BN>::kSmem, st, a);
}

template <int EPI>
cudaError_t launch_mm(int bn, MmArgs& a, int batch, int sms, cudaStream_t st)
{
    const int sb = bn > kBM ? bn : kBM;
    a.sb = sb;
    a.tiles_n = (a.n + bn - 1) / bn;
    a.tiles_m = (a.m + kBM - 1) / kBM;
    if (a.lower) {
        const int blocks = (a.m + sb - 1) / sb;
        a.tiles_per_matrix = (sb / kBM) * (sb / bn) * (blocks * (blocks + 1) / 2);
    } else {
        a.tiles_per_matrix = a.tiles_n * a.tiles_m;
    }
    a.tiles = a.tiles_per_matrix * batch;
    if (bn == 256) return launch_mm_as<256, EPI>(a, sms, st);
    if (bn == 128) return launch_mm_as<128, EPI>(a, sms, st);
    return launch_mm_as<64, EPI>(a, sms, st);
}

bool set_operands(MmArgs& m, const Planes& a, int a_mode, const Planes& b, int b_mode, int products, int batch)
{
    m.a_mode = a_mode;
    m.b_mode = b_mode;
    m.products = products;
    bool ok = encode(&m.a[0], a, a.hi, batch) && encode(&m.b[0], b, b.hi, batch);
    if (products == 3) ok = ok && encode(&m.a[1], a, a.lo, batch) && encode(&m.b[1], b, b.lo, batch);
    return ok;
}

void set_addend(MmArgs& m, const Planes& p)
{
    m.add_hi = p.hi;
    m.add_lo = p.lo;
    m.add_ld = p.ld;
    m.add_stride = p.stride;
}

void set_result(MmArgs& m, const Planes& p)
{
    m.out_hi = p.hi;
    m.out_lo = p.lo;
    m.out_ld = p.ld;
    m.out_stride = p.stride;
}

}  // namespace

size_t ns_workspace_bytes(int rows, int cols, int batch, int products, bool muon)
{
    return layout_of(rows, cols, batch, products, muon).end;
}

#define ZK_GO(expr)                             \
    do {                                        \
        const cudaError_t e_ = (expr);          \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

cudaError_t launch_mm_starved(void* scratch, zero_dev_scalars* sc, unsigned long long timeout_ns, cudaStream_t st)
{
    const Planes p = planes_at(scratch, 0, 64 * 64, 64, 64, false);
    const Planes r = planes_at(scratch, 64 * 64 * 2, 64 * 64, 64, 64, false);
    MmArgs k;
    std::memset(&k, 0, sizeof(k));
    k.m = k.n = k.k = 64;
    k.sc = sc;
    k.timeout_ns = timeout_ns;
    k.starve = 1;
    if (!set_operands(k, p, kMajorK, p, kMajorK, 1, 1)) return cudaErrorInvalidValue;
    set_result(k, r);
    return launch_mm<EPI_PLANES>(64, k, 1, 1, st);
}

cudaError_t launch_ns(const NsArgs& a, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    const bool muon = a.out == nullptr, wide = a.rows <= a.cols;
    const int m = wide ? a.rows : a.cols;
    const Layout l = layout_of(a.rows, a.cols, a.batch, a.products, muon);
    Planes x[2] = {planes_at(a.ws, l.x[0], l.x_plane, a.rows, a.cols, true), planes_at(a.ws, l.x[1], l.x_plane, a.rows, a.cols, true)};
    const Planes g = planes_at(a.ws, l.g, l.s_plane, m, m, a.products == 3);
    const Planes p = planes_at(a.ws, l.p, l.s_plane, m, m, a.products == 3);

    // the norm and x_0
    PrepArgs pr;
    std::memset(&pr, 0, sizeof(pr));
    pr.rows = a.rows;
    pr.cols = a.cols;
    pr.chunks = (a.cols + 7) / 8;
    pr.eps = a.eps;
    pr.parts = reinterpret_cast<double*>(static_cast<char*>(a.ws) + l.parts);
    pr.hi = x[0].hi;
    pr.lo = x[0].lo;
    pr.out_ld = x[0].ld;
    pr.out_stride = x[0].stride;
    // CTAs a matrix: four chunks a thread, eight CTAs an SM over the batch
    const long long chunks = static_cast<long long>(a.rows) * pr.chunks;
    long long per = (chunks + 1023) / 1024, most = (8LL * sms + a.batch - 1) / a.batch;
    if (per > most) per = most;
    if (per > kMaxNsParts) per = kMaxNsParts;
    const dim3 grid(static_cast<unsigned>(per), a.batch);
    if (muon) {
        MuonArgs mu;
        std::memset(&mu, 0, sizeof(mu));
        for (int q = 0; q < a.n_d; ++q) mu.rank[q] = a.ranks[q];
        mu.n_d = a.n_d;
        mu.dtype = a.in_dtype;
        mu.nesterov = a.nesterov;
        mu.divisor = a.divisor;
        mu.mu = a.mu;
        mu.momentum = a.momentum;
        mu.u = reinterpret_cast<float*>(static_cast<char*>(a.ws) + l.u);
        mu.stride = a.flat_stride;
        mu.elems = static_cast<uint32_t>(a.rows) * static_cast<uint32_t>(a.cols);
        mu.u_stride = (static_cast<long long>(mu.elems) + 7) / 8 * 8;
        mu.parts = pr.parts;
        pr.in = mu.u;
        pr.dtype = ZERO_FP32;
        pr.ld = a.cols;
        pr.stride = mu.u_stride;
        pr.vec = a.cols % 4 == 0;
        ZK_GO(launch_after(muon_direction, grid, dim3(256), 0, st, mu));
    } else {
        const int v = 16 / dtype_bytes(a.in_dtype);
        pr.in = a.in;
        pr.dtype = a.in_dtype;
        pr.ld = a.in_ld;
        pr.stride = a.in_stride;
        pr.vec = reinterpret_cast<uintptr_t>(a.in) % 16 == 0 && a.in_ld % v == 0 && a.in_stride % v == 0;
        ZK_GO(launch_after(ns_sqnorm, grid, dim3(256), 0, st, pr));
    }
    ZK_GO(launch_after(ns_scale, grid, dim3(256), 0, st, pr, static_cast<int>(per)));

    // one tile width for the call (the stored triangle's blocks go by it)
    const long long wide_tiles = static_cast<long long>(a.batch) * ((a.rows + kBM - 1) / kBM) * ((a.cols + 255) / 256);
    const int bn = wide_tiles >= sms ? 256 : 2 * wide_tiles >= sms ? 128 : 64;

    MmArgs base;
    std::memset(&base, 0, sizeof(base));
    base.sc = a.sc;
    base.timeout_ns = kDefaultTimeoutNs;
    for (int s = 0; s < a.steps; ++s) {
        const Planes& xi = x[s & 1];
        const Planes& xo = x[(s & 1) ^ 1];
        const float ca = a.coef[s][0], cb = a.coef[s][1], cc = a.coef[s][2];
        MmArgs k = base;   // G = x x^T
        k.m = k.n = m;
        k.k = wide ? a.cols : a.rows;
        k.lower = 1;
        k.alpha = kInvScale;
        if (!set_operands(k, xi, wide ? kMajorK : kMajorMN, xi, wide ? kMajorK : kMajorMN, a.products, a.batch)) return cudaErrorInvalidValue;
        set_result(k, g);
        ZK_GO(launch_mm<EPI_PLANES>(bn, k, a.batch, sms, st));

        k = base;          // P = b G + c G G
        k.m = k.n = k.k = m;
        k.lower = 1;
        k.alpha = cc * kInvScale;
        k.beta = cb;
        if (!set_operands(k, g, kSymLower, g, kSymLower, a.products, a.batch)) return cudaErrorInvalidValue;
        set_addend(k, g);
        set_result(k, p);
        ZK_GO(launch_mm<EPI_ADD>(bn, k, a.batch, sms, st));

        k = base;          // x <- a x + P x, or a x + x P
        k.m = a.rows;
        k.n = a.cols;
        k.k = m;
        k.alpha = kInvScale;
        k.beta = ca;
        if (!(wide ? set_operands(k, p, kSymLower, xi, kMajorMN, a.products, a.batch)
                   : set_operands(k, xi, kMajorK, p, kSymLower, a.products, a.batch)))
            return cudaErrorInvalidValue;
        set_addend(k, xi);
        if (s + 1 < a.steps) {
            set_result(k, xo);
            ZK_GO(launch_mm<EPI_ADD>(bn, k, a.batch, sms, st));
            continue;
        }
        // the last step leaves x itself: scaled back, in its own type
        k.alpha *= kInvScale;
        k.beta *= kInvScale;
        if (!muon) {
            const int v = 16 / dtype_bytes(a.out_dtype);
            k.out = a.out;
            k.out_dtype = a.out_dtype;
            k.out_ld = a.out_ld;
            k.out_stride = a.out_stride;
            k.out_vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_ld % v == 0 && a.out_stride % v == 0;
            ZK_GO(launch_mm<EPI_OUT>(bn, k, a.batch, sms, st));
        } else {
            k.master = a.master;
            k.lp = a.lp;
            k.out_dtype = a.lp_dtype;
            k.out_ld = a.cols;
            k.out_stride = a.flat_stride;
            k.out_vec = a.cols % 8 == 0;
            k.decay = a.decay;
            k.step = a.step;
            ZK_GO(launch_mm<EPI_MUON>(bn, k, a.batch, sms, st));
        }
    }
    return cudaSuccess;
}

}  // namespace zk
