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
// lo*hi + hi*lo + hi*hi, for results kept in more than bf16: 3e-7 to 4e-6 off,
// up to 3e-5 with a side of 4096, where the accumulator's own dropped bits (it
// truncates at each addition of a 16-deep slice) outweigh the operands'.
//
// Work and floor.  With m the short and n the long side, a step multiplies
// m (m + 1) n + m^2 (m + 1) + 2 m^2 n times and adds as often (G and P are
// symmetric: half their blocks), three times that with products = 3; at 1912
// TFLOP/s (a large library product's rate) 4096 x 14336 cannot take less than
// 2.07 ms, twelve 768 x 768 57 us.  Large matrices are bound by the tensor
// cores and, in effect, by power (4096 x 14336: 2.84 ms, 1.4 PFLOP/s).
// Mid sizes are bound by what fifteen dependent products cost beside their
// MMAs: a meeting of the CTAs (1 to 2 us), the first tiles' way from L2 (1 us)
// and the last tiles' results (2 to 6 us); a 256 x 256 matrix, whose products
// take 1 us each, pays 6.4 us a product.  Hence one launch for the whole
// iteration (a launch for each product: 12 x 768 x 768 390 us, now 222), the
// depth of a tile split among CTAs where tiles are few, and 32 x 32 pieces of
// results that go out in whole 64-byte lines.
#include <climits>
#include <cstring>

#include "zk_launch.h"
#include "zk_ns.cuh"
#include "zk_ops.h"
#include "zk_tc.cuh"

namespace zk {
namespace {

constexpr int kBM = 128;       // output rows of a CTA (TMEM lanes); a pair of CTAs shares tiles of twice as many
constexpr int kBK = 64;        // depth of a pipeline stage: 128 bytes, one swizzle line
constexpr int kBox = 64;       // rows (columns) of an operand that one TMA copy brings, 8 KB
constexpr int kBoxBytes = kBox * kBK * 2;
constexpr int kThreads = 352;  // producer, MMA, eight epilogue warps, one that plans the next phase
constexpr int kEpiWarps = 8;
constexpr int kTurnBytes = 32 * 32 * 4;   // of an epilogue warp's 32 x 32 turning buffer
constexpr int kMaxNsParts = 1024;
constexpr int kStrip = 16;     // 128-row tiles of a strip (see tile_of)
constexpr int kBarStride = 32; // words between the groups' barrier counters: a line each
constexpr unsigned kPoison = 0x80000000u;

// how an operand lies in memory: its depth contiguous (K-major), its rows
// contiguous (MN-major), or a symmetric matrix of which only the blocks of
// `sb` x `sb` on and under the diagonal are stored
enum { kMajorK = 0, kMajorMN = 1, kSymLower = 2 };
struct DevPlanes {
    __half* hi;
    __half* lo;                  // may be null
    long long ld, stride;        // elements
};

struct NsKernelArgs {
    CUtensorMap xmap[2][2], gmap[2], pmap[2];   // hi and lo planes
    DevPlanes x[2], g, p;
    int rows, cols, m, wide, batch;
    int steps, products;
    int groups, ctas;            // CTAs of a group (CG = 2: pairs); a group takes every groups-th matrix
    int split[3];                // CTAs that share a tile's depth: for G, P and x
    float coef[kNsMaxSteps][3];
    // x_0
    const void* in;
    int in_dtype, in_vec, chunks;
    long long in_ld, in_stride;
    float eps;
    const float4* parts;         // [batch][parts_n] sums of squares
    int parts_n;
    // the result
    int res;                     // RES_OUT or RES_MUON
    void* out;
    int out_dtype, out_vec;
    long long out_ld, out_stride;
    float* master;
    void* lp;
    float decay, step;
    // exchange between CTAs
    unsigned* group_bar;         // [groups] counters, kBarStride words apart
    unsigned* tile_bar;          // [groups][ctas]
    float* partial;              // [groups * ctas][128 * BN]
    zero_dev_scalars* sc;
    int guarded;                 // nothing to do where sc's non-finite flag is set (loss scaling)
    int starve;                  // issue no copy, so that every wait runs out
    unsigned long long timeout_ns;
};

struct Tile {
    int m0, n0;
};

// One product: alpha * A B^T + beta * addend over an m x n result.
struct Phase {
    const CUtensorMap* a;               // hi; lo follows
    const CUtensorMap* b;
    int a_mode, b_mode;
    int m, n, k;
    int lower;                   // only blocks on and under the diagonal
    int tiles_m, tiles_n, tiles, split;
    Tile first;                  // this CTA's first tile
    unsigned tile_target;        // tile_bar's count once all parts of a tile of this phase are there
    int res;
    float alpha, beta;
    const __half* add_hi;        // this matrix's; rows out.ld apart
    const __half* add_lo;
    DevPlanes out;               // RES_PLANES*: this matrix's
    void* res_out;               // RES_OUT, RES_MUON: this matrix's result, or master and 16-bit weights
    float* master;
    int res_dtype, res_vec;
    long long res_ld;
    float decay, step;
};

// side of the blocks in which a symmetric matrix is stored
__host__ __device__ constexpr int sym_block(int cg, int bn) { return bn > kBM * cg ? bn : kBM * cg; }

// Tile t of a phase.  Lower-triangle phases number the tiles of block row I
// (sb rows, (I + 1) * sb columns) after those of the rows above.  Others go in
// strips of kStrip row tiles, column by column: the tiles in flight at a time
// form a near-square block, whose operands stay in L2.
template <int CG, int BN>
__device__ __forceinline__ Tile tile_of(const Phase& a, int t)
{
    constexpr int BM = kBM * CG, kStripTiles = kStrip / CG;
    Tile r;
    if (!a.lower) {
        const int strip = t / (kStripTiles * a.tiles_n), first = strip * kStripTiles;
        const int rows = a.tiles_m - first < kStripTiles ? a.tiles_m - first : kStripTiles;
        t -= first * a.tiles_n;
        r.m0 = (first + t % rows) * BM;
        r.n0 = t / rows * BN;
        return r;
    }
    constexpr int SB = sym_block(CG, BN);
    constexpr int kRows = SB / BM, kCols = SB / BN;
    int i = static_cast<int>((sqrtf(1.0f + 8.0f * static_cast<float>(t / (kRows * kCols))) - 1.0f) * 0.5f);
    while (kRows * kCols * ((i + 1) * (i + 2) / 2) <= t) ++i;
    while (i > 0 && kRows * kCols * (i * (i + 1) / 2) > t) --i;
    t -= kRows * kCols * (i * (i + 1) / 2);
    const int width = (i + 1) * kCols;
    r.m0 = (i * kRows + t / width) * BM;
    r.n0 = t % width * BN;
    return r;
}

// the depth from which an operand's tile at mn0 is read MN-major
__device__ __forceinline__ int mn_from(int mode, int sb, int mn0)
{
    return mode == kMajorK ? INT_MAX : mode == kMajorMN ? 0 : (mn0 & -sb) + sb;
}

template <int CG, int BOXES>
__device__ __forceinline__ void load_operand(unsigned char* dst, const CUtensorMap* map, bool mn, int mn0, int k0, int b, uint64_t* bar)
{
#pragma unroll
    for (int h = 0; h < BOXES; ++h)
        tma_load_3d<CG>(dst + h * kBoxBytes, map, mn ? mn0 + h * kBox : k0, mn ? k0 : mn0 + h * kBox, b, bar);
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
// eight consecutive values of a pair of planes (lo may be null: zeros), from
// L2: another SM may have written them a moment ago
struct Addend {
    uint4 h, l;
    __device__ __forceinline__ void zero() { h = l = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __half* hi, const __half* lo)
    {
        h = __ldcg(reinterpret_cast<const uint4*>(hi));
        l = lo != nullptr ? __ldcg(reinterpret_cast<const uint4*>(lo)) : make_uint4(0, 0, 0, 0);
    }
};

// eight fp32 values in register pairs
struct Eight {
    f32x2 v[4];
    __device__ __forceinline__ void set(const float4& p, const float4& q)
    {
        v[0] = pack2(p.x, p.y), v[1] = pack2(p.z, p.w), v[2] = pack2(q.x, q.y), v[3] = pack2(q.z, q.w);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void scale(f32x2 alpha)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], alpha);
    }
    // alpha * v + beta * (hi + lo)
    __device__ __forceinline__ void combine(f32x2 alpha, f32x2 beta, const Addend& x)
    {
        const uint32_t hw[4] = {x.h.x, x.h.y, x.h.z, x.h.w}, lw[4] = {x.l.x, x.l.y, x.l.z, x.l.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = half2_up(hw[i]), q = half2_up(lw[i]);
            v[i] = fma2(beta, add2(pack2(p.x, p.y), pack2(q.x, q.y)), mul2(alpha, v[i]));
        }
    }
};

__device__ __forceinline__ void put_planes8(const Eight& x, __half* hi, __half* lo)
{
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack2(x.v[i], a, b);
        const __half2 h = __floats2half2_rn(a, b);
        hw[i] = *reinterpret_cast<const uint32_t*>(&h);
        if (lo != nullptr) {
            const float2 f = __half22float2(h);
            const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
            lw[i] = *reinterpret_cast<const uint32_t*>(&l);
        }
    }
    *reinterpret_cast<uint4*>(hi) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    if (lo != nullptr) *reinterpret_cast<uint4*>(lo) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
}

// what becomes of a phase's sums: a pair of fp16 planes, the result, or the weights
enum { RES_PLANES = 0, RES_OUT = 1, RES_MUON = 2 };

// What the results of a phase need, in registers.  Addends and results that are
// planes lie alike: one offset (in elements, below 2^32 in any matrix) for all.
struct Results {
    int m, n, res;
    float alpha, beta;
    const __half* add_hi;
    const __half* add_lo;
    __half* hi;
    __half* lo;
    uint32_t ld;

    __device__ __forceinline__ explicit Results(const Phase& ph)
        : m(ph.m), n(ph.n), res(ph.res), alpha(ph.alpha), beta(ph.beta), add_hi(ph.add_hi), add_lo(ph.add_lo), hi(ph.out.hi),
          lo(ph.out.lo), ld(static_cast<uint32_t>(ph.out.ld))
    {
    }
    __device__ __forceinline__ void load(bool there, uint32_t at, Addend& x) const
    {
        x.zero();
        if (there && add_hi != nullptr) x.load(add_hi + at, add_lo != nullptr ? add_lo + at : nullptr);
    }
};

// The last phase: x itself, to the result or into the weights; n of the eight
// values exist.  Once a call, so kept out of the other phases' way.
__device__ __noinline__ void put_last(const Phase* ph, int row, int col, Eight u)
{
    const int n = ph->n - col;
    const long long o = row * ph->res_ld + col;
    const bool vec = ph->res_vec;
    float v[8];
    u.get(v);
    if (ph->res == RES_OUT) {
        put_row8(ph->res_out, ph->res_dtype, o, v, n, vec);
        return;
    }
    put_weights8(ph->master, ph->res_out, ph->res_dtype, o, v, n, vec, ph->decay, ph->step);
}

// eight sums of one row from column `col`, to where they belong
__device__ __forceinline__ void put_results(const Results& r, const Phase& ph, int row, int col, uint32_t at, const Addend& x, Eight& u)
{
    u.combine(pack2(r.alpha, r.alpha), pack2(r.beta, r.beta), x);
    if (r.res == RES_PLANES) {
        put_planes8(u, r.hi + at, r.lo != nullptr ? r.lo + at : nullptr);
    } else {
        put_last(&ph, row, col, u);
    }
}

// 32 columns of this warp's 32 rows of sums, one row a thread
template <int BN, bool JOINT>
__device__ __forceinline__ void load_sums(uint32_t tmem, float (&v)[32])
{
    tmem_load32(tmem, v);
    if (JOINT) {
        float w[32];
        tmem_load32(tmem + BN, w);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += w[i];
    }
}

__device__ __forceinline__ void smem_put(uint32_t addr, float a, float b, float c, float d)
{
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ float4 smem_get(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The results of a whole tile, by eight warps: `quarter` the 32 TMEM lanes
// (rows) this one may read, `half` its half of the columns.  A lane of TMEM is
// a row; memory wants whole rows side by side.  32 x 32 sums at a time turn in
// shared memory (16-byte chunks, swizzled by the row: chunk i of row l at
// l * 128 + (i ^ l % 8) * 16): lane l then has the columns 8 (l % 4) + .. of the
// rows l / 4 + 8 i.  What the results need from memory is loaded before the
// sums.  turn: the buffer, on 128 bytes.
template <int BN, bool JOINT>
__device__ __forceinline__ void tile_results(const Results& r, const Phase& ph, const Tile& tl, uint32_t tmem, int quarter,
                                             int half, int lane, uint32_t turn)
{
    const int row0 = tl.m0 + quarter * 32 + lane / 4;
    const uint32_t down = 8 * r.ld;
    const uint32_t in = turn + lane * 128 + (lane & 7) * 16;
    const uint32_t out = turn + lane / 4 * 128 + ((lane % 4 * 2) ^ (lane / 4)) * 16;
    int col = tl.n0 + half * (BN / 2) + lane % 4 * 8;
    uint32_t at = static_cast<uint32_t>(row0) * r.ld + col;
#pragma unroll 1
    for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32, col += 32, at += 32) {
        if (tl.n0 + c >= r.n) break;
        Addend x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r.load(row0 + 8 * i < r.m && col < r.n, at + i * down, x[i]);
        __syncwarp();
        constexpr int kAt = JOINT ? 16 : 32;   // sums at a time: two accumulators' 32 would spill
#pragma unroll
        for (int h = 0; h < 32 / kAt; ++h) {
            float v[kAt];
            if constexpr (JOINT) {
                tmem_sum16(tmem + c + 16 * h, tmem + BN + c + 16 * h, v);
            } else {
                tmem_load32(tmem + c, v);
            }
#pragma unroll
            for (int i = 0; i < kAt / 4; ++i)
                smem_put(in ^ (64 * h + 16 * i), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Eight u;
            u.set(smem_get(out + 1024 * i), smem_get((out ^ 16) + 1024 * i));
            if (row0 + 8 * i < r.m && col < r.n) put_results(r, ph, row0 + 8 * i, col, at + i * down, x[i], u);
        }
    }
}

// One part's share of a tile whose depth is split: the sums of all parts, in
// their order, for BN / 8 / split groups of eight columns.  `parts` is the
// first part's [group][row][8], the next one lies `apart` of those further on;
// t: this thread of 256.
constexpr int kMaxSplit = 8;
template <int BN>
__device__ __forceinline__ void split_results(const Results& r, const Phase& ph, const Tile& tl, const float* parts, int part,
                                              int split, int apart, int t)
{
    const int units = BN / 8 / split;
#pragma unroll 1
    for (int i = t; i < units * kBM; i += kEpiWarps * 32) {
        const int unit = part * units + i % units, k = i / units;
        const int row = tl.m0 + k, col = tl.n0 + 8 * unit;
        if (row >= r.m || col >= r.n) continue;
        const uint32_t at = static_cast<uint32_t>(row) * r.ld + col;
        Addend x;
        r.load(true, at, x);
        const float4* p = reinterpret_cast<const float4*>(parts + unit * (kBM * 8) + k * 8);
        Eight u;
        u.set(make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        for (int q = 0; q < split; q += 2) {   // an even number of parts
            Eight y, z;
            y.set(__ldcg(p), __ldcg(p + 1));
            p += apart * (kBM * BN / 4);
            z.set(__ldcg(p), __ldcg(p + 1));
            p += apart * (kBM * BN / 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) u.v[e] = add2(add2(u.v[e], y.v[e]), z.v[e]);
        }
        put_results(r, ph, row, col, at, x, u);
    }
}

// Wait until *count, which others raise, reaches target; false (and an abort)
// when the limit ran out or one of them gave up.
__device__ __forceinline__ bool wait_count(unsigned* count, unsigned target, volatile int* abort_flag,
                                           unsigned long long timeout_ns)
{
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        if (v & kPoison) break;
        if (v >= target) return true;
        if ((it & 63u) == 63u && (*abort_flag || globaltimer_ns() - t0 > timeout_ns)) break;
    }
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ void raise_count(unsigned* count)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
}

// ------------------------------------------------- norms and first operands
struct PrepArgs {
    const void* in;
    int dtype, vec;
    long long ld, stride;
    int rows, cols, chunks;      // chunks: groups of eight columns in a row
    float4* parts;               // [batch][gridDim.x] sums of squares
    unsigned* counters;          // cleared for the products' kernel
    int n_counters;
};

__device__ __forceinline__ void clear_counters(unsigned* c, int n)
{
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < n; i += blockDim.x) c[i] = 0;
}

// The sums of squares of every matrix, a partial sum for each CTA.  Reads the
// input once: 4096 x 14336 bf16 in 28 us (4.2 TB/s, 1% of the call), 12 x 768 x
// 768 in 6 us.  Four loads under way a thread cost registers and were slower
// (43 and 9 us).
__global__ void __launch_bounds__(256) ns_sqnorm(const __grid_constant__ PrepArgs a)
{
    __shared__ float4 red[8];
    pdl_wait();
    clear_counters(a.counters, a.n_counters);
    const uint32_t total = static_cast<uint32_t>(a.rows) * a.chunks;
    const long long base = blockIdx.y * a.stride;
    SquareSum s;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
        const uint32_t row = i / static_cast<uint32_t>(a.chunks);
        float v[8];
        load_row8(a.in, a.dtype, a.vec, base + row * a.ld, a.cols, i - row * a.chunks, v);
        s.add8(v);
    }
    const float4 sums = block_sums(s.value(), red);
    if (threadIdx.x == 0) a.parts[blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x] = sums;
}

// Dynamic loss scaling: flags a step in which an averaged gradient is not finite,
// before anything of it is written.  Reads the ranks' gradients once: 2 x 4096 x
// 4096 over four ranks in 53 us (268 MB, 5 TB/s), 768 x 2304 over eight in 10 us;
// only calls with loss scaling launch it.
__global__ void __launch_bounds__(256) muon_check(const __grid_constant__ MuonArgs a)
{
    pdl_wait();
    if (muon_skips(a)) return;
    const MuonMean mean(a);
    bool bad = false;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i * 8u < a.elems; i += gridDim.x * 256) {
        const uint32_t left = a.elems - 8 * i;
        float g[8];
        rank_sums8(a, blockIdx.y * a.stride + 8ll * i, left < 8 ? static_cast<int>(left) : 8, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) bad |= !is_finite_f32(mean.of(g[e]));
    }
    if (bad) atomicOr(&a.sc->nonfinite, 1);
}

// The update direction of every matrix, with the sums of its squares: reads the
// ranks' gradients and the momentum once, writes the momentum and the direction
// in fp32.  Bound by memory: 2 x 4096 x 4096 over four ranks in 98 us (6.8
// TB/s, 1.7% of the step); 768 x 2304 over eight ranks, 50 MB, in 15 us.
__global__ void __launch_bounds__(256) muon_direction(const __grid_constant__ MuonArgs a)
{
    __shared__ float4 red[8];
    pdl_wait();
    if (muon_skips(a)) return;
    const MuonMean mean(a);
    clear_counters(a.counters, a.n_counters);
    SquareSum s;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i * 8u < a.elems; i += gridDim.x * 256) {
        float u[8];
        muon_direction8(a, mean, blockIdx.y, i, u);
        s.add8(u);
    }
    const float4 sums = block_sums(s.value(), red);
    if (threadIdx.x == 0) a.parts[blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x] = sums;
}

// ------------------------------------------------------------ the products
// JOINT (three products): a stage holds both planes of both operands, and the
// small products lo*hi + hi*lo have an accumulator of their own, so that the
// large one is added to no more often than with one product (each addition
// drops low bits).  Otherwise a stage holds one plane of each, and three
// products are three passes over the depth, the small ones first.
// CG = 2: a pair of CTAs shares a tile of 256 rows.  Each brings its 128 rows
// of A and half of B's, and holds its rows' sums.  An SM takes 64 bytes a clock
// from L2, and a 64-deep stage's MMAs keep its tensor core busy for 2 BN clocks
// (three times that JOINT).  Alone, a 128 x 128 tile's stage (32 KB) takes 512
// clocks to arrive for 256 of MMAs, JOINT 1007 for 768, a 128 x 256 tile's 690
// to 750 for 512; a pair's 256 x 256 tile brings 32 KB a CTA for 512 clocks of
// MMAs, and measures 518.
//
// The forms, us for the whole five steps (timed side by side, cold L2):
//                           one CTA 128    pair 128    pair 256
//     24 x 384 x 384             135         167         183
//     4 x 1024 x 1024            182         227         205
//     12 x 768 x 768             231         231         229
//     12 x 768 x 768, three      363         325         370
//     2048 x 2048, three         455         396         518
//     4096 x 4096               1362        1306         939
// A 128 x 256 tile of one CTA was slower than the best of these everywhere, so
// there is none.
template <int CG, int BN, bool JOINT>
struct MmShape {
    static constexpr int kABytes = kBM * kBK * 2, kBBytes = BN / CG * kBK * 2;
    static constexpr int kStageBytes = (kABytes + kBBytes) * (JOINT ? 2 : 1);
    static constexpr int kRing = 192 * 1024;
    static constexpr int kStages = kRing / kStageBytes;
    static constexpr int kAccCols = BN * (JOINT ? 2 : 1);   // of one of the two TMEM buffers
    static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kTurnBytes + 1024;   // + alignment of the ring
    static constexpr int kSb = sym_block(CG, BN);
};

// Phase `kind` (0: G = x x^T, 1: P = b G + c G G, 2: x <- a x + P x) of step s
// of matrix b.
template <int CG, int BN>
__device__ __forceinline__ void set_phase(Phase& ph, const NsKernelArgs& a, int s, int kind, int b, const unsigned (&done)[3])
{
    const DevPlanes& xi = a.x[s & 1];
    const DevPlanes& xo = a.x[(s & 1) ^ 1];
    const CUtensorMap* xm = a.xmap[s & 1];
    constexpr int SB = sym_block(CG, BN), BM = kBM * CG;
    const bool last = s + 1 == a.steps;
    ph.lower = kind < 2;
    ph.res = RES_PLANES;
    ph.alpha = kInvScale;
    ph.beta = 0.0f;
    ph.add_hi = ph.add_lo = nullptr;
    if (kind == 0) {
        ph.a = ph.b = xm;
        ph.a_mode = ph.b_mode = a.wide ? kMajorK : kMajorMN;
        ph.m = ph.n = a.m;
        ph.k = a.wide ? a.cols : a.rows;
        ph.out = a.g;
    } else if (kind == 1) {
        ph.a = ph.b = a.gmap;
        ph.a_mode = ph.b_mode = kSymLower;
        ph.m = ph.n = ph.k = a.m;
        ph.alpha = a.coef[s][2] * kInvScale;
        ph.beta = a.coef[s][1];
        ph.add_hi = a.g.hi + b * a.g.stride;
        ph.add_lo = a.g.lo != nullptr ? a.g.lo + b * a.g.stride : nullptr;
        ph.out = a.p;
    } else {
        ph.a = a.wide ? a.pmap : xm;
        ph.b = a.wide ? xm : a.pmap;
        ph.a_mode = a.wide ? kSymLower : kMajorK;
        ph.b_mode = a.wide ? kMajorMN : kSymLower;
        ph.m = a.rows;
        ph.n = a.cols;
        ph.k = a.m;
        ph.beta = a.coef[s][0];
        ph.add_hi = xi.hi + b * xi.stride;
        ph.add_lo = xi.lo + b * xi.stride;
        ph.out = xo;
        if (last) {   // x itself leaves: scaled back
            ph.res = a.res;
            ph.alpha *= kInvScale;
            ph.beta *= kInvScale;
            ph.res_dtype = a.out_dtype;
            ph.res_vec = a.out_vec;
            ph.res_ld = a.out_ld;
            ph.decay = a.decay;
            ph.step = a.step;
            const long long at = b * a.out_stride;
            if (a.res == RES_MUON) {
                ph.master = a.master + at;
                ph.res_out = a.lp != nullptr ? static_cast<uint16_t*>(a.lp) + at : nullptr;
            } else {
                ph.res_out = static_cast<char*>(a.out) + at * (a.out_dtype == ZERO_FP32 ? 4 : 2);
            }
        }
    }
    ph.out.hi += b * ph.out.stride;
    if (ph.out.lo != nullptr) ph.out.lo += b * ph.out.stride;
    ph.tiles_m = (ph.m + BM - 1) / BM;
    ph.tiles_n = (ph.n + BN - 1) / BN;
    const int blocks = (a.m + SB - 1) / SB;
    const int sym = (SB / BM) * (SB / BN) * (blocks * (blocks + 1) / 2);
    const int up = ((a.rows + BM - 1) / BM) * ((a.cols + BN - 1) / BN);
    ph.tiles = ph.lower ? sym : up;
    ph.split = a.split[kind];
    // a tile's counter has been raised by every earlier phase that had the tile
    const int unit = blockIdx.x % a.ctas / CG, t = unit / ph.split;
    ph.tile_target = ph.split;
    for (int q = 0; q < 3; ++q)
        if (a.split[q] > 1 && t < (q < 2 ? sym : up)) ph.tile_target += done[q] * a.split[q];
    const int first = ph.split > 1 ? t : unit;
    if (first < ph.tiles) ph.first = tile_of<CG, BN>(ph, first);
}

// x_0 = g / (|g| + eps) of matrix b, scaled, as a pair: this CTA's part.  Once
// a matrix, so kept out of the phases' registers.
__device__ __noinline__ void first_operand(const NsKernelArgs& a, int b, int cta, float4* red, float* shared_scale)
{
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = threadIdx.x; i < a.parts_n; i += kThreads) add_sums(q, a.parts[static_cast<long long>(b) * a.parts_n + i]);
    const float f = block_scale(block_sums(q, red), a.eps, shared_scale);
    const uint32_t chunks = a.chunks, total = static_cast<uint32_t>(a.rows) * chunks, stride = a.ctas * kThreads;
    const void* in = a.in;
    const int dtype = a.in_dtype, cols = a.cols;
    const bool vec = a.in_vec;
    const long long base = b * a.in_stride, ld = a.in_ld, out_ld = a.x[0].ld;
    __half* hi = a.x[0].hi + b * a.x[0].stride;
    __half* lo = a.x[0].lo + b * a.x[0].stride;
    for (uint32_t i = cta * kThreads + threadIdx.x; i < total; i += 4 * stride) {   // four loads under way
        float v[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t j = i + k * stride, row = j / chunks;
            if (j < total) load_row8(in, dtype, vec, base + row * ld, cols, j - row * chunks, v[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t j = i + k * stride, row = j / chunks;
            if (j >= total) break;
            Eight u;
            u.set(make_float4(v[k][0], v[k][1], v[k][2], v[k][3]), make_float4(v[k][4], v[k][5], v[k][6], v[k][7]));
            u.scale(pack2(f, f));
            const long long o = row * out_ld + 8 * (j - row * chunks);
            put_planes8(u, hi + o, lo + o);
        }
    }
}

// The whole iteration in one launch.  The grid is `groups` of `ctas` CTAs, all
// resident (a cooperative launch); a group takes its matrices one after the
// other and meets at a counter in memory between products.  Within a product
// the CTAs (CG = 2: the pairs) share the tiles, or, where there are fewer
// tiles than units, each tile's depth (its parts meet at a counter of the tile
// and each adds up its share of the columns, in order).  Within a CTA one warp
// keeps a ring of 64-deep operand tiles full by TMA, one issues the MMAs into
// one of two TMEM accumulators, eight turn the other one into results, and one
// works out the next phase meanwhile (0.4 us that would stand between two
// products).
//
// What the clocks go to beside the MMAs, in a phase: about 1k for the block's
// barrier and the release, 2 to 4k for the meeting, 2.2k until the first stage
// is there, 3.4 to 6.1k for the results of a 128 x 128 tile of a CTA, 6.8 to
// 13k for 128 x 256 (the upper figures beside the next tile's MMAs), 13k for an
// exchange of partial sums.  The results are bound by latency: a 32 x 32 piece
// takes 1.2 to 2k clocks whether it leaves by plain stores or by TMA.  Sixteen
// warps for them left 96 registers a thread, which spilled: 20 to 40% slower
// everywhere; so did loading a piece's addends ahead.
template <int CG, int BN, bool JOINT>
__global__ void __launch_bounds__(kThreads, 1) ns_kernel(const __grid_constant__ NsKernelArgs a)
{
    using S = MmShape<CG, BN, JOINT>;
    if (a.guarded && *reinterpret_cast<volatile int*>(&a.sc->nonfinite) != 0) return;   // the same for every thread
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;
    __shared__ Phase plan[2];
    __shared__ int stop_flag;
    __shared__ float4 red[kThreads / 32];
    __shared__ float shared_scale;
    unsigned char* ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023u)) % 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x / a.ctas, cta = blockIdx.x % a.ctas;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0, unit = cta / CG, units = a.ctas / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kEpiWarps * CG);
        }
        mbar_init(&drain, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<CG>(&tmem_base, 2 * S::kAccCols);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) pair_sync();   // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    const uint32_t turn = smem_u32(ring) + S::kStages * S::kStageBytes + (warp - 2) * kTurnBytes;   // of the epilogue warps

    // where the roles are in the ring and the accumulators, over all phases
    Slot<S::kStages> slot;
    Slot<2> acc;
    uint32_t count = 0;          // producer: stages issued; MMA: accumulators begun
    unsigned met = 0;            // thread 0's: arrivals at the group's meetings
    unsigned done[3] = {0, 0, 0};   // the planning thread's: phases of each kind
    bool stop = false;
    int turn_of = 0;             // which of the two plans is the phase's
    if (threadIdx.x == kThreads - 32) {
        set_phase<CG, BN>(plan[0], a, 0, 0, group, done);
        ++done[0];
    }

    for (int b = group; b < a.batch && !stop; b += a.groups) {
        first_operand(a, b, cta, red, &shared_scale);
        for (int phase = 0; phase < 3 * a.steps; ++phase) {
            // the group's results of the phase before, for everyone's TMA loads
            // (the barrier orders this CTA's before thread 0's release)
            fence_proxy_async_global();
            __syncthreads();
            if (threadIdx.x == 0) {
                met += a.ctas;
                if (a.ctas > 1) {
                    if (abort_flag) {
                        atomicOr(a.group_bar + group * kBarStride, kPoison);
                    } else {
                        raise_count(a.group_bar + group * kBarStride);
                        wait_count(a.group_bar + group * kBarStride, met, &abort_flag, a.timeout_ns);
                    }
                }
                stop_flag = abort_flag;
            }
            __syncthreads();
            if (stop_flag) {   // the same for every thread
                stop = true;
                break;
            }
            const Phase& ph = plan[turn_of];
            turn_of ^= 1;

            const int first = ph.split > 1 ? unit / ph.split : unit, step = ph.split > 1 ? INT_MAX / 2 : units;
            const int part = ph.split > 1 ? unit % ph.split : 0;
            const int stages = (ph.k + kBK - 1) / kBK;
            const int k_from = stages * part / ph.split * kBK, k_to = stages * (part + 1) / ph.split * kBK;
            const int pass0 = JOINT ? 2 : 3 - a.products;

            if (warp == kThreads / 32 - 1) {
                // the next phase, of this matrix or of the group's next one
                if (lane == 0) {
                    const int next = phase + 1 < 3 * a.steps ? phase + 1 : 0;
                    set_phase<CG, BN>(plan[turn_of], a, next / 3, next % 3, next > 0 ? b : b + a.groups, done);
                    ++done[next % 3];
                }
                __syncwarp();
            } else if (warp == 0) {
                // Whole warps walk these two loops, one lane of them issues: what
                // the issued instructions need is then the same in all lanes and
                // stays in uniform registers.
                fence_proxy_async_global();
                bool ok = true;
                for (int t = first; ok && t < ph.tiles; t += step) {
                    const Tile tl = t == first ? ph.first : tile_of<CG, BN>(ph, t);
                    const int am = mn_from(ph.a_mode, S::kSb, tl.m0), bm = mn_from(ph.b_mode, S::kSb, tl.n0);
                    const int m0 = tl.m0 + rank * kBM, n0 = tl.n0 + rank * (BN / CG);   // this CTA's share
                    for (int pass = pass0; ok && pass < 3; ++pass) {
                        const CUtensorMap* ma = ph.a + (pass == 0);
                        const CUtensorMap* mb = ph.b + (pass == 1);
                        for (int k0 = k_from; k0 < k_to; k0 += kBK) {
                            if (count >= S::kStages &&
                                !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[slot.i], slot.parity ^ 1, &abort_flag, a.timeout_ns))) {
                                abort_flag = 1;
                                ok = false;
                                break;
                            }
                            if (!a.starve && elect_one()) {
                                unsigned char* p = ring + slot.i * S::kStageBytes;
                                uint64_t* bar = &full[slot.i];
                                // the leader's barrier counts both CTAs' bytes
                                if (rank == 0) mbar_arrive_expect_tx(bar, CG * S::kStageBytes);
                                load_operand<CG, kBM / kBox>(p, ma, k0 >= am, m0, k0, b, bar);
                                load_operand<CG, BN / CG / kBox>(p + S::kABytes, mb, k0 >= bm, n0, k0, b, bar);
                                if (JOINT) {
                                    p += S::kABytes + S::kBBytes;
                                    load_operand<CG, kBM / kBox>(p, ma + 1, k0 >= am, m0, k0, b, bar);
                                    load_operand<CG, BN / CG / kBox>(p + S::kABytes, mb + 1, k0 >= bm, n0, k0, b, bar);
                                }
                            }
                            __syncwarp();
                            slot.next();
                            ++count;
                        }
                    }
                }
            } else if (warp == 1) {
                const uint32_t ring_at = smem_u32(ring);
                bool ok = rank == 0;   // a pair's leader issues for both
                for (int t = first; ok && t < ph.tiles; t += step) {
                    const Tile tl = t == first ? ph.first : tile_of<CG, BN>(ph, t);
                    const int am = mn_from(ph.a_mode, S::kSb, tl.m0), bm = mn_from(ph.b_mode, S::kSb, tl.n0);
                    if (count >= 2 && !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&acc_empty[acc.i], acc.parity ^ 1, &abort_flag, a.timeout_ns))) {
                        abort_flag = 1;
                        break;
                    }
                    ++count;
                    tc_fence_after();
                    const uint32_t d = tmem + acc.i * S::kAccCols;
                    uint32_t more = 0;   // 0: the accumulator starts anew
                    for (int pass = pass0; ok && pass < 3; ++pass) {
                        for (int k0 = k_from; k0 < k_to; k0 += kBK) {
                            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[slot.i], slot.parity, &abort_flag, a.timeout_ns))) {
                                abort_flag = 1;
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const bool a_mn = k0 >= am, b_mn = k0 >= bm;
                            const uint32_t idesc = instr_desc(kBM * CG, BN, a_mn, b_mn);
                            const uint32_t p = ring_at + slot.i * S::kStageBytes;
                            const uint32_t da = smem_desc_lo(p), db = smem_desc_lo(p + S::kABytes);
                            // sixteen values of depth: 32 bytes along a line, or sixteen lines
                            const uint32_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sb = b_mn ? 2048 >> 4 : 32 >> 4;
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < kBK / 16; ++k) {
                                    mma_f16<CG>(d, da + k * sa, db + k * sb, idesc, k > 0 ? 1u : more);
                                    if (JOINT) {
                                        constexpr uint32_t kLo = (S::kABytes + S::kBBytes) >> 4;
                                        mma_f16<CG>(d + BN, da + kLo + k * sa, db + k * sb, idesc, k > 0 ? 1u : more);
                                        mma_f16<CG>(d + BN, da + k * sa, db + kLo + k * sb, idesc, 1u);
                                    }
                                }
                                mma_commit<CG>(&empty[slot.i]);
                            }
                            __syncwarp();
                            more = 1;
                            slot.next();
                        }
                    }
                    if (ok && elect_one()) mma_commit<CG>(&acc_full[acc.i]);
                    __syncwarp();
                    acc.next();
                }
            } else {
                const int quarter = warp & 3;         // the TMEM lanes this warp may read
                const int half = (warp - 2) >> 2;     // its half of the columns
                const Results res(ph);
#pragma unroll 1
                for (int t = first; t < ph.tiles; t += step) {
                    Tile tl = t == first ? ph.first : tile_of<CG, BN>(ph, t);
                    tl.m0 += rank * kBM;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&acc_full[acc.i], acc.parity, &abort_flag, a.timeout_ns))) {
                        abort_flag = 1;
                        if (ph.split == 1) break;
                        // the other warps of the CTA still meet below
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + acc.i * S::kAccCols + (static_cast<uint32_t>(quarter * 32) << 16);
                    if (ph.split == 1) {
                        tile_results<BN, JOINT>(res, ph, tl, d, quarter, half, lane, turn);
                    } else {
                        // this part's sums, [group of eight columns][row][8]
                        float* mine = a.partial + static_cast<long long>(blockIdx.x) * (kBM * BN) + (quarter * 32 + lane) * 8;
#pragma unroll 1
                        for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
                            float v[32];
                            load_sums<BN, JOINT>(d + c, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                __stcg(reinterpret_cast<float4*>(mine + (c / 8 + i / 2) * (kBM * 8)) + (i & 1),
                                       make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2)
                            mbar_arrive_leader(&acc_empty[acc.i]);
                        else
                            mbar_arrive(&acc_empty[acc.i]);
                    }
                    acc.next();
                    if (ph.split == 1) continue;
                    // the tile's parts meet, then each adds up its columns (the
                    // barrier orders this CTA's sums before the release)
                    named_bar_sync(1, kEpiWarps * 32);
                    if (threadIdx.x == 64 && !abort_flag) {
                        unsigned* bar = a.tile_bar + group * a.ctas + t * CG + rank;
                        raise_count(bar);
                        wait_count(bar, ph.tile_target, &abort_flag, a.timeout_ns);
                    }
                    named_bar_sync(1, kEpiWarps * 32);
                    if (abort_flag) break;
                    split_results<BN>(res, ph, tl, a.partial + static_cast<long long>(blockIdx.x - part * CG) * (kBM * BN), part,
                                      ph.split, CG, threadIdx.x - 64);
                }
            }
        }
    }
    __syncthreads();
    if (CG == 2) pair_sync();   // neither issues anything any more
    if (warp == 0) {
        if (lane == 0 && rank == 0 && abort_flag && !a.starve) {
            // nothing of ours (nor, counted here, of the other CTA's) may still
            // be landing when the memory goes away
            for (uint32_t i = count > S::kStages ? count - S::kStages : 0; i < count; ++i)
                mbar_wait_bounded(&full[i % S::kStages], (i / S::kStages) & 1, nullptr, 1000000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // TMEM and the barriers are given up only after the last MMA
        if (rank == 0 && elect_one()) mma_commit<CG>(&drain);
        __syncwarp();
        mbar_wait_bounded(&drain, 0, nullptr, 1000000000ull);
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) pair_sync();
    tc_fence_after();
    if (warp == 1) tmem_free<CG>(tmem, 2 * S::kAccCols);
    if (threadIdx.x == 0 && abort_flag && a.sc != nullptr) atomicOr(&a.sc->status, ZERO_DEV_TIMEOUT);
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

// How a call is cut up.
struct Plan {
    int cg, bn, joint;
    int groups, ctas;
    int split[3];
    double us;
};

// Times of a CTA or a pair, in us, that the choice goes by, fitted to shapes
// timed in each form.  Of 32 calls (sixteen shapes from 256 x 256 to 4096 x 4096,
// one and three products) timed in every form side by side, the chosen form is the
// best or within 1% of it for 27 and within 4% for all (single matrices of 512 to
// 1024 with three products, where the pair form 128 wide is 2 to 4% faster): a
// 64-deep stage, the results of a tile beside the next tile's products
// and alone at the end, the same with an exchange of partial sums, the meeting
// of a group and the first copies after it.
struct Costs {
    double stage, results, end, split_end, meet, alone;
};
Costs costs_of(int cg, int bn, int joint)
{
    if (cg == 1) return {joint ? 0.53 : 0.27, 4.6, 3.0, 7.0, 3.2, 2.2};
    if (bn == 256) return {0.29, 6.5, 5.0, 14.0, 3.9, 2.9};
    return {joint ? 0.41 : 0.21, 5.2, 3.4, 7.4, 3.9, 2.9};
}

long long sym_tiles(int m, int cg, int bn)
{
    const int sb = sym_block(cg, bn);
    const long long blocks = (m + sb - 1) / sb;
    return static_cast<long long>(sb / (kBM * cg)) * (sb / bn) * (blocks * (blocks + 1) / 2);
}
long long all_tiles(int rows, int cols, int cg, int bn)
{
    return static_cast<long long>((rows + kBM * cg - 1) / (kBM * cg)) * ((cols + bn - 1) / bn);
}

// the time of one product with `tiles` tiles and `stages` stages each on
// `units` CTAs or pairs, and how many of them share a tile
double phase_us(long long tiles, int stages, const Costs& c, int passes, int units, int& split)
{
    const double mma = stages * passes * c.stage;
    const long long rounds = (tiles + units - 1) / units;
    double best = mma + (rounds - 1) * (mma > c.results ? mma : c.results) + c.end;
    split = 1;
    for (int q = 2; q <= kMaxSplit && q <= stages && tiles * q <= units; q *= 2) {
        const double us = static_cast<double>((stages + q - 1) / q) * passes * c.stage + c.split_end;
        if (us < best) best = us, split = q;
    }
    return best;
}

Plan plan_of(int rows, int cols, int batch, int products, int sms)
{
    const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    Plan best;
    std::memset(&best, 0, sizeof(best));
    for (int kind = 0; kind < 3; ++kind) {
        Plan p;
        p.cg = kind == 0 ? 1 : 2;
        p.bn = kind == 2 ? 256 : 128;
        p.joint = p.bn == 128 && products == 3;
        const Costs c = costs_of(p.cg, p.bn, p.joint);
        const int passes = p.joint ? 1 : products;
        const long long sym = sym_tiles(m, p.cg, p.bn), up = all_tiles(rows, cols, p.cg, p.bn);
        const int all = sms / p.cg;
        int last = 0;
        for (p.groups = 1; p.groups <= batch && p.groups <= all; ++p.groups) {
            const int turns = (batch + p.groups - 1) / p.groups;
            if (turns == last) continue;   // the same with smaller groups
            last = turns;
            for (int alone = 0; alone < 2; ++alone) {
                // as they are, then a unit alone: without the meetings
                const int units = alone ? 1 : all / p.groups;
                p.ctas = units * p.cg;
                const double us = phase_us(sym, (n + kBK - 1) / kBK, c, passes, units, p.split[0]) +
                                  phase_us(sym, (m + kBK - 1) / kBK, c, passes, units, p.split[1]) +
                                  phase_us(up, (m + kBK - 1) / kBK, c, passes, units, p.split[2]);
                p.us = turns * (us + 3 * (units > 1 ? c.meet : c.alone));
                if (best.bn == 0 || p.us < best.us) best = p;
            }
        }
    }
    long long most = 0;
    for (int q = 0; q < 3; ++q) {
        const long long tiles = q < 2 ? sym_tiles(m, best.cg, best.bn) : all_tiles(rows, cols, best.cg, best.bn);
        if (most < tiles * best.split[q]) most = tiles * best.split[q];
    }
    if (most * best.cg < best.ctas) best.ctas = static_cast<int>(most) * best.cg;   // CTAs that would only wait
    return best;
}

struct Layout {
    size_t parts, counters, partial, u, x[2], g, p, end;
    long long x_plane, s_plane;   // elements of one plane
    int planes;
};

constexpr int kMaxSms = 160;      // GB300 has 152

// CTAs that take a matrix's norm: `want` of them, but no more than eight an SM
// over the batch
int parts_of(int batch, long long want, int sms)
{
    const long long most = (8LL * sms + batch - 1) / batch;
    if (want > most) want = most;
    return static_cast<int>(want < kMaxNsParts ? want : kMaxNsParts);
}

Layout layout_of(int rows, int cols, int batch, int products, bool muon)
{
    Layout l;
    const long long m = rows < cols ? rows : cols;
    l.planes = products == 3 ? 2 : 1;
    l.x_plane = static_cast<long long>(batch) * rows * up64(cols);
    l.s_plane = static_cast<long long>(batch) * m * up64(m);
    size_t at = 0;
    l.counters = at;
    at += up256(static_cast<size_t>(kMaxSms) * (kBarStride + 1) * sizeof(unsigned));
    l.parts = at;
    at += up256(static_cast<size_t>(batch) * parts_of(batch, kMaxNsParts, kMaxSms) * sizeof(float4));
    l.partial = at;
    at += static_cast<size_t>(kMaxSms) * kBM * 256 * sizeof(float);
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
    return n < kMaxSms ? n : kMaxSms;
}

template <int CG, int BN, bool JOINT>
cudaError_t launch_ns_as(const NsKernelArgs& a, cudaStream_t st)
{
    constexpr int smem = MmShape<CG, BN, JOINT>::kSmem;
    const auto k = ns_kernel<CG, BN, JOINT>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c;
    std::memset(&c, 0, sizeof(c));
    c.gridDim = dim3(a.groups * a.ctas);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    c.attrs = at;
    if (CG == 2) {
        at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[c.numAttrs].val.clusterDim.x = 2;
        at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
        ++c.numAttrs;
    }
    if (a.ctas > CG) {   // CTAs that wait for one another are resident together
        at[c.numAttrs].id = cudaLaunchAttributeCooperative;
        at[c.numAttrs].val.cooperative = 1;
        ++c.numAttrs;
    }
    count_launch();
    return cudaLaunchKernelEx(&c, k, a);
}

cudaError_t launch_products(const Plan& p, const NsKernelArgs& a, cudaStream_t st)
{
    if (p.cg == 1) return p.joint ? launch_ns_as<1, 128, true>(a, st) : launch_ns_as<1, 128, false>(a, st);
    if (p.bn == 256) return launch_ns_as<2, 256, false>(a, st);
    return p.joint ? launch_ns_as<2, 128, true>(a, st) : launch_ns_as<2, 128, false>(a, st);
}

bool set_planes(DevPlanes& d, CUtensorMap* maps, const Planes& p, int batch)
{
    d.hi = p.hi;
    d.lo = p.lo;
    d.ld = p.ld;
    d.stride = p.stride;
    return encode(&maps[0], p, p.hi, batch) && (p.lo == nullptr || encode(&maps[1], p, p.lo, batch));
}

}  // namespace

size_t ns_workspace_bytes(int rows, int cols, int batch, int products, bool muon)
{
    return layout_of(rows, cols, batch, products, muon).end;
}

void ns_plan(int rows, int cols, int batch, int products, int sms, zero_matrix_plan* out)
{
    std::memset(out, 0, sizeof(*out));
    out->products = products;
    if (small_ns_fits(rows, cols, products)) {
        out->groups = batch;
        return;
    }
    const Plan p = plan_of(rows, cols, batch, products, sms < kMaxSms ? sms : kMaxSms);
    out->tile_rows = kBM * p.cg;
    out->tile_cols = p.bn;
    out->groups = p.groups;
    out->units = p.ctas / p.cg;
    std::memcpy(out->split, p.split, sizeof(out->split));
}

#define ZK_GO(expr)                             \
    do {                                        \
        const cudaError_t e_ = (expr);          \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

cudaError_t launch_mm_starved(void* scratch, zero_dev_scalars* sc, unsigned long long timeout_ns, cudaStream_t st)
{
    // one 64 x 64 matrix: its planes in the scratch are never read or written
    // (the input is empty)
    NsKernelArgs k;
    std::memset(&k, 0, sizeof(k));
    const Planes p = planes_at(scratch, 0, 64 * 64, 64, 64, false);
    k.rows = k.cols = k.m = 64;
    k.wide = k.batch = k.steps = k.products = k.groups = k.ctas = k.split[0] = k.split[1] = k.split[2] = 1;
    k.eps = 1.0f;
    k.sc = sc;
    k.starve = 1;
    k.timeout_ns = timeout_ns;
    if (!set_planes(k.x[0], k.xmap[0], p, 1) || !set_planes(k.g, k.gmap, p, 1)) return cudaErrorInvalidValue;
    Plan plan;
    std::memset(&plan, 0, sizeof(plan));
    plan.cg = 1;
    plan.bn = 128;
    return launch_products(plan, k, st);
}

cudaError_t launch_ns(const NsArgs& a, cudaStream_t st)
{
    const bool muon = a.out == nullptr, wide = a.rows <= a.cols;
    const int m = wide ? a.rows : a.cols;
    const Layout l = layout_of(a.rows, a.cols, a.batch, a.products, muon);
    char* ws = static_cast<char*>(a.ws);
    unsigned* counters = reinterpret_cast<unsigned*>(ws + l.counters);
    float4* parts = reinterpret_cast<float4*>(ws + l.parts);
    MuonArgs mu;
    if (muon) {
        std::memset(&mu, 0, sizeof(mu));
        for (int q = 0; q < a.n_d; ++q) mu.rank[q] = a.ranks[q];
        mu.n_d = a.n_d;
        mu.dtype = a.in_dtype;
        mu.nesterov = a.nesterov;
        mu.loss_scaling = a.loss_scaling;
        mu.clipping = a.clipping;
        mu.sc = a.sc;
        mu.divisor = a.divisor;
        mu.mu = a.mu;
        mu.momentum = a.momentum;
        mu.u = reinterpret_cast<float*>(ws + l.u);
        mu.stride = a.flat_stride;
        mu.elems = static_cast<uint32_t>(a.rows) * static_cast<uint32_t>(a.cols);
        mu.u_stride = (static_cast<long long>(mu.elems) + 7) / 8 * 8;
        mu.parts = parts;
        mu.counters = counters;
        mu.n_counters = kMaxSms * (kBarStride + 1);
    }
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    // the norm: CTAs a matrix, four chunks a thread (Muon, with more to load for
    // each: one; 768 x 768 over 16 ranks, the whole step, 218 -> 203 us), eight CTAs an SM over the batch
    const int chunks = (a.cols + 7) / 8, want = muon ? 256 : 1024;
    const int parts_n = parts_of(a.batch, (static_cast<long long>(a.rows) * chunks + want - 1) / want, sms);
    const dim3 grid(static_cast<unsigned>(parts_n), a.batch);
    if (muon && a.loss_scaling) ZK_GO(launch_after(muon_check, grid, dim3(256), 0, st, mu));
    if (small_ns_fits(a.rows, a.cols, a.products)) return launch_small_ns(a, muon ? &mu : nullptr, st);
    const Plan plan = plan_of(a.rows, a.cols, a.batch, a.products, sms);
    NsKernelArgs k;
    std::memset(&k, 0, sizeof(k));
    bool ok = true;
    for (int i = 0; i < 2; ++i) ok = ok && set_planes(k.x[i], k.xmap[i], planes_at(ws, l.x[i], l.x_plane, a.rows, a.cols, true), a.batch);
    ok = ok && set_planes(k.g, k.gmap, planes_at(ws, l.g, l.s_plane, m, m, a.products == 3), a.batch);
    ok = ok && set_planes(k.p, k.pmap, planes_at(ws, l.p, l.s_plane, m, m, a.products == 3), a.batch);
    if (!ok) return cudaErrorInvalidValue;
    k.rows = a.rows;
    k.cols = a.cols;
    k.m = m;
    k.wide = wide;
    k.batch = a.batch;
    k.steps = a.steps;
    k.products = a.products;
    k.groups = plan.groups;
    k.ctas = plan.ctas;
    std::memcpy(k.split, plan.split, sizeof(k.split));
    std::memcpy(k.coef, a.coef, sizeof(k.coef));
    k.chunks = chunks;
    k.eps = a.eps;
    k.parts = parts;
    k.group_bar = counters;
    k.tile_bar = counters + kMaxSms * kBarStride;
    k.partial = reinterpret_cast<float*>(ws + l.partial);
    k.sc = a.sc;
    k.timeout_ns = kDefaultTimeoutNs;

    k.parts_n = parts_n;
    if (muon) {
        k.in = mu.u;
        k.in_dtype = ZERO_FP32;
        k.in_ld = a.cols;
        k.in_stride = mu.u_stride;
        k.in_vec = a.cols % 4 == 0;
        k.res = RES_MUON;
        k.guarded = a.loss_scaling;
        k.master = a.master;
        k.lp = a.lp;
        k.out_dtype = a.lp_dtype;
        k.out_ld = a.cols;
        k.out_stride = a.flat_stride;
        k.out_vec = a.cols % 8 == 0;
        k.decay = a.decay;
        k.step = a.step;
        ZK_GO(launch_after(muon_direction, grid, dim3(256), 0, st, mu));
    } else {
        k.in = a.in;
        k.in_dtype = a.in_dtype;
        k.in_ld = a.in_ld;
        k.in_stride = a.in_stride;
        k.in_vec = wide_rows(a.in, a.in_dtype, a.in_ld, a.in_stride);
        k.res = RES_OUT;
        k.out = a.out;
        k.out_dtype = a.out_dtype;
        k.out_ld = a.out_ld;
        k.out_stride = a.out_stride;
        k.out_vec = wide_rows(a.out, a.out_dtype, a.out_ld, a.out_stride);
        PrepArgs pr;
        std::memset(&pr, 0, sizeof(pr));
        pr.in = k.in;
        pr.dtype = k.in_dtype;
        pr.vec = k.in_vec;
        pr.ld = k.in_ld;
        pr.stride = k.in_stride;
        pr.rows = a.rows;
        pr.cols = a.cols;
        pr.chunks = k.chunks;
        pr.parts = parts;
        pr.counters = counters;
        pr.n_counters = kMaxSms * (kBarStride + 1);
        ZK_GO(launch_after(ns_sqnorm, grid, dim3(256), 0, st, pr));
    }
    return launch_products(plan, k, st);
}

}  // namespace zk
