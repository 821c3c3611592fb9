// zk_norm.cu -- layer norm, forward and backward with the weight gradients.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y = (x - mean) * rstd * gain + bias
//   h = dy * gain,  xhat = (x - mean) * rstd
//   dx = rstd * (h - mean_C(h) - xhat * mean_C(h * xhat))
//   dgain = sum over rows of dy * xhat,  dbias = sum over rows of dy
//
// Every sum is fp32; the results are rounded once, to the tensor's type.  The
// sum of squares is taken about the mean in a second pass over the row (in
// registers), so an offset in x costs the variance no digits.  xhat is
// (x - mean) * rstd for fp32; for 16-bit x, whose own digits end long before, it
// is x * rstd - mean * rstd in one fused operation (the difference costs 16-bit
// rows up to 8% forward, bound by issue as they are, and fp32 rows nothing).
//
// Bound: memory.  Forward reads x and writes y, backward reads x and dy and
// writes dx; at 6788 GB/s (a copy's rate) 8192 x 4096 bf16 cannot take less than
// 19.8 us forward and 29.7 us backward.  Measured, call after call in a graph:
// forward 22.9 us (0.86 of a copy), 16384 x 4096 42.4 us (0.93); backward 16384 x
// 4096 72.8 us (0.81; fp32 131 us, 0.91), its second kernel included.  Next to
// memory it is issue: a CTA of sixteen warps an SM, 53% of the issue slots busy,
// fixed-latency and shared-memory waits in between; every instruction a row fewer
// showed (the root and the division 4 to 9%, addresses kept from row to row 4 to
// 20%).  Few rows are bound by latency: 8 x 768 2.3 us, 256 x 768 backward 6.3 us
// (two kernels, the second's start hidden behind the first).  Rows that do not lie
// on 16-byte words pay for it: 2999 x 1601 fp32 forward 11.6 us alike and 12.1 us
// with unlike gaps (floor 5.7), 5003 x 1601 fp16 backward 21.8 us (floor 7.1).
#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"
#include "zk_rows.cuh"
#include "zk_tc.cuh"

namespace zk {
namespace {

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

// ------------------------------------------------------------- row pipelines
// A row is cut into chunks of 16 bytes (V = 8 or 4 columns).  A group of
// `warps` warps takes R consecutive rows at a time, thread t of the group the
// chunks t, t + width, ... of each (NCH of them); a persistent CTA of `groups`
// groups walks the rows.  A thread's columns never change, so weights and
// column sums stay in registers, and the rows to come are already on their way
// into a ring of DEPTH stages in shared memory (16-byte asynchronous copies).
// Sixteen columns a thread spread what a row costs each thread besides its
// columns (the two sums over the group); a row to a warp, 128 columns a thread,
// left too few loads under way (41 us forward where this takes 25, 70 us
// backward at 8192 x 4096), eight columns a thread and four rows at a time took
// 106 us backward at 16384 x 4096, two rows at a time spilled (139 us).  Values
// stay packed two to a register pair, and operations on pairs (f32x2) halve the
// issue slots.
//
// How the rows lie (MODE):
//   kAligned  bases, strides and the width are multiples of 16 bytes.  A thread
//             fills and empties its own ring slots alone.
//   kAlike    not that, but equal rows of all arrays start equally far into a
//             16-byte word (an odd width without gaps).  A CTA takes rows eight
//             apart, which all start alike, and cuts them where memory's words
//             lie: chunk j holds the columns from V j - first on.  Slots stay
//             private; only a row's first and last word need care.
//   kFours    fp32 rows that lie differently: cut as the results' words lie, the
//             inputs copied four bytes at a time.
//   kMixed    16-bit rows that lie differently: cut as the results' words lie,
//             the inputs' words copied as they lie; a chunk is two of them, its
//             own thread's and the next one's, shifted into place.
enum { kAligned = 0, kAlike = 1, kMixed = 2, kFours = 3 };
__host__ __device__ constexpr bool by_words(int mode) { return mode != kAligned; }
// Where rows begin and end inside a word but slots are private, thread 0 takes
// the last chunk and all others one less: the two chunks that need care are then
// in one warp (16384 x 1601 bf16 backward 52.4 -> 48.8 us).
__host__ __device__ constexpr bool by_turns(int mode) { return mode == kAlike || mode == kFours; }

// 16 bytes from byte `off` (0 .. 15, the same in every thread) of two words
__device__ __forceinline__ uint4 shifted(const uint4& p, const uint4& q, uint32_t off)
{
    uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (off & 2u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The rows of a group: row(k) of the set at r0 is r0 + k * apart.  Groups that
// share a warp (LANES < 32) walk on while the first of them has rows: r0 < end.
template <int MODE, int R, int LANES>
struct Walk {
    static constexpr int apart = by_words(MODE) ? 8 : 1;
    long long r0, step, end;
    __device__ __forceinline__ Walk(int grp, int groups, long long rows)
    {
        end = rows + (LANES < 32 ? grp % (32 / LANES) * R * apart : 0);
        if (by_words(MODE)) {   // gridDim.x is a multiple of 8
            r0 = (blockIdx.x & 7) + 8ll * ((blockIdx.x >> 3) * groups + grp) * R;
            step = 8ll * (gridDim.x >> 3) * groups * R;
        } else {
            r0 = (static_cast<long long>(blockIdx.x) * groups + grp) * R;
            step = static_cast<long long>(gridDim.x) * groups * R;
        }
    }
};

// V weights from column c on, in whichever type they have; `none` without a
// vector, 0 where there is no such column
template <int V>
__device__ __forceinline__ void weights_at(const void* w, int dt, int c, int cols, float none, f32x2 (&v)[V / 2])
{
    float f[V];
    const uintptr_t at = reinterpret_cast<uintptr_t>(w) + static_cast<intptr_t>(c) * (dt == ZERO_FP32 ? 4 : 2);
    if (w != nullptr && c >= 0 && c + V <= cols && at % 16 == 0) {
        if (dt == ZERO_FP32) {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const float4 x = *(reinterpret_cast<const float4*>(at) + e / 4);
                f[e] = x.x, f[e + 1] = x.y, f[e + 2] = x.z, f[e + 3] = x.w;
            }
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(at);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const uint32_t x = p[e];
                f[2 * e] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::lo(x) : Lp<ZERO_FP16>::lo(x);
                f[2 * e + 1] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::hi(x) : Lp<ZERO_FP16>::hi(x);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = c + e < 0 || c + e >= cols ? 0.0f : w == nullptr ? none : weight_at(w, dt, c + e);
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) v[e] = pack2(f[2 * e], f[2 * e + 1]);
}

constexpr int kMaxWarps = 16;   // of a group

// Sums of N values over a group of `warps` warps (LANES < 32: of so many lanes
// of one), the same in all its threads.  Each shuffle step carries as many
// values as are still apart (N = 4: six shuffles for twenty); red: this group's
// kMaxWarps * N floats.
template <int N, int LANES>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red, int warps, int bar, int width, int wg)
{
    static_assert(N == 1 || N == 2 || N == 4 || N == 8, "");
    const int lane = threadIdx.x & 31;
    // halve the values while lanes are left to carry them: the upper lane bits
    // end up naming the value a lane holds
    int o = LANES / 2;
#pragma unroll
    for (int n = N; n > 1; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = up ? v[k + n / 2] : v[k], send = up ? v[k] : v[k + n / 2];
            v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    }
    float x = v[0];
#pragma unroll
    for (int q = LANES / 2 / N; q > 0; q /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, q);
    constexpr int kStep = LANES / N;   // lane k * kStep holds value k
    if (LANES < 32 || warps == 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = N == 1 ? x : __shfl_sync(0xFFFFFFFFu, x, k * kStep, LANES);
        return;
    }
    if (lane % kStep == 0) red[wg * N + lane / kStep] = x;
    named_bar_sync(bar, width);
    // red holds kMaxWarps rows of N (zeros past the group's warps): every lane
    // takes N / 2 neighbouring sums, and lanes with the same values meet
    constexpr int P = N > 1 ? N / 2 : 1;
    float y[P];
#pragma unroll
    for (int k = 0; k < P; ++k) y[k] = red[(lane * P + k) % (kMaxWarps * N)];
#pragma unroll
    for (int q = N > 1 ? 2 : 1; q < (N > 1 ? 32 : 16); q *= 2)
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] += __shfl_xor_sync(0xFFFFFFFFu, y[k], q);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = N > 1 ? __shfl_sync(0xFFFFFFFFu, y[k % P], k / P) : y[0];
}

// words of shared memory that one row's copy takes (kMixed): its chunks, and
// one more for the shift
__host__ __device__ constexpr int row_words(int chunks) { return chunks + 1; }

// zeros in this thread's ring slots for chunks that its rows do not have
template <int ROWS, int NCH>
__device__ __forceinline__ void clear_slots(uint4* ring, int t, int width, int here)
{
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        if (t + i * width >= here)
            for (int k = 0; k < ROWS; ++k) ring[(k * NCH + i) * blockDim.x] = make_uint4(0, 0, 0, 0);
}

// the threads of a group meet (a group of one warp, or less, needs no barrier of its own)
__device__ __forceinline__ void group_sync(int grp, int warps, int width)
{
    if (warps <= 1)
        __syncwarp();
    else
        named_bar_sync(1 + grp, width);
}

// Forward: one read, one write.  Two rows at a time, so that their sums share
// the group's barriers.
template <int DT, int NCH, int R, int DEPTH, int MINB, int MODE, int LANES = 32>
__global__ void __launch_bounds__(512, MINB)
    ln_forward_rows(const __grid_constant__ LnArgs a, int width, int groups)
{
    using T = typename El<DT>::T;
    constexpr int V = kV<DT>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[2][8][kMaxWarps * R];
    if (LANES < 32) width = LANES;
    const int warps = width / 32, grp = threadIdx.x / width, t = threadIdx.x % width, wg = t >> 5;
    const int words = row_words((a.cols + 2 * V - 2) / V);
    Walk<MODE, R, LANES> walk(grp, groups, a.rows);
    long long& r0 = walk.r0;
    const long long step = walk.step;
    // columns of a result row's first word that belong to the row before
    const int first = by_words(MODE) ? static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.out) + r0 * a.out_stride) & 15u) / sizeof(T)) : 0;
    const int here = by_words(MODE) ? (first + a.cols + V - 1) / V : a.cols / V;   // words of a row
    // the i-th chunk of this thread, and its first column
    auto chunk = [&](int i) { return !by_turns(MODE) ? t + i * width : i == 0 && t == 0 ? here - 1 : t + i * width - 1; };
    auto column = [&](int i) { return chunk(i) * V - first; };
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    for (int i = threadIdx.x; i < 2 * 8 * kMaxWarps * R; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_launch();
    f32x2 gain[NCH][V / 2], bias[NCH][V / 2];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        weights_at<V>(a.gain, a.w_dtype, t + i * width < here ? column(i) : a.cols, a.cols, 1.0f, gain[i]);
        weights_at<V>(a.bias, a.w_dtype, t + i * width < here ? column(i) : a.cols, a.cols, 0.0f, bias[i]);
    }
    const RowSource<DT> x(a.x, a.x_stride, a.rows, a.cols);
    // [DEPTH][R][NCH][threads]; kMixed: a group's [DEPTH][R][words]
    uint4* ring = reinterpret_cast<uint4*>(smem) + (MODE != kMixed ? threadIdx.x : grp * DEPTH * R * words);
    const uint32_t x_off = MODE == kMixed ? (x.row(r0) - first * sizeof(T)) & 15u : 0u;   // of any chunk in its first word
    // words of a stage; where the next rows go and come from
    const int stage = MODE != kMixed ? R * NCH * blockDim.x : R * words;
    uint4* into = ring;
    long long rf = r0;
    const T* xf = x.base + r0 * x.stride;
    if (MODE != kMixed)   // slots of chunks past the row are never written again
        clear_slots<DEPTH * R, NCH>(ring, t, width, here);
    auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long r = rf + k * walk.apart;
            if (r >= a.rows) break;
            // only these rows' words may reach past the array
            const bool ends = MODE == kMixed || a.cols < V || r == 0 || r == a.rows - 1;
            if (MODE != kMixed) {
                const T* q = xf + k * walk.apart * x.stride;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
                    if (t + i * width < here) {
                        uint4* p = into + (k * NCH + i) * blockDim.x;
                        if (MODE == kAligned)
                            cp_async16(p, q + chunk(i) * V);
                        else if (MODE == kFours)
                            x.copy_fours(p, q, column(i), a.cols);
                        else
                            x.copy_word(p, reinterpret_cast<uintptr_t>(q + column(i)), reinterpret_cast<uintptr_t>(q), reinterpret_cast<uintptr_t>(q + a.cols), ends);
                    }
            } else {
                const uintptr_t row = reinterpret_cast<uintptr_t>(xf + k * walk.apart * x.stride), to = row + static_cast<uintptr_t>(a.cols) * sizeof(T);
                const uintptr_t at = row - first * sizeof(T) - x_off;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
                    if (t + i * width < here) x.copy_if_any(into + k * words + chunk(i), at + 16u * chunk(i), row, to, ends);
                if (t == 0) x.copy_if_any(into + k * words + here, at + 16u * here, row, to, ends);
            }
        }
        cp_async_commit();
        rf += step;
        xf += step * x.stride;
        into = into == ring + (DEPTH - 1) * stage ? ring : into + stage;
    };
    for (int s = 0; s < DEPTH - 1; ++s) fetch();
    const uint4* from = ring;
    T* yr = static_cast<T*>(a.out) + r0 * a.out_stride;
    for (; r0 < walk.end; r0 += step, yr += step * a.out_stride, from = from == ring + (DEPTH - 1) * stage ? ring : from + stage) {
        cp_async_wait<DEPTH - 2>();
        if (MODE == kMixed) group_sync(grp, warps, width);
        uint4 w[R][NCH];
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                // (rows past the last: whatever lies there, and no result)
                if (MODE != kMixed) {
                    w[k][i] = from[(k * NCH + i) * blockDim.x];
                    if (by_words(MODE)) w[k][i] = masked<DT>(w[k][i], column(i), a.cols);
                } else {
                    w[k][i] = make_uint4(0, 0, 0, 0);
                    if (t + i * width >= here || r0 + k * walk.apart >= a.rows) continue;
                    const uint4* p = from + k * words + chunk(i);
                    w[k][i] = masked<DT>(shifted(p[0], p[1], x_off), column(i), a.cols);
                }
            }
        fetch();
        float mean[R], rstd[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f32x2 sum = 0;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                f32x2 f[V / 2];
                widen<DT>(w[k][i], f);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) sum = add2(sum, f[e]);
            }
            mean[k] = both(sum);
        }
        group_sums<R, LANES>(mean, red[0][grp & 7], warps, 1 + grp, width, wg);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] *= inv_c;
            const f32x2 m = pack2(mean[k], mean[k]);
            f32x2 sum = 0;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = column(i);
                if (t + i * width >= here) break;
                forget(w[k][i]);
                if (MODE == kAligned || (c >= 0 && c + V <= a.cols)) {
                    f32x2 f[V / 2];
                    widen<DT>(w[k][i], f);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        f[e] = sub2(f[e], m);
                        sum = fma2(f[e], f[e], sum);
                    }
                } else {
                    float f[V], part = 0.0f;
                    widen<DT>(w[k][i], f);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c + e >= 0 && c + e < a.cols) part = fmaf(f[e] - mean[k], f[e] - mean[k], part);
                    sum = add2(sum, pack2(part, 0.0f));
                }
            }
            rstd[k] = both(sum);
        }
        group_sums<R, LANES>(rstd, red[1][grp & 7], warps, 1 + grp, width, wg);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long r = r0 + k * walk.apart;
            if (r >= a.rows) break;
            rstd[k] = inverse_root(rstd[k] * inv_c + a.eps);
            const uintptr_t y = reinterpret_cast<uintptr_t>(yr + k * walk.apart * a.out_stride);
            const Centred<DT> row(mean[k], rstd[k]);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = column(i);
                if (t + i * width >= here) break;
                f32x2 f[V / 2];
                float o[V];
                forget(w[k][i]);
                widen<DT>(w[k][i], f);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) f[e] = fma2(row.xhat(f[e]), gain[i][e], bias[i][e]);
                unpack(f, o);
                if (MODE == kAligned)
                    __stcs(reinterpret_cast<uint4*>(y) + t + i * width, narrowed<DT>(o));
                else
                    put_word<DT>(y, c, a.cols, narrowed<DT>(o));
            }
            if (t == 0) {
                if (a.mean_out != nullptr) a.mean_out[r] = mean[k];
                if (a.rstd_out != nullptr) a.rstd_out[r] = rstd[k];
            }
        }
    }
}

// Backward: dx, and the column sums of the rows the CTA took, in one pass.  Each
// CTA leaves one row of partial sums (at most 304), not an atomic: the same
// bits every time.
template <int DT, int NCH, int R, int DEPTH, int MINB, int MODE, int LANES = 32>
__global__ void __launch_bounds__(512, MINB)
    ln_backward_rows_fused(const __grid_constant__ LnArgs a, int width, int groups)
{
    using T = typename El<DT>::T;
    constexpr int V = kV<DT>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[2][8][kMaxWarps * 2 * R];
    if (LANES < 32) width = LANES;
    const int warps = width / 32, grp = threadIdx.x / width, t = threadIdx.x % width, wg = t >> 5;
    const int words = row_words((a.cols + 2 * V - 2) / V);
    Walk<MODE, R, LANES> walk(grp, groups, a.rows);
    long long& r0 = walk.r0;
    const long long step = walk.step;
    // columns of a result row's first word that belong to the row before
    const int first = by_words(MODE) ? static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.out) + r0 * a.out_stride) & 15u) / sizeof(T)) : 0;
    const int here = by_words(MODE) ? (first + a.cols + V - 1) / V : a.cols / V;   // words of a row
    // the i-th chunk of this thread, and its first column
    auto chunk = [&](int i) { return !by_turns(MODE) ? t + i * width : i == 0 && t == 0 ? here - 1 : t + i * width - 1; };
    auto column = [&](int i) { return chunk(i) * V - first; };
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    for (int i = threadIdx.x; i < 2 * 8 * kMaxWarps * 2 * R; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_launch();
    f32x2 gain[NCH][V / 2], dg2[NCH][V / 2], db2[NCH][V / 2];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        weights_at<V>(a.gain, a.w_dtype, t + i * width < here ? column(i) : a.cols, a.cols, 1.0f, gain[i]);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) dg2[i][e] = db2[i][e] = 0;
    }
    const RowSource<DT> x(a.x, a.x_stride, a.rows, a.cols), dy(a.dy, a.dy_stride, a.rows, a.cols);
    // [DEPTH][R][2][NCH][threads]; kMixed: a group's [DEPTH][R][2][words]
    uint4* ring = reinterpret_cast<uint4*>(smem) + (MODE != kMixed ? threadIdx.x : grp * 2 * DEPTH * R * words);
    // of any chunk in its first word
    const uint32_t x_off = MODE == kMixed ? (x.row(r0) - first * sizeof(T)) & 15u : 0u;
    const uint32_t d_off = MODE == kMixed ? (dy.row(r0) - first * sizeof(T)) & 15u : 0u;
    // words of a stage; where the next rows go and come from
    const int stage = MODE != kMixed ? 2 * R * NCH * blockDim.x : 2 * R * words;
    int into = 0;
    if (MODE != kMixed)   // slots of chunks past the row are never written again
        clear_slots<DEPTH * R * 2, NCH>(ring, t, width, here);
    auto fetch = [&](long long rf) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long r = rf + k * walk.apart;
            if (r >= a.rows) break;
            const bool ends = MODE == kMixed || a.cols < V || r == 0 || r == a.rows - 1;
            if (MODE != kMixed) {
                const T* q = x.base + r * x.stride;
                const T* d = dy.base + r * dy.stride;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
                    if (t + i * width < here) {
                        uint4* p = ring + into + (k * 2 * NCH + i) * blockDim.x;
                        const int c = column(i);
                        if (MODE == kAligned) {
                            cp_async16(p, q + c);
                            cp_async16(p + NCH * blockDim.x, d + c);
                        } else if (MODE == kFours) {
                            x.copy_fours(p, q, c, a.cols);
                            dy.copy_fours(p + NCH * blockDim.x, d, c, a.cols);
                        } else {
                            x.copy_word(p, reinterpret_cast<uintptr_t>(q + c), reinterpret_cast<uintptr_t>(q), reinterpret_cast<uintptr_t>(q + a.cols), ends);
                            dy.copy_word(p + NCH * blockDim.x, reinterpret_cast<uintptr_t>(d + c), reinterpret_cast<uintptr_t>(d), reinterpret_cast<uintptr_t>(d + a.cols), ends);
                        }
                    }
            } else {
                uint4* p = ring + into + k * 2 * words;
                const uintptr_t xr = x.row(r), dr = dy.row(r), n = static_cast<uintptr_t>(a.cols) * sizeof(T);
                const uintptr_t xa = xr - first * sizeof(T) - x_off, da = dr - first * sizeof(T) - d_off;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
                    if (t + i * width < here) {
                        x.copy_if_any(p + chunk(i), xa + 16u * chunk(i), xr, xr + n, ends);
                        dy.copy_if_any(p + words + chunk(i), da + 16u * chunk(i), dr, dr + n, ends);
                    }
                if (t == 0) {
                    x.copy_if_any(p + here, xa + 16u * here, xr, xr + n, ends);
                    dy.copy_if_any(p + words + here, da + 16u * here, dr, dr + n, ends);
                }
            }
        }
        cp_async_commit();
        into = into == (DEPTH - 1) * stage ? 0 : into + stage;
    };
    for (int s = 0; s < DEPTH - 1; ++s) fetch(r0 + s * step);
    float mean[R], rstd[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const long long r = r0 + k * walk.apart;
        mean[k] = r < a.rows ? a.mean[r] : 0.0f;
        rstd[k] = r < a.rows ? a.rstd[r] : 0.0f;
    }
    int buf = 0;
    for (int from = 0; r0 < walk.end; r0 += step, from = from == (DEPTH - 1) * stage ? 0 : from + stage, buf ^= 1) {
        cp_async_wait<DEPTH - 2>();
        if (MODE == kMixed) group_sync(grp, warps, width);
        uint4 wx[R][NCH], wd[R][NCH];
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                if (MODE == kMixed || R > 1 || LANES < 32) {   // (else a loop's row is there)
                    wx[k][i] = wd[k][i] = make_uint4(0, 0, 0, 0);
                    if (t + i * width >= here || r0 + k * walk.apart >= a.rows) continue;
                }
                if (MODE != kMixed) {
                    const uint4* p = ring + from + (k * 2 * NCH + i) * blockDim.x;
                    wx[k][i] = p[0];
                    wd[k][i] = p[NCH * blockDim.x];
                    if (by_words(MODE)) {
                        const int c = column(i);
                        wx[k][i] = masked<DT>(wx[k][i], c, a.cols);
                        wd[k][i] = masked<DT>(wd[k][i], c, a.cols);
                    }
                } else {
                    const uint4* p = ring + from + k * 2 * words + chunk(i);
                    const int c = column(i);
                    wx[k][i] = masked<DT>(shifted(p[0], p[1], x_off), c, a.cols);
                    wd[k][i] = masked<DT>(shifted(p[words], p[words + 1], d_off), c, a.cols);
                }
            }
        fetch(r0 + (DEPTH - 1) * step);
        float next_mean[R], next_rstd[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long r = r0 + step + k * walk.apart;
            next_mean[k] = r < a.rows ? a.mean[r] : 0.0f;
            next_rstd[k] = r < a.rows ? a.rstd[r] : 0.0f;
        }
        // chunks and columns past the row are zeros and add nothing
        float sum[2 * R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const Centred<DT> row(mean[k], rstd[k]);
            f32x2 s1 = 0, s2 = 0;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                f32x2 xv[V / 2], dv[V / 2];
                widen<DT>(wx[k][i], xv);
                widen<DT>(wd[k][i], dv);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const f32x2 xhat = row.xhat(xv[e]), h = mul2(dv[e], gain[i][e]);
                    dg2[i][e] = fma2(dv[e], xhat, dg2[i][e]);
                    db2[i][e] = add2(db2[i][e], dv[e]);
                    s1 = add2(s1, h);
                    s2 = fma2(h, xhat, s2);
                }
            }
            sum[2 * k] = both(s1);
            sum[2 * k + 1] = both(s2);
        }
        group_sums<2 * R, LANES>(sum, red[buf][grp & 7], warps, 1 + grp, width, wg);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r0 + k * walk.apart >= a.rows) break;
            const uintptr_t out = reinterpret_cast<uintptr_t>(static_cast<T*>(a.out) + (r0 + k * walk.apart) * a.out_stride);
            // dx = rstd * (dy * gain - s1 - xhat * s2)
            const float s1 = sum[2 * k] * inv_c, s2 = sum[2 * k + 1] * inv_c;
            // = rstd * (dy * gain + x * n2 + n1), fp32: (x - mean) * n2 and no mean in n1
            const float q2 = -s2 * rstd[k], q1 = DT == ZERO_FP32 ? -s1 : fmaf(-mean[k], q2, -s1);
            const f32x2 rs = pack2(rstd[k], rstd[k]), n1 = pack2(q1, q1), n2 = pack2(q2, q2), m = pack2(mean[k], mean[k]);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = column(i);
                if (t + i * width >= here) break;
                f32x2 xv[V / 2], dv[V / 2];
                float o[V];
                forget(wx[k][i]);
                forget(wd[k][i]);
                widen<DT>(wx[k][i], xv);
                widen<DT>(wd[k][i], dv);
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    xv[e] = mul2(rs, fma2(DT == ZERO_FP32 ? sub2(xv[e], m) : xv[e], n2, fma2(dv[e], gain[i][e], n1)));
                unpack(xv, o);
                if (MODE == kAligned)
                    __stcs(reinterpret_cast<uint4*>(out) + t + i * width, narrowed<DT>(o));
                else
                    put_word<DT>(out, c, a.cols, narrowed<DT>(o));
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) mean[k] = next_mean[k], rstd[k] = next_rstd[k];
    }
    float dg[NCH][V], db[NCH][V];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        unpack(dg2[i], dg[i]);
        unpack(db2[i], db[i]);
    }
    // the CTA's column sums: its row groups add up pairwise through the ring's
    // memory (free by then), then one row of partial sums leaves
    float* p = a.parts + static_cast<long long>(blockIdx.x) * 2 * a.pitch;
    float* acc = reinterpret_cast<float*>(smem);
    if (groups > 1) {
        cp_async_wait<0>();
        __syncthreads();
        for (int n = groups, h = (n + 1) / 2; n > 1; n = h, h = (n + 1) / 2) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int k = (i * V + e) * 2 * width + t;
                    if (grp >= h && grp < n) {
                        acc[(grp - h) * NCH * V * 2 * width + k] = dg[i][e];
                        acc[(grp - h) * NCH * V * 2 * width + k + width] = db[i][e];
                    }
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NCH; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int k = (i * V + e) * 2 * width + t;
                    if (grp < n - h) {
                        dg[i][e] += acc[grp * NCH * V * 2 * width + k];
                        db[i][e] += acc[grp * NCH * V * 2 * width + k + width];
                    }
                }
            __syncthreads();
        }
    }
    if (grp == 0) {
        // chunk by chunk: column c lies at c + first (the sums past a row are zeros)
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (t + i * width >= here) break;
            const int c = chunk(i) * V;
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                *reinterpret_cast<float4*>(p + c + e) = make_float4(dg[i][e], dg[i][e + 1], dg[i][e + 2], dg[i][e + 3]);
                *reinterpret_cast<float4*>(p + a.pitch + c + e) = make_float4(db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]);
            }
        }
    }
}

// ------------------------------------------------------ any width, any stride
// For rows too wide for the pipelines above.  One CTA a row; the row is read
// three times forward and twice backward, all but the first from cache.
// VEC: every row lies on 16-byte words and is a whole number of them; else one
// element at a time.  A piece is what a thread takes at once (V columns or one).
// 4096 x 16384 bf16: forward 73 us (3.7 TB/s; floor 39.6), backward 171 us (floor
// 59; its second kernel reads x and dy again); one element at a time 234 and 324.
template <int DT, bool VEC>
constexpr int kPiece = VEC ? kV<DT> : 1;
constexpr int kWideThreads = 512;

template <int DT, bool VEC>
__device__ __forceinline__ void get_piece(const void* row, int c, float (&v)[kPiece<DT, VEC>])
{
    const typename El<DT>::T* p = static_cast<const typename El<DT>::T*>(row) + c;
    if constexpr (VEC)
        widen<DT>(*reinterpret_cast<const uint4*>(p), v);
    else
        v[0] = El<DT>::up(*p);
}
template <int DT, bool VEC>
__device__ __forceinline__ void put_piece(void* row, int c, const float (&v)[kPiece<DT, VEC>])
{
    typename El<DT>::T* p = static_cast<typename El<DT>::T*>(row) + c;
    if constexpr (VEC)
        __stcs(reinterpret_cast<uint4*>(p), narrowed<DT>(v));
    else
        *p = El<DT>::down(v[0]);
}
template <int DT, bool VEC>
__device__ __forceinline__ void get_weights(const void* w, int dt, int c, int cols, float none, float (&v)[kPiece<DT, VEC>])
{
    if constexpr (VEC) {
        f32x2 p[kV<DT> / 2];
        weights_at<kV<DT>>(w, dt, c, cols, none, p);
        unpack(p, v);
    } else {
        v[0] = w == nullptr ? none : weight_at(w, dt, c);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kWideThreads, 2) ln_forward_any(const __grid_constant__ LnArgs a)
{
    using T = typename El<DT>::T;
    constexpr int P = kPiece<DT, VEC>;
    __shared__ float red[32];
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    pdl_wait();
    pdl_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        T* y = static_cast<T*>(a.out) + r * a.out_stride;
        float s = 0.0f;
#pragma unroll 4
        for (int c = threadIdx.x * P; c < a.cols; c += kWideThreads * P) {
            float v[P];
            get_piece<DT, VEC>(x, c, v);
#pragma unroll
            for (int e = 0; e < P; ++e) s += v[e];
        }
        const float mean = block_sum(s, red) * inv_c;
        float q = 0.0f;
#pragma unroll 4
        for (int c = threadIdx.x * P; c < a.cols; c += kWideThreads * P) {
            float v[P];
            get_piece<DT, VEC>(x, c, v);
#pragma unroll
            for (int e = 0; e < P; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
        }
        const float rstd = inverse_root(block_sum(q, red) * inv_c + a.eps);
#pragma unroll 2
        for (int c = threadIdx.x * P; c < a.cols; c += kWideThreads * P) {
            float v[P], g[P], b[P];
            get_piece<DT, VEC>(x, c, v);
            get_weights<DT, VEC>(a.gain, a.w_dtype, c, a.cols, 1.0f, g);
            get_weights<DT, VEC>(a.bias, a.w_dtype, c, a.cols, 0.0f, b);
#pragma unroll
            for (int e = 0; e < P; ++e) v[e] = fmaf((v[e] - mean) * rstd, g[e], b[e]);
            put_piece<DT, VEC>(y, c, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean_out != nullptr) a.mean_out[r] = mean;
            if (a.rstd_out != nullptr) a.rstd_out[r] = rstd;
        }
    }
}

// the two row means of the backward pass
template <int DT, bool VEC>
__global__ void __launch_bounds__(kWideThreads, 2) ln_backward_rows(const __grid_constant__ LnArgs a)
{
    using T = typename El<DT>::T;
    constexpr int P = kPiece<DT, VEC>;
    __shared__ float red[32];
    const float inv_c = 1.0f / static_cast<float>(a.cols);
    pdl_wait();
    pdl_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 2
        for (int c = threadIdx.x * P; c < a.cols; c += kWideThreads * P) {
            float v[P], d[P], g[P];
            get_piece<DT, VEC>(x, c, v);
            get_piece<DT, VEC>(dy, c, d);
            get_weights<DT, VEC>(a.gain, a.w_dtype, c, a.cols, 1.0f, g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float h = d[e] * g[e];
                s1 += h;
                s2 = fmaf(h, (v[e] - mean) * rstd, s2);
            }
        }
        s1 = block_sum(s1, red) * inv_c;
        s2 = block_sum(s2, red) * inv_c;
        if (threadIdx.x == 0) {
            a.rowsums[2 * r] = s1;
            a.rowsums[2 * r + 1] = s2;
        }
    }
}

// dx and the partial column sums: blockIdx.x takes 256 pieces of columns,
// blockIdx.y every gridDim.y-th row, a few under way at a time
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) ln_backward_cols(const __grid_constant__ LnArgs a)
{
    using T = typename El<DT>::T;
    constexpr int P = kPiece<DT, VEC>, K = 2;
    const int c = (blockIdx.x * 256 + threadIdx.x) * P;
    pdl_wait();
    pdl_launch();
    if (c >= a.cols) return;
    float g[P], dg[P], db[P];
    get_weights<DT, VEC>(a.gain, a.w_dtype, c, a.cols, 1.0f, g);
#pragma unroll
    for (int e = 0; e < P; ++e) dg[e] = db[e] = 0.0f;
    for (long long r0 = blockIdx.y; r0 < a.rows; r0 += K * static_cast<long long>(gridDim.y)) {
        float v[K][P], d[K][P];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long r = r0 + k * static_cast<long long>(gridDim.y);
            if (r >= a.rows) break;
            get_piece<DT, VEC>(static_cast<const T*>(a.x) + r * a.x_stride, c, v[k]);
            get_piece<DT, VEC>(static_cast<const T*>(a.dy) + r * a.dy_stride, c, d[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long r = r0 + k * static_cast<long long>(gridDim.y);
            if (r >= a.rows) break;
            const float mean = a.mean[r], rstd = a.rstd[r], s1 = a.rowsums[2 * r], s2 = a.rowsums[2 * r + 1];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float xhat = (v[k][e] - mean) * rstd;
                dg[e] = fmaf(d[k][e], xhat, dg[e]);
                db[e] += d[k][e];
                v[k][e] = rstd * (d[k][e] * g[e] - s1 - xhat * s2);
            }
            put_piece<DT, VEC>(static_cast<T*>(a.out) + r * a.out_stride, c, v[k]);
        }
    }
    float* p = a.parts + static_cast<long long>(blockIdx.y) * 2 * a.pitch + c;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        p[e] = dg[e];
        p[a.pitch + e] = db[e];
    }
}

// The partial column sums, in a fixed order: 32 columns a CTA, sixteen slices
// of the parts side by side.  5 MB for 4096 columns, out of L2; 2 to 3 us after
// the rows' kernel, whose end it waits for (fp64 sums: 3 us more).
__global__ void __launch_bounds__(512) ln_backward_finish(const __grid_constant__ LnArgs a, int parts, uint32_t firsts)
{
    __shared__ float red[16][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    const bool bias = i >= a.cols;
    const float* p = a.parts + (bias ? i - a.cols + a.pitch : i);
    pdl_wait();
    float s = 0.0f;
    if (i < 2 * a.cols) {
        // a CTA's sums begin where its rows do (all eight kinds in turn: bits
        // 4 k .. of `firsts`)
#pragma unroll 10
        for (int k = slice; k < parts; k += 16) s += p[static_cast<long long>(k) * 2 * a.pitch + (firsts >> 4 * (k & 7) & 15u)];
    }
    red[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || i >= 2 * a.cols) return;
    void* out = bias ? a.dbias : a.dgain;
    if (out == nullptr) return;
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = red[k][lane];
#pragma unroll
    for (int n = 8; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += v[k + n];
    put_weight(out, a.w_dtype, bias ? i - a.cols : i, v[0]);
}

// ------------------------------------------------------------------- host
constexpr size_t kSmemOptin = 227 * 1024;   // that a CTA may have
constexpr size_t kRowSmem = 220 * 1024;     // of it, for rows and partial sums

// how a launch cuts its rows up
struct RowShape {
    int width, groups, threads;
    long long grid;
};

// Groups share a CTA of up to 512 threads, fewer where the rows would not
// cover the SMs otherwise.
RowShape row_shape(const LnArgs& a, int width, int r, int per_sm, size_t group_smem, int sms, bool eights)
{
    RowShape s;
    s.width = width;
    const long long sets = (a.rows + r - 1) / r;
    const long long spread = (sets + sms - 1) / sms;
    s.groups = 32 * kMaxWarps / width;
    if (s.groups > static_cast<int>(kRowSmem / per_sm / group_smem)) s.groups = static_cast<int>(kRowSmem / per_sm / group_smem);
    if (s.groups > spread) s.groups = static_cast<int>(spread);
    if (width < 32) s.groups = (s.groups + 32 / width - 1) / (32 / width) * (32 / width);   // whole warps
    s.threads = width * s.groups;
    s.grid = (sets + s.groups - 1) / s.groups;
    if (s.grid > static_cast<long long>(sms) * per_sm) s.grid = static_cast<long long>(sms) * per_sm;
    if (eights) s.grid = s.grid < 8 ? 8 : s.grid / 8 * 8;   // eight kinds of rows
    return s;
}

// words a thread's chunks have to cover: rows cut by words may begin inside one
template <int DT>
int chunks_of(int cols, int mode)
{
    return (cols + kV<DT> - 1 + (by_words(mode) ? kV<DT> - 1 : 0)) / kV<DT>;
}

// How equal rows of the arrays (null: none) lie; strides in elements.
template <int DT>
int mode_of(int cols, const void* p, long long ps, const void* q, long long qs, const void* r, long long rs)
{
    constexpr int V = kV<DT>;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q), c = r != nullptr ? reinterpret_cast<uintptr_t>(r) : a;
    if (r == nullptr) rs = ps;
    if (cols % V == 0 && ps % V == 0 && qs % V == 0 && rs % V == 0 && a % 16 == 0 && b % 16 == 0 && c % 16 == 0) return kAligned;
    return a % 16 == b % 16 && a % 16 == c % 16 && ps % V == qs % V && ps % V == rs % V ? kAlike : DT == ZERO_FP32 ? kFours : kMixed;
}

template <typename K>
cudaError_t launch_rows(K kernel, const LnArgs& a, const RowShape& s, size_t smem, cudaStream_t st)
{
    if (smem > 40 * 1024) {   // 48 KB without asking, the static arrays included
        // The limit belongs to the kernel, not to the call: the same for every
        // call, so that one on another host thread cannot lower it in between.
        static_assert(kRowSmem <= kSmemOptin - 4 * 1024, "and the static arrays");
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRowSmem));
        if (e != cudaSuccess) return e;
    }
    return launch_after(kernel, dim3(static_cast<unsigned>(s.grid)), dim3(s.threads), smem, st, a, s.width, s.groups);
}

template <int DT, int NCH, int R, int DEPTH, int MINB, int MODE, int LANES = 32>
cudaError_t forward_as(const LnArgs& a, int sms, cudaStream_t st)
{
    const int chunks = chunks_of<DT>(a.cols, MODE);
    const int width = LANES < 32 ? LANES : (chunks + 32 * NCH - 1) / (32 * NCH) * 32;
    const size_t per = 16u * R * (MODE != kMixed ? static_cast<size_t>(DEPTH) * NCH * width : static_cast<size_t>(DEPTH) * row_words(chunks));
    const RowShape s = row_shape(a, width, R, MINB, per, sms, by_words(MODE));
    return launch_rows(ln_forward_rows<DT, NCH, R, DEPTH, MINB, MODE, LANES>, a, s, per * s.groups, st);
}

template <int DT, int NCH, int R, int DEPTH, int MINB, int MODE, int LANES = 32>
cudaError_t backward_as(const LnArgs& a, int sms, cudaStream_t st, int& parts)
{
    const int chunks = chunks_of<DT>(a.cols, MODE);
    const int width = LANES < 32 ? LANES : (chunks + 32 * NCH - 1) / (32 * NCH) * 32;
    const size_t per = 16u * R * (MODE != kMixed ? static_cast<size_t>(2 * DEPTH) * NCH * width : static_cast<size_t>(2 * DEPTH) * row_words(chunks));
    RowShape s = row_shape(a, width, R, MINB, per, sms, by_words(MODE));
    if (s.grid > kLnMaxParts) s.grid = kLnMaxParts;
    parts = static_cast<int>(s.grid);
    size_t smem = per * s.groups;
    const size_t sums = static_cast<size_t>(s.groups / 2) * 2 * NCH * kV<DT> * s.width * sizeof(float);
    if (smem < sums) smem = sums;
    return launch_rows(ln_backward_rows_fused<DT, NCH, R, DEPTH, MINB, MODE, LANES>, a, s, smem, st);
}

// A thread holds 16 columns of a row (one chunk of it where the row has no more
// than a warp's worth), so that what a row costs each thread besides its
// columns is spread; sixteen warps then hold kMaxCols columns.
constexpr int kMaxCols = 8192;
static_assert(kMaxCols - 2 * 8 >= kLnWide, "narrower rows never take the general kernels");
template <int DT>
constexpr int kNch = 16 / kV<DT>;
// Rows of up to a warp's chunks, one to LANES lanes: the fewest of 8, 16 and 32
// that hold them, so that few lanes idle and a warp's instructions serve several
// rows (400000 x 64 bf16: 58 us forward and 80 backward with a warp a row, 21 and
// 35 with eight lanes; x 128: 58 and 83, 39 and 57 with sixteen).  Two CTAs an
// SM forward where 64 registers a thread are enough; the forms for 16-bit rows
// that are not aligned would spill.
template <int DT, int LANES>
cudaError_t forward_narrow(const LnArgs& a, int mode, int sms, cudaStream_t st)
{
    if (mode == kAligned) return forward_as<DT, 1, 2, 4, 2, kAligned, LANES>(a, sms, st);
    if (mode == kAlike) return forward_as<DT, 1, 2, 4, DT == ZERO_FP32 ? 2 : 1, kAlike, LANES>(a, sms, st);
    return forward_as<DT, 1, 2, 3, DT == ZERO_FP32 ? 2 : 1, DT == ZERO_FP32 ? kFours : kMixed, LANES>(a, sms, st);
}
template <int DT, int LANES>
cudaError_t backward_narrow(const LnArgs& a, int mode, int sms, cudaStream_t st, int& parts)
{
    if (mode == kAligned) return backward_as<DT, 1, 2, 3, 1, kAligned, LANES>(a, sms, st, parts);
    if (mode == kAlike) return backward_as<DT, 1, 2, 3, 1, kAlike, LANES>(a, sms, st, parts);
    return backward_as<DT, 1, 2, 3, 1, DT == ZERO_FP32 ? kFours : kMixed, LANES>(a, sms, st, parts);
}

template <int DT>
cudaError_t forward_of(const LnArgs& a, cudaStream_t st)
{
    constexpr int V = kV<DT>;
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    const int mode = mode_of<DT>(a.cols, a.x, a.x_stride, a.out, a.out_stride, nullptr, 0);
    constexpr int N = kNch<DT>;
    const int chunks = chunks_of<DT>(a.cols, mode);
    if (chunks <= 8) return forward_narrow<DT, 8>(a, mode, sms, st);
    if (chunks <= 16) return forward_narrow<DT, 16>(a, mode, sms, st);
    if (chunks <= 32) return forward_narrow<DT, 32>(a, mode, sms, st);
    if (chunks <= kMaxCols / V) {
        if (mode == kAligned) return forward_as<DT, N, 2, 3, 1, kAligned>(a, sms, st);
        // (fp32 rows up to 4096 columns go eight a thread: 1601 wide 13.7 -> 12.0 us)
        if (mode == kAlike) return chunks <= 1024 ? forward_as<DT, 2, 2, 3, 1, kAlike>(a, sms, st) : forward_as<DT, N, 2, 3, 1, kAlike>(a, sms, st);
        if constexpr (DT == ZERO_FP32)
            return chunks <= 1024 ? forward_as<DT, 2, 2, 3, 1, kFours>(a, sms, st) : forward_as<DT, N, 2, 3, 1, kFours>(a, sms, st);
        else
            return forward_as<DT, N, 2, 3, 1, kMixed>(a, sms, st);
    }
    const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
    if (mode == kAligned) return launch_after(ln_forward_any<DT, true>, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads), 0, st, a);
    return launch_after(ln_forward_any<DT, false>, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads), 0, st, a);
}

template <int DT>
cudaError_t backward_of(const LnArgs& args, cudaStream_t st)
{
    LnArgs a = args;
    uint32_t firsts = 0;
    constexpr int V = kV<DT>;
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    int parts = static_cast<int>(a.rows < kLnMaxParts ? a.rows : kLnMaxParts);
    if (a.rows > 0) {
        const int mode = mode_of<DT>(a.cols, a.x, a.x_stride, a.out, a.out_stride, a.dy, a.dy_stride);
        if (by_words(mode))
            for (int k = 0; k < 8; ++k)
                firsts |= static_cast<uint32_t>((reinterpret_cast<uintptr_t>(a.out) + k * a.out_stride * dtype_bytes(DT)) % 16 / dtype_bytes(DT)) << 4 * k;
        constexpr int N = kNch<DT>;
        const int chunks = chunks_of<DT>(a.cols, mode);
        cudaError_t e;
        if (chunks <= 8) {
            e = backward_narrow<DT, 8>(a, mode, sms, st, parts);
        } else if (chunks <= 16) {
            e = backward_narrow<DT, 16>(a, mode, sms, st, parts);
        } else if (chunks <= 32) {
            e = backward_narrow<DT, 32>(a, mode, sms, st, parts);
        } else if (chunks <= kMaxCols / V) {
            // (fp32 rows up to 4096 columns that are not aligned go eight a
            // thread: with sixteen these forms spill, 1601 wide 24.8 -> 19.6 us)
            if (mode == kAligned)
                e = backward_as<DT, N, 1, 3, 1, kAligned>(a, sms, st, parts);
            else if (mode == kAlike)
                e = chunks <= 1024 ? backward_as<DT, 2, 1, 3, 1, kAlike>(a, sms, st, parts) : backward_as<DT, N, 1, 3, 1, kAlike>(a, sms, st, parts);
            else if constexpr (DT == ZERO_FP32)
                e = chunks <= 1024 ? backward_as<DT, 2, 1, 3, 1, kFours>(a, sms, st, parts) : backward_as<DT, N, 1, 3, 1, kFours>(a, sms, st, parts);
            else
                e = backward_as<DT, N, 1, 3, 1, kMixed>(a, sms, st, parts);
        } else {
            const long long grid = a.rows < (1 << 30) ? a.rows : (1 << 30);
            firsts = 0;
            const bool vec = mode == kAligned;
            const int across = (a.cols + 256 * (vec ? V : 1) - 1) / (256 * (vec ? V : 1));
            // as many CTAs as the SMs hold at a time: a part more is two rows of
            // sums more (304 parts: 209 and 249 us for 4096 x 16384 and 500 x 65536,
            // so 171 and 120); sixteen at least keep the chains of sums short
            int most = ((vec ? 3 : 8) * sms + across - 1) / across;
            if (most < 16) most = 16;
            if (parts > most) parts = most;
            const dim3 cols(across, parts);
            const auto rows_of = vec ? ln_backward_rows<DT, true> : ln_backward_rows<DT, false>;
            const auto cols_of = vec ? ln_backward_cols<DT, true> : ln_backward_cols<DT, false>;
            e = launch_after(rows_of, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads), 0, st, a);
            if (e == cudaSuccess) e = launch_after(cols_of, cols, dim3(256), 0, st, a);
        }
        if (e != cudaSuccess) return e;
    }
    if (a.dgain == nullptr && a.dbias == nullptr) return cudaSuccess;
    return launch_after(ln_backward_finish, dim3((2 * a.cols + 31) / 32), dim3(512), 0, st, a, parts, firsts);
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
