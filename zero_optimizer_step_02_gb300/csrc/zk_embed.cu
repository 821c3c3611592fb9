// zk_embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale * table[id[t]]
//   dtable[v] = scale * (sum over the tokens t with id[t] = v, in their order, of dout[t])
//
// The gradient takes two kernels.  The first sorts the tokens by id, stably: a
// CTA has a range of ids to itself, walks all tokens and counts its own, each of
// its warps over a stretch of the tokens, so that a position in the sorted order
// is the number of tokens with a smaller id, which the CTA counts by the way, and
// two prefix sums in shared memory; nothing is exchanged between CTAs.
// The second kernel cuts the sorted order into windows of equal length and gives
// each (in slabs of columns) to a warp, which adds up its tokens' rows and writes
// one out wherever the id changes: as much work for every warp, however often an
// id comes up.  A row that crosses windows is left as a partial sum by each, and
// the last warps to finish add them up in order: no result depends on who that was.
// A warp that is done writes its share of the zeros of the rows that no token names,
// which is most of the table where there are more rows than tokens.
//
// What a call cannot do without, at a copy's rate, and what it takes (us; bf16):
//   lookup, 16384 of 128256 x 4096     28.1   34.2: rows of 8 KB from all over memory
//   gradient, 16384 to 128256 x 4096    175    201: the table's zeros, at a copy's
//       rate; 10 of it are the sort, which moves nothing of that
//   gradient, 8192 to 50257 x 768      13.2   25.0: the sort (8), then the rows of a
//       window, eight at a time, and the parts of the row with the most tokens
//   added to, 5000 to 1031 x 333 fp32   1.3   19.2: the same latencies
#include <cstring>

#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"
#include "zk_rows.cuh"
#include "zk_tc.cuh"

namespace zk {
namespace {

constexpr int kLane8 = 8;           // columns a lane holds of a slab
constexpr int kSlab = 32 * kLane8;
constexpr int kGatherThreads = 256;

template <typename ID>
__device__ __forceinline__ bool names_a_row(ID id, const EmbedArgs& a)
{
    return id >= 0 && static_cast<unsigned long long>(id) < static_cast<unsigned long long>(a.vocab) && static_cast<long long>(id) != a.padding_id;
}

// eight columns of a row from `c` on: WORDS 16-byte words (c a multiple of 8),
// else columns 32 apart from c on; 0 where there is none
template <int DT, bool WORDS>
__device__ __forceinline__ void load8(const typename El<DT>::T* p, int c, int cols, float (&x)[8])
{
    if constexpr (WORDS) {
        if (c + 8 <= cols) {
            if constexpr (DT == ZERO_FP32) {
                const float4 a = *reinterpret_cast<const float4*>(p + c), b = *reinterpret_cast<const float4*>(p + c + 4);
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            } else {
                widen<DT>(*reinterpret_cast<const uint4*>(p + c), x);
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = WORDS ? c + e : c + 32 * e;
        x[e] = i < cols ? El<DT>::up(p[i]) : 0.0f;
    }
}

template <int DT, bool WORDS>
__device__ __forceinline__ void store8(typename El<DT>::T* p, int c, int cols, const float (&x)[8])
{
    if constexpr (WORDS) {
        if (c + 8 <= cols) {
            if constexpr (DT == ZERO_FP32) {
                __stcs(reinterpret_cast<float4*>(p + c), make_float4(x[0], x[1], x[2], x[3]));
                __stcs(reinterpret_cast<float4*>(p + c + 4), make_float4(x[4], x[5], x[6], x[7]));
            } else {
                __stcs(reinterpret_cast<uint4*>(p + c), narrowed<DT>(x));
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = WORDS ? c + e : c + 32 * e;
        if (i < cols) p[i] = El<DT>::down(x[e]);
    }
}

// ----------------------------------------------------------------- lookup
// `lanes` threads (a power of two, up to the CTA) take a token's row, eight columns
// each at a time.
template <int TD, int OD, typename ID, bool WORDS>
__global__ void __launch_bounds__(kGatherThreads) embed_forward(const __grid_constant__ EmbedArgs a)
{
    const int lanes = 1 << a.lanes_log2, per = kGatherThreads >> a.lanes_log2;
    const int mine = threadIdx.x & (lanes - 1), group = threadIdx.x >> a.lanes_log2;
    const long long step = static_cast<long long>(gridDim.x) * per;
    for (long long t = static_cast<long long>(blockIdx.x) * per + group; t < a.tokens; t += step) {
        const ID id = static_cast<const ID*>(a.ids)[t];
        typename El<OD>::T* out = static_cast<typename El<OD>::T*>(a.out) + t * a.out_stride;
        const bool row = names_a_row(id, a);
        if (!row && mine == 0 && static_cast<long long>(id) != a.padding_id && a.sc != nullptr) atomicOr(&a.sc->status, ZERO_DEV_BAD_INDEX);
        const typename El<TD>::T* from = static_cast<const typename El<TD>::T*>(a.table) + (row ? static_cast<long long>(id) : 0) * a.table_stride;
        // (not WORDS: lanes 32 apart take a slab's columns, one after another)
#pragma unroll 2
        for (int k = mine; k < a.slabs * 32; k += lanes) {
            const int c = WORDS ? 8 * k : (k >> 5) * kSlab + (k & 31);
            if (c >= a.cols) continue;
            float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (row) {
                load8<TD, WORDS>(from, c, a.cols, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= a.scale;
            }
            store8<OD, WORDS>(out, c, a.cols, x);
        }
    }
}

// ------------------------------------------------------- tokens by their ids
constexpr int kSortWarps = 16;
constexpr int kSortStep = 8;    // tokens a lane loads at a time
constexpr int kSortKept = 256;  // tokens of its range that a warp keeps from the first walk

__device__ __forceinline__ int block_total(int v, int* red, int* before)
{
    // inclusive over the warp, then over the warps; *before: of the threads ahead
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) red[w] = s;
    __syncthreads();
    int ahead = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kSortWarps; ++i) {
        if (i < w) ahead += red[i];
        all += red[i];
    }
    *before = ahead + s - v;
    return all;
}

// Where a token's id lies: its row as 32 bits (ids go up to 2^28), or -1.
template <typename ID>
__device__ __forceinline__ uint32_t row_of(ID id, const EmbedArgs& a)
{
    return names_a_row(id, a) ? static_cast<uint32_t>(id) : 0xFFFFFFFFu;
}

template <typename ID>
__global__ void __launch_bounds__(kSortWarps * 32) embed_sort(const __grid_constant__ EmbedArgs a)
{
    extern __shared__ int counts[];   // [warps][range], then [range + 1] starts
    __shared__ int red[kSortWarps];
    __shared__ int2 kept[kSortWarps][kSortKept];   // tokens of the range with their ids in it, in order
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, range = a.range;
    const long long lo = static_cast<long long>(blockIdx.x) * range;
    const uint32_t lo32 = static_cast<uint32_t>(lo);
    int* mine = counts + w * range;
    int* starts = counts + kSortWarps * range;
    for (int i = threadIdx.x; i < kSortWarps * range; i += blockDim.x) counts[i] = 0;
    pdl_wait();
    pdl_launch();
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.n_tickets; i += static_cast<long long>(gridDim.x) * blockDim.x)
        a.tickets[i] = 0;
    __syncthreads();
    const ID* ids = static_cast<const ID*>(a.ids);
    const int tokens = static_cast<int>(a.tokens);
    const int per = (tokens + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;
    const int from = w * per, to = from + per < tokens ? from + per : tokens;
    // how often each id of the range comes up in the warp's stretch; tokens with smaller ids
    int below = 0, held = 0;
    bool bad = false;
    ID next[kSortStep];
    const auto read = [&](int t0) {
#pragma unroll
        for (int k = 0; k < kSortStep; ++k) {
            const int t = t0 + 32 * k + lane;
            next[k] = t < to ? ids[t] : static_cast<ID>(a.padding_id);
        }
    };
    read(from);
    for (int t0 = from; t0 < to; t0 += 32 * kSortStep) {
        ID id[kSortStep];
#pragma unroll
        for (int k = 0; k < kSortStep; ++k) id[k] = next[k];
        read(t0 + 32 * kSortStep);
#pragma unroll
        for (int k = 0; k < kSortStep; ++k) {
            const int t = t0 + 32 * k + lane;
            const uint32_t r = t < to ? row_of(id[k], a) : 0xFFFFFFFFu, i = r - lo32;
            bad |= t < to && r == 0xFFFFFFFFu && static_cast<long long>(id[k]) != a.padding_id;
            const bool own = r != 0xFFFFFFFFu && i < static_cast<uint32_t>(range);
            below += r < lo32 ? 1 : 0;
            const uint32_t owners = __ballot_sync(0xFFFFFFFFu, own);
            if (owners == 0u) continue;
            if (own) {
                atomicAdd(&mine[i], 1);
                const int at = held + __popc(owners & ((1u << lane) - 1u));
                if (at < kSortKept) kept[w][at] = make_int2(t, static_cast<int>(i));
            }
            held += __popc(owners);
        }
    }
    int ahead;
    const int base = block_total(below, red, &ahead);
    if (__syncthreads_or(bad) && blockIdx.x == 0 && threadIdx.x == 0 && a.sc != nullptr) atomicOr(&a.sc->status, ZERO_DEV_BAD_INDEX);
    // each id's tokens start where the smaller ids' end; each warp's where the earlier warps' end
    int done = base;
    for (int i0 = 0; i0 < range; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        int n = 0;
        if (i < range) {
#pragma unroll
            for (int k = 0; k < kSortWarps; ++k) {
                const int c = counts[k * range + i];
                counts[k * range + i] = n;
                n += c;
            }
        }
        const int all = block_total(n, red, &ahead);
        if (i < range) {
            starts[i] = done + ahead;
            if (lo + i < a.vocab) a.start[lo + i] = done + ahead;
            if (lo + i == a.vocab - 1) a.start[a.vocab] = done + ahead + n;
        }
        done += all;
    }
    if (threadIdx.x == 0) starts[range] = done;
    __syncthreads();
    // the tokens to their places, 32 at a time: those that the warp kept, or its stretch once more
    const auto place = [&](bool own, int t, int i) {
        const uint32_t owners = __ballot_sync(0xFFFFFFFFu, own);
        if (owners == 0u) return;
        if (own) {
            const uint32_t same = __match_any_sync(owners, i);
            const int rank = __popc(same & ((1u << lane) - 1u)), n = mine[i];
            __syncwarp(owners);
            if (rank == 0) mine[i] = n + __popc(same);
            a.list[starts[i] + n + rank] = make_int2(t, static_cast<int>(lo32) + i);
        }
        __syncwarp();
    };
    if (held <= kSortKept) {
        __syncwarp();
        for (int j = 0; j < held; j += 32) {
            const int2 k = j + lane < held ? kept[w][j + lane] : make_int2(0, 0);
            place(j + lane < held, k.x, k.y);
        }
    } else {
        for (int t0 = from; t0 < to; t0 += 32 * kSortStep) {
            ID id[kSortStep];
#pragma unroll
            for (int k = 0; k < kSortStep; ++k) {
                const int t = t0 + 32 * k + lane;
                id[k] = t < to ? ids[t] : static_cast<ID>(a.padding_id);
            }
#pragma unroll
            for (int k = 0; k < kSortStep; ++k) {
                const int t = t0 + 32 * k + lane;
                const uint32_t r = t < to ? row_of(id[k], a) : 0xFFFFFFFFu, i = r - lo32;
                place(r != 0xFFFFFFFFu && i < static_cast<uint32_t>(range), t, static_cast<int>(i));
            }
        }
    }
}

// ---------------------------------------------------------------- the rows
// Rows that a lane has under way: as many as 32 registers hold with what they are
// added to (eight of each spill; 16384 tokens added to 128256 x 4096 90 us, with
// four 76).  Two CTAs an SM: the parts' sums take 128 registers, and with three or
// four CTAs of fewer 16384 to 128256 x 4096 takes 222 to 234 us, not 203.
template <int TD, int OD, bool ACC>
constexpr int kAhead = ACC || TD == ZERO_FP32 || OD == ZERO_FP32 ? 4 : 8;

// Eight columns as they lie in memory, so that a row under way takes no more
// registers than its bytes do.
template <int DT, bool WORDS>
struct Eight {
    static constexpr int N = WORDS ? (DT == ZERO_FP32 ? 2 : 1) : 2;
    uint4 w[N];          // not WORDS: the elements' bits, 32 or two times 16

    __device__ __forceinline__ void load(const typename El<DT>::T* p, int c, int cols)
    {
        if (WORDS && c + 8 <= cols) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p + c)[i];
            return;
        }
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = WORDS ? c + e : c + 32 * e;
            u[e] = 0u;
            if (i < cols) u[e] = DT == ZERO_FP32 ? reinterpret_cast<const uint32_t*>(p)[i] : reinterpret_cast<const uint16_t*>(p)[i];
        }
        if constexpr (DT == ZERO_FP32) {
            w[0] = make_uint4(u[0], u[1], u[2], u[3]);
            w[N - 1] = make_uint4(u[4], u[5], u[6], u[7]);
        } else {
            w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
        }
    }
    __device__ __forceinline__ void widened(float (&x)[8]) const
    {
        if constexpr (DT == ZERO_FP32) {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[N - 1].x, w[N - 1].y, w[N - 1].z, w[N - 1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(u[e]);
        } else {
            widen<DT>(w[0], x);
        }
    }
};

// A row of the gradient: the sum scaled, added to what was there (ACC).
template <int TD, bool WORDS, bool ACC>
__device__ __forceinline__ void put_gradient(const EmbedArgs& a, int v, int c, const float (&sum)[8], const Eight<TD, WORDS>& was)
{
    float x[8];
    if constexpr (ACC) {
        was.widened(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(sum[e], a.scale, x[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sum[e] * a.scale;
    }
    store8<TD, WORDS>(static_cast<typename El<TD>::T*>(a.dtable) + v * a.table_stride, c, a.cols, x);
}

// Window w's part of row v, which other windows have parts of too: piece 2 w where
// the row goes on from the window before or starts with this one, else 2 w + 1.
// The last warp to come of eight windows in a row adds their parts up, and the last
// of those (if there are more than eight windows) the eights' sums: a row with a
// tenth of all tokens has dozens of windows, and one warp to add them all up waits
// for memory as often.
template <int TD, bool WORDS, bool ACC>
__device__ __noinline__ void put_part(const EmbedArgs& a, int v, int w, int slab, int c, float4 lo, float4 hi)
{
    constexpr int kParts = 8;
    float sum[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int lane = threadIdx.x & 31;
    const int s = a.start[v], e = a.start[v + 1];
    const int w_first = s / a.window, windows = (e - 1) / a.window - w_first + 1;
    const int first = 2 * w_first + (s % a.window != 0);
    const auto place = [&](int x) { return static_cast<long long>(x == 0 ? first : 2 * (w_first + x)) * a.slabs + slab; };
    const auto put = [&](int x) {
        float* mine = a.partials + place(x) * kSlab + lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) __stcg(mine + 32 * k, sum[k]);
        __threadfence();
        __syncwarp();
    };
    // whether this warp is the last of n with this ticket
    const auto last_of = [&](int n, long long ticket) {
        int before = 0;
        if (lane == 0) before = atomicAdd(&a.tickets[ticket], 1);
        if (__shfl_sync(0xFFFFFFFFu, before, 0) != n - 1) return false;
        __threadfence();
        return true;
    };
    // the sum of windows x0, x0 + step, ... under end, eight of them under way
    const auto add_up = [&](int x0, int step, int end) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
        for (; x0 < end; x0 += kParts * step) {
            float q[kParts][8];
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const float* from = a.partials + place(x0 + i * step < end ? x0 + i * step : x0) * kSlab + lane;
#pragma unroll
                for (int k = 0; k < 8; ++k) q[i][k] = __ldcg(from + 32 * k);
            }
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (x0 + i * step < end) sum[k] += q[i][k];
        }
    };
    const int x = w - w_first, x0 = x / kParts * kParts, x1 = x0 + kParts < windows ? x0 + kParts : windows;
    put(x);
    if (!last_of(x1 - x0, place(x0))) return;
    Eight<TD, WORDS> was;
    if (ACC && windows <= kParts) was.load(static_cast<const typename El<TD>::T*>(a.dtable) + v * a.table_stride, c, a.cols);
    add_up(x0, 1, x1);
    if (windows > kParts) {
        put(x0);
        // the row's second window holds nothing else, so its other piece's ticket is free
        if (!last_of((windows + kParts - 1) / kParts, place(1) + a.slabs)) return;
        if (ACC) was.load(static_cast<const typename El<TD>::T*>(a.dtable) + v * a.table_stride, c, a.cols);
        add_up(0, kParts, windows);
    }
    put_gradient<TD, WORDS, ACC>(a, v, c, sum, was);
}

// Zeros into the rows that no token names, dealt out evenly among all warps.
template <int TD>
__device__ __forceinline__ void write_zeros(const EmbedArgs& a, long long warp, long long warps, int lane)
{
    using T = typename El<TD>::T;
    const bool words = reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0 && a.table_stride * sizeof(T) % 16 == 0 && a.cols * sizeof(T) % 16 == 0;
    const int per = words ? a.cols * static_cast<int>(sizeof(T)) / 16 : 0;
    const long long to = a.vocab * (warp + 1) / warps;
    for (long long v0 = a.vocab * warp / warps; v0 < to; v0 += 32) {
        uint32_t none = __ballot_sync(0xFFFFFFFFu, v0 + lane < to && a.start[v0 + lane] == a.start[v0 + lane + 1]);
        T* rows = static_cast<T*>(a.dtable) + v0 * a.table_stride;
        if (words && per < 32) {   // narrow rows: 16 bytes after 16 bytes over all of them
            for (int i = lane; i < 32 * per; i += 32) {
                const int r = i / per;
                if (none >> r & 1u) __stcs(reinterpret_cast<uint4*>(rows + r * a.table_stride) + (i - r * per), make_uint4(0u, 0u, 0u, 0u));
            }
            continue;
        }
        for (; none != 0u; none &= none - 1u) {
            T* row = rows + (__ffs(none) - 1) * a.table_stride;
            if (words) {
#pragma unroll 4
                for (int k = lane; k < per; k += 32) __stcs(reinterpret_cast<uint4*>(row) + k, make_uint4(0u, 0u, 0u, 0u));
                continue;
            }
            // whole words inside the row, single elements at its ends
            const uintptr_t from = reinterpret_cast<uintptr_t>(row), end = from + static_cast<uintptr_t>(a.cols) * sizeof(T);
            const uintptr_t first = (from + 15) / 16 * 16, last = end / 16 * 16;
            if (first >= last) {
                for (int k = lane; k < a.cols; k += 32) row[k] = T(0);
                continue;
            }
            if (lane < static_cast<int>((first - from) / sizeof(T))) row[lane] = T(0);
            if (lane < static_cast<int>((end - last) / sizeof(T))) reinterpret_cast<T*>(last)[lane] = T(0);
#pragma unroll 4
            for (uintptr_t p = first + 16 * lane; p < last; p += 512) __stcs(reinterpret_cast<uint4*>(p), make_uint4(0u, 0u, 0u, 0u));
        }
    }
}

template <int TD, int OD, bool WORDS, bool ACC>
__global__ void __launch_bounds__(kGatherThreads, 2) embed_rows(const __grid_constant__ EmbedArgs a)
{
    using T = typename El<OD>::T;
    constexpr int kA = kAhead<TD, OD, ACC>;
    const int lane = threadIdx.x & 31, slab = blockIdx.y, c = slab * kSlab + (WORDS ? 8 * lane : lane);
    const int step = gridDim.x * (kGatherThreads / 32);
    pdl_wait();
    const int total = a.start[a.vocab], windows = (total + a.window - 1) / a.window;
    const T* rows = static_cast<const T*>(a.dout);
    for (int w = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); w < windows; w += step) {
        const int w0 = w * a.window, w1 = w0 + a.window < total ? w0 + a.window : total;
        float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        bool open = false;      // the row that is being added up began in an earlier window
        for (int j0 = w0; j0 < w1; j0 += 32) {
            // the tokens and rows of 32 positions, and whether a row ends with each
            const int n = w1 - j0 < 32 ? w1 - j0 : 32;
            const int2 mine = lane < n ? a.list[j0 + lane] : make_int2(0, -1);
            const int behind = j0 + n < total ? a.list[j0 + n].y : -1;
            const int after = __shfl_down_sync(0xFFFFFFFFu, mine.y, 1);
            const uint32_t ends = __ballot_sync(0xFFFFFFFFu, lane < n && mine.y != (lane == n - 1 ? behind : after));
            if (j0 == w0) open = w0 > 0 && a.list[w0 - 1].y == __shfl_sync(0xFFFFFFFFu, mine.y, 0);
            for (int j = 0; j < n; j += kA) {
                Eight<OD, WORDS> x[kA];
                Eight<TD, WORDS> was[ACC ? kA : 1];
#pragma unroll
                for (int k = 0; k < kA; ++k) {
                    const int t = __shfl_sync(0xFFFFFFFFu, mine.x, (j + k) & 31), v = __shfl_sync(0xFFFFFFFFu, mine.y, (j + k) & 31);
                    if (j + k < n) {
                        x[k].load(rows + static_cast<long long>(t) * a.out_stride, c, a.cols);
                        if (ACC && (ends >> (j + k) & 1u)) was[k].load(static_cast<const typename El<TD>::T*>(a.dtable) + v * a.table_stride, c, a.cols);
                    }
                }
#pragma unroll
                for (int k = 0; k < kA; ++k) {
                    if (j + k < n) {
                        float f[8];
                        x[k].widened(f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[e] += f[e];
                        const bool end = ends >> (j + k) & 1u, border = j0 + j + k + 1 == w1;   // of the row, of the window
                        if (end || border) {
                            const int v = __shfl_sync(0xFFFFFFFFu, mine.y, j + k);
                            if (open || !end)
                                put_part<TD, WORDS, ACC>(a, v, w, slab, c, make_float4(sum[0], sum[1], sum[2], sum[3]), make_float4(sum[4], sum[5], sum[6], sum[7]));
                            else
                                put_gradient<TD, WORDS, ACC>(a, v, c, sum, was[ACC ? k : 0]);
                            open = false;
#pragma unroll
                            for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
                        }
                    }
                }
            }
        }
    }
    if (!ACC)
        write_zeros<TD>(a, (static_cast<long long>(blockIdx.x) * gridDim.y + slab) * (kGatherThreads / 32) + (threadIdx.x >> 5),
                        static_cast<long long>(gridDim.x) * gridDim.y * (kGatherThreads / 32), lane);
}

// ------------------------------------------------------------------- host
template <int TD, int OD>
bool in_words(const EmbedArgs& a, const void* table, const void* rows)
{
    const int tb = dtype_bytes(TD), ob = dtype_bytes(OD);
    return reinterpret_cast<uintptr_t>(table) % 16 == 0 && reinterpret_cast<uintptr_t>(rows) % 16 == 0 && a.table_stride * tb % 16 == 0 &&
           a.out_stride * ob % 16 == 0;
}

template <int TD, int OD, typename ID>
cudaError_t forward_as(EmbedArgs& a, cudaStream_t st)
{
    const bool words = in_words<TD, OD>(a, a.table, a.out);
    // threads of a row: as many as it has eights of columns, whole warps where it is not in words
    const int eights = words ? (a.cols + 7) / 8 : a.slabs * 32;
    a.lanes_log2 = words ? 0 : 5;
    while ((1 << a.lanes_log2) < eights && (1 << a.lanes_log2) < kGatherThreads) ++a.lanes_log2;
    const long long per = kGatherThreads >> a.lanes_log2, most = 1ll << 24, ctas = (a.tokens + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    count_launch();
    if (words) embed_forward<TD, OD, ID, true><<<grid, kGatherThreads, 0, st>>>(a);
    else embed_forward<TD, OD, ID, false><<<grid, kGatherThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int TD, int OD, typename ID>
cudaError_t backward_as(EmbedArgs& a, cudaStream_t st)
{
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    const auto bytes = [](int range) { return ((kSortWarps + 1) * range + 1) * static_cast<int>(sizeof(int)); };
    cudaError_t e = cudaFuncSetAttribute(embed_sort<ID>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kEmbedRange));
    if (e != cudaSuccess) return e;
    const unsigned sorters = static_cast<unsigned>((a.vocab + a.range - 1) / a.range);
    if ((e = launch_after(embed_sort<ID>, dim3(sorters), dim3(kSortWarps * 32), bytes(a.range), st, a)) != cudaSuccess) return e;
    // a warp for every window and slab, and warps enough to write zeros
    const long long windows = (a.tokens + a.window - 1) / a.window, zeros = a.accumulate ? 1 : (2 * sms + a.slabs - 1) / a.slabs;
    long long ctas = (windows + kGatherThreads / 32 - 1) / (kGatherThreads / 32);
    if (ctas < zeros) ctas = zeros;
    const dim3 grid(static_cast<unsigned>(ctas), a.slabs);
    const bool words = in_words<TD, OD>(a, a.dtable, a.dout);
    const auto rows = a.accumulate ? (words ? embed_rows<TD, OD, true, true> : embed_rows<TD, OD, false, true>)
                                   : (words ? embed_rows<TD, OD, true, false> : embed_rows<TD, OD, false, false>);
    return launch_after(rows, grid, dim3(kGatherThreads), 0, st, a);
}

template <int TD, int OD>
cudaError_t typed2(EmbedArgs& a, bool forward, cudaStream_t st)
{
    if (forward) return a.id_bits == 32 ? forward_as<TD, OD, int>(a, st) : forward_as<TD, OD, long long>(a, st);
    return a.id_bits == 32 ? backward_as<TD, OD, int>(a, st) : backward_as<TD, OD, long long>(a, st);
}

template <int TD>
cudaError_t typed(EmbedArgs& a, bool forward, cudaStream_t st)
{
    if (a.dtype == ZERO_FP32) return typed2<TD, ZERO_FP32>(a, forward, st);
    return a.dtype == ZERO_BF16 ? typed2<TD, ZERO_BF16>(a, forward, st) : typed2<TD, ZERO_FP16>(a, forward, st);
}

cudaError_t launch(EmbedArgs& a, bool forward, cudaStream_t st)
{
    if (a.table_dtype == ZERO_FP32) return typed<ZERO_FP32>(a, forward, st);
    return a.table_dtype == ZERO_BF16 ? typed<ZERO_BF16>(a, forward, st) : typed<ZERO_FP16>(a, forward, st);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// A window of the sorted order.  A call waits for a window's tokens, eight under
// way at a time, and then for the parts of the row with the most tokens (in text 6
// to 10 % of all), eight at a time: 32 tokens, or fewer (a power of two, eight at
// least) where that leaves less than eight warps to each of 152 SMs.  Longer where
// there would be more than 4096 windows, whose partial sums the workspace holds.
int embed_window(long long tokens, int cols)
{
    long long w = 32;
    while (w > 8 && (tokens + w - 1) / w * embed_slabs(cols) < 152 * 8) w /= 2;
    while ((tokens + w - 1) / w > 4096) w *= 2;
    return static_cast<int>(w);
}

int embed_slabs(int cols) { return (cols + kSlab - 1) / kSlab; }

// where the workspace's parts begin: starts, list, tickets, partial sums, end
void embed_layout(long long tokens, long long vocab, int cols, size_t at[5])
{
    const int w = embed_window(tokens, cols);
    const size_t pieces = static_cast<size_t>(2 * ((tokens + w - 1) / w)) * embed_slabs(cols);
    at[0] = 0;
    at[1] = round256(static_cast<size_t>(vocab + 1) * sizeof(int));
    at[2] = at[1] + round256(static_cast<size_t>(tokens) * sizeof(int2));
    at[3] = at[2] + round256(pieces * sizeof(int));
    at[4] = at[3] + pieces * kSlab * sizeof(float);
}

cudaError_t launch_embed_forward(EmbedArgs a, cudaStream_t st)
{
    if (a.tokens == 0) return cudaSuccess;
    a.slabs = embed_slabs(a.cols);
    return launch(a, true, st);
}

cudaError_t launch_embed_backward(EmbedArgs a, void* ws, cudaStream_t st)
{
    a.slabs = embed_slabs(a.cols);
    a.window = embed_window(a.tokens, a.cols);
    a.range = static_cast<int>((a.vocab + kEmbedSorters - 1) / kEmbedSorters);
    if (a.range > kEmbedRange) a.range = kEmbedRange;
    size_t at[5];
    embed_layout(a.tokens, a.vocab, a.cols, at);
    char* w = static_cast<char*>(ws);
    a.start = reinterpret_cast<int*>(w + at[0]);
    a.list = reinterpret_cast<int2*>(w + at[1]);
    a.tickets = reinterpret_cast<int*>(w + at[2]);
    a.partials = reinterpret_cast<float*>(w + at[3]);
    a.n_tickets = 2 * ((a.tokens + a.window - 1) / a.window) * a.slabs;
    return launch(a, false, st);
}

}  // namespace zk
