// zk_join.cu -- the residual join with the norms around it, forward and backward.
//
//   post(o) = (o - mean_o) * rstd_o * gain + bias   (rms: mean 0; or o itself)
//   hout = a h + gate * post(o),  y = pre(hout)
//   d = dhout + the gradient of pre at hout,  dh = a d,  dgate = d * post(o)
//   do = the gradient of post under gate * d
// With xhat a norm's normalised row, u the gradient of its result times its gain
// and E the mean over the columns, its gradient is rstd * (u - E(u) - xhat E(u
// xhat)); for rms without E(u).
//
// The weight gradients are sums over the rows of four products a column,
//   d ohat, d  (with the gate's factor where every token has its own)  and
//   dy xhat, dy:
// a gate that all rows share and post's gain only scale the first two, so
//   dgate = gain sum(d ohat) + bias sum(d),  dgain = gate sum(d ohat), ...
//
// What a call cannot do without, at a copy's rate, and what it takes (us; bf16, rms
// before and after, a gate vector, in a graph of calls):
//   forward   8192 x 4096   39.6   52      backward   8192 x 4096   59.4   100
//             16384 x 768   14.9   23                 16384 x 768   22.3    50
//             4096 x 16384  79.2  156                 4096 x 16384   119   349
//             5003 x 1601    9.5   32                 5003 x 1601   14.2    53  (fp16)
// Not memory but a row's own chain bounds them: words in, a sum over the team, the
// next norm's sum, words out, with sixteen warps an SM (eight backward from 2048
// columns on), as the weights and column sums of a thread's columns fill the
// registers (and, 512 threads forward above 4096 columns, up to 280 bytes of spills a
// thread); so the work is in few barriers, in sums dealt out among the lanes and
// in addresses that only advance.  In a cluster a sum costs a message's way, and
// rows of odd widths twice the instructions a column.
#include <cstring>
#include <initializer_list>

#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"
#include "zk_rows.cuh"
#include "zk_tc.cuh"

namespace zk {
namespace {

// ------------------------------------------------------------------ the rows
// A row is cut into 16-byte words.  A team of `width` threads takes R rows at a
// time, each thread the same NCH words of every row, so that weights and column
// sums stay in registers; rows of more than a CTA's words are shared by a cluster
// of CTAs.  The rows to come are on their way into a ring of DEPTH stages in
// shared memory, slots that a thread fills and empties alone.
//
// How the rows lie (MODE):
//   kWhole   rows are whole words in all arrays
//   kAlike   rows start equally far into a word in all arrays.  Where that is not
//            the same for all rows, a CTA takes rows eight apart, which all start
//            alike.  A row's first and last words are masked.
//   kSingle  each thread takes single elements, as many as its words would hold,
//            one after another across the team.
enum { kWhole = 0, kAlike = 1, kSingle = 2 };
constexpr int kTeamMax = 512;
constexpr int kApart = 8;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float into the shared memory of CTA `rank`, counted there by the barrier at the same place as `bar`
__device__ __forceinline__ void send(float* p, uint64_t* bar, uint32_t rank, float v)
{
    uint32_t at, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at), "r"(__float_as_uint(v)), "r"(b) : "memory");
}

// What a thread knows of its place.
struct Place {
    int team, t;         // team in the CTA, thread in the team
    int width;           // threads of a team
    int rank, ctas;      // in the cluster
    int first;           // columns that rows start past a word (kAlike)
};

constexpr int kClusterMax = 8;
constexpr int kSums = 4;   // sums over a team at a time, at most
constexpr int kTeamWarps = kClusterMax * kTeamMax / 32;
static_assert(kClusterMax <= 32 / kSums, "a lane for every CTA to send a sum to");
struct TeamShared {
    float red[2][kSums * kTeamWarps];
    uint64_t bar[2];
    int abort;           // sums did not come: nobody waits for the next ones
};

// Sums over a team, N at a time (1, 2 or 4), as many calls from every thread of
// the CTA.  A shuffle moves 32 lanes a clock for the whole SM, four times less than
// an addition takes: the lanes first deal the sums out among themselves (half of
// them go on with one half of the sums), so that N sums over a warp take 5 to 6
// shuffles, not 5 N.  Warps leave theirs in shared memory, in two buffers that take
// turns, so that one barrier a call is enough: who writes a buffer again has
// passed the barrier of the call between, which all its readers reached later.  In
// a cluster every warp sends its sums to all the CTAs, whose barriers count the
// bytes that have come; that orders nothing else, where a cluster barrier's release
// would wait for the rows' stores (8192 x 8192, layer norms: 1.2 us a sum).  A
// barrier is used again two calls later, when all the cluster's warps have read
// the call before.
template <bool CL>
struct TeamSum {
    TeamShared& sh;
    int width, lane, warps, ctas;
    int first;           // the team's warps in a buffer
    int own;             // this warp there
    int turn, phase;

    __device__ __forceinline__ TeamSum(TeamShared& s, const Place& p) : sh(s), width(p.width), lane(p.t & 31), warps(p.width >> 5), ctas(p.ctas), turn(0), phase(0)
    {
        first = CL ? 0 : p.team * warps;
        own = (CL ? p.rank : p.team) * warps + (p.t >> 5);
        if constexpr (CL) {
            if (threadIdx.x == 0) {
                mbar_init(&sh.bar[0], 1);
                mbar_init(&sh.bar[1], 1);
                sh.abort = 0;
                fence_barrier_init();
            }
            cluster_sync();
        }
    }

    __device__ __forceinline__ static float swap(float v, int o) { return __shfl_xor_sync(0xFFFFFFFFu, v, o); }

    // the warp's sum number lane / (32 / N)
    template <int N>
    __device__ __forceinline__ float dealt(const float (&v)[N]) const
    {
        float x;
        if constexpr (N == 4) {
            const bool up = lane & 16, odd = lane & 8;
            const float a = (up ? v[2] : v[0]) + swap(up ? v[0] : v[2], 16), b = (up ? v[3] : v[1]) + swap(up ? v[1] : v[3], 16);
            x = (odd ? b : a) + swap(odd ? a : b, 8);
        } else if constexpr (N == 2) {
            const bool up = lane & 16;
            x = (up ? v[1] : v[0]) + swap(up ? v[0] : v[1], 16);
        } else {
            x = v[0] + swap(v[0], 16);
        }
        return over_share<32 / N>(x);
    }
    template <int kShare>
    __device__ __forceinline__ static float over_share(float x)
    {
#pragma unroll
        for (int o = kShare == 32 ? 8 : kShare / 2; o > 0; o >>= 1) x += swap(x, o);
        return x;
    }

    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N], const Place& p)
    {
        constexpr int kShare = 32 / N;   // lanes that end up with the same sum
        if (!CL && width < 32) {   // a power of two
            for (int o = width >> 1; o > 0; o >>= 1) {
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] += swap(v[k], o);
            }
            return;
        }
        float x = dealt(v);
        if (CL || warps > 1) {
            float* buf = sh.red[turn] + lane / kShare * kTeamWarps;
            if constexpr (CL) {
                if (threadIdx.x == 0) mbar_arrive_expect_tx(&sh.bar[turn], static_cast<uint32_t>(ctas * warps * N * 4));
                if (lane % kShare < ctas) send(buf + own, &sh.bar[turn], lane % kShare, x);
                __syncwarp();
                const bool came = mbar_wait_bounded(&sh.bar[turn], phase, &sh.abort, kDefaultTimeoutNs);
                if (!came) sh.abort = 1;
                x = came ? 0.0f : __uint_as_float(0x7FC00000u);   // a row whose sums did not come is NaN
                for (int i = lane % kShare; i < ctas * warps; i += kShare) x += buf[first + i];
                phase ^= turn;
                if constexpr (N == 1) x += swap(x, 16);
            } else {
                if (lane % kShare == 0) buf[own] = x;
                named_bar_sync(1 + p.team, width);
                // sixteen warps at most
                const int i = lane % (kShare < 16 ? kShare : 16);
                x = i < warps ? buf[first + i] : 0.0f;
                if (kShare < 16 && i + kShare < warps) x += buf[first + i + kShare];
            }
            turn ^= 1;
            x = over_share<kShare>(x);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = N == 1 ? x : __shfl_sync(0xFFFFFFFFu, x, k * kShare);
    }
};

// Which rows a team takes: r0 + i * step + q * apart, q < R; `turns` values of i
// at most in any team of the CTA or cluster, `mine` with such a row for q in this.
template <int R>
struct Walk {
    long long r0, step;
    int turns, mine[R];

    __device__ __forceinline__ Walk(const JoinArgs& a, const Place& p, int teams)
    {
        const long long group = blockIdx.x / p.ctas, groups = gridDim.x / p.ctas, apart = a.apart;
        const long long lane = group / apart * teams;
        r0 = group % apart + apart * R * (lane + p.team);
        step = apart * R * (groups / apart) * teams;
        const auto count = [&](long long first) { return first < a.rows ? static_cast<int>((a.rows - first + step - 1) / step) : 0; };
        turns = count(group % apart + apart * R * lane);
#pragma unroll
        for (int q = 0; q < R; ++q) mine[q] = count(r0 + q * apart);
    }
};

// A thread's columns.
template <int DT, int NCH, int MODE>
struct Cols {
    static constexpr int V = kV<DT>;
    int c[NCH];          // first column of the word
    int base, apart;     // kSingle: column of element e is base + e * apart
    bool some[NCH], any, whole;   // whether there is a word; whether any is; whether all are, inside the row

    __device__ __forceinline__ Cols(const Place& p, int cols)
    {
        const int all = p.ctas * p.width, g = p.rank * p.width + p.t;
        base = g;
        apart = all;
        whole = true;
        any = MODE == kSingle;
        if constexpr (MODE != kSingle) {
            const int words = (cols + p.first + V - 1) / V;
#pragma unroll
            for (int k = 0; k < NCH; ++k) {
                // kAlike: slot 0 takes the last word, so that a row's two words
                // that need care are in one warp
                const int slot = g + k * all;
                const int j = MODE == kWhole ? slot : slot == 0 ? words - 1 : slot - 1;
                some[k] = slot < words;
                any = any || some[k];
                c[k] = some[k] ? j * V - p.first : cols;
                whole = whole && some[k] && c[k] >= 0 && c[k] + V <= cols;
            }
        }
    }
    // column of element e of word k, and whether it is one
    __device__ __forceinline__ int at(int k, int e) const { return MODE != kSingle ? c[k] + e : base + (k * V + e) * apart; }
    __device__ __forceinline__ bool is(int k, int e, int cols) const
    {
        const int i = at(k, e);
        return i >= 0 && i < cols;
    }
};

// Where a thread's first word of the row of this turn lies in the arrays, in bytes
// from their starts (kSingle: where the row does).  Arrays of one kind share rows'
// places: the residual's, the block's output's, the next block's input's, a gate's
// for every token.  (An address for each array took twice the registers.)
enum { kH = 0, kO = 1, kY = 2, kG = 3 };
template <int DT, int NCH, int MODE>
struct Places {
    long long at[4];

    __device__ __forceinline__ Places(const JoinArgs& a, long long row, const Cols<DT, NCH, MODE>& c)
    {
        constexpr int es = sizeof(typename El<DT>::T);
#pragma unroll
        for (int k = 0; k < 4; ++k) at[k] = (row * a.stride[k] + (MODE != kSingle ? c.c[0] : 0)) * es;
    }
    template <bool TOK>
    __device__ __forceinline__ void advance(const JoinArgs& a)
    {
#pragma unroll
        for (int k = 0; k < (TOK ? 4 : 3); ++k) at[k] += a.step[k];
    }
};

// The arrays that a thread reads, row by row.  Slot of word k of array n of row q
// of a stage: ((q * NA + n) * NCH + k) * apart bytes on.
template <int DT, int NCH, int R, int NA, int MODE, bool FORWARD>
struct Inputs {
    using T = typename El<DT>::T;
    static constexpr int V = kV<DT>;
    const Cols<DT, NCH, MODE>& c;
    const JoinArgs& a;
    const Walk<R>& walk;
    int apart;
    bool plain;          // this thread's words are whole

    __device__ __forceinline__ static constexpr int kind(int n)
    {
        return FORWARD ? (n == 0 ? kH : n == 1 ? kO : kG) : (n == 1 ? kY : n == 3 ? kO : n == 4 ? kG : kH);
    }

    __device__ __forceinline__ Inputs(const Cols<DT, NCH, MODE>& cols, const JoinArgs& args, const Walk<R>& w) : c(cols), a(args), walk(w), apart(blockDim.x * 16)
    {
        plain = c.whole;
    }
    // (a forward pass has all of its arrays)
    __device__ __forceinline__ bool there(int n) const { return FORWARD || a.in[n] != nullptr; }

    // zeros where nothing will come
    __device__ __forceinline__ void clear(unsigned char* mine, int stages) const
    {
        if constexpr (MODE != kSingle) {
            for (int i = 0; i < stages * R; ++i)
#pragma unroll
                for (int n = 0; n < NA; ++n)
                    if (!plain || !there(n))
                        for (int k = 0; k < NCH; ++k) *reinterpret_cast<uint4*>(mine + ((i * NA + n) * NCH + k) * apart) = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // turn i's rows into a stage's slots; `ahead` turns from the one that `places` holds
    __device__ __forceinline__ void issue(unsigned char* slot, int i, int ahead, const Places<DT, NCH, MODE>& places) const
    {
        if constexpr (MODE != kSingle) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (i < walk.mine[q]) {
                    if (plain) {
#pragma unroll
                        for (int n = 0; n < NA; ++n) {
                            if (!there(n)) continue;
                            const char* p = static_cast<const char*>(a.in[n]) + (ahead * a.step[kind(n)] + q * a.gap[kind(n)]) + places.at[kind(n)];
#pragma unroll
                            for (int k = 0; k < NCH; ++k)
                                cp_async16(slot + ((q * NA + n) * NCH + k) * apart, p + (c.c[k] - c.c[0]) * static_cast<int>(sizeof(T)));
                        }
                    } else {
                        some_words(slot, i, q);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NA * NCH; ++n) *reinterpret_cast<uint4*>(slot + (q * NA * NCH + n) * apart) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            cp_async_commit();
        }
    }
    __device__ __forceinline__ void some_words(unsigned char* slot, int i, int q) const
    {
        const long long row = walk.r0 + i * walk.step + q * a.apart;
        const bool ends = row < a.edge || row >= a.rows - a.edge;
#pragma unroll
        for (int n = 0; n < NA; ++n) {
            if (a.in[n] == nullptr) continue;
            const RowSource<DT> src(a.in[n], a.stride[kind(n)], a.rows, a.cols);
            const uintptr_t from = src.row(row), to = from + static_cast<uintptr_t>(a.cols) * sizeof(T);
#pragma unroll
            for (int k = 0; k < NCH; ++k)
                if (c.some[k])
                    src.copy_word(reinterpret_cast<uint4*>(slot + ((q * NA + n) * NCH + k) * apart),
                                  from + static_cast<intptr_t>(c.c[k]) * static_cast<intptr_t>(sizeof(T)), from, to, ends);
        }
    }

    // array n of row q of turn i, which `places` holds; zeros for what is not there
    __device__ __forceinline__ void read(f32x2 (&x)[NCH * V / 2], int n, int q, const unsigned char* slot, int i, const Places<DT, NCH, MODE>& places) const
    {
        if constexpr (MODE != kSingle) {
            uint4 w[NCH];
#pragma unroll
            for (int k = 0; k < NCH; ++k) w[k] = *reinterpret_cast<const uint4*>(slot + ((q * NA + n) * NCH + k) * apart);
            if (MODE == kAlike && !c.whole) {
#pragma unroll
                for (int k = 0; k < NCH; ++k) w[k] = masked<DT>(w[k], c.c[k], a.cols);
            }
#pragma unroll
            for (int k = 0; k < NCH; ++k) {
                f32x2 v[V / 2];
                widen<DT>(w[k], v);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) x[k * V / 2 + e] = v[e];
            }
        } else {
            const bool active = a.in[n] != nullptr && i < walk.mine[q];
            const T* r = reinterpret_cast<const T*>(static_cast<const char*>(a.in[n]) + q * a.gap[kind(n)] + places.at[kind(n)]);
#pragma unroll
            for (int e = 0; e < NCH * V; e += 2) {
                const int lo = c.at(0, e), hi = c.at(0, e + 1);
                x[e / 2] = pack2(active && lo < a.cols ? El<DT>::up(r[lo]) : 0.0f, active && hi < a.cols ? El<DT>::up(r[hi]) : 0.0f);
            }
        }
    }
};

// A thread's words of row q of an array of kind K.
template <int K, int DT, int NCH, int MODE>
__device__ __forceinline__ void put_row(void* array, int q, const uint4 (&w)[NCH], const Cols<DT, NCH, MODE>& c, const JoinArgs& a, const Places<DT, NCH, MODE>& places)
{
    using T = typename El<DT>::T;
    char* at = static_cast<char*>(array) + q * a.gap[K] + places.at[K];
    if constexpr (MODE != kSingle) {
        if (c.whole) {
#pragma unroll
            for (int k = 0; k < NCH; ++k) __stcs(reinterpret_cast<uint4*>(at + (c.c[k] - c.c[0]) * static_cast<int>(sizeof(T))), w[k]);
        } else if (c.any) {
#pragma unroll
            for (int k = 0; k < NCH; ++k)
                if (c.some[k]) put_word<DT>(reinterpret_cast<uintptr_t>(at - c.c[0] * static_cast<int>(sizeof(T))), c.c[k], a.cols, w[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int e = 0; e < kV<DT>; ++e) {
                if (!c.is(k, e, a.cols)) continue;
                if constexpr (sizeof(T) == 4)
                    reinterpret_cast<uint32_t*>(at)[c.at(k, e)] = u[e];
                else
                    reinterpret_cast<T*>(at)[c.at(k, e)] = static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1)));
            }
        }
    }
}

template <int DT, int NCH>
__device__ __forceinline__ void to_words(const f32x2 (&x)[NCH * kV<DT> / 2], uint4 (&w)[NCH])
{
    float f[NCH * kV<DT>];
    unpack(x, f);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
        float v[kV<DT>];
#pragma unroll
        for (int e = 0; e < kV<DT>; ++e) v[e] = f[k * kV<DT> + e];
        w[k] = narrowed<DT>(v);
    }
}

// a vector's columns of this thread; `none` without a vector, 0 where there is no column
template <int DT, int NCH, int MODE>
__device__ __forceinline__ void read_vector(f32x2 (&x)[NCH * kV<DT> / 2], const void* w, int dt, float none, const Cols<DT, NCH, MODE>& c, int cols)
{
    constexpr int V = kV<DT>;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float lo = !c.is(k, e, cols) ? 0.0f : w == nullptr ? none : weight_at(w, dt, c.at(k, e));
            const float hi = !c.is(k, e + 1, cols) ? 0.0f : w == nullptr ? none : weight_at(w, dt, c.at(k, e + 1));
            x[(k * V + e) / 2] = pack2(lo, hi);
        }
    }
}

// zeros where there is no column (a mean was taken off everywhere)
template <int DT, int NCH, int MODE>
__device__ __forceinline__ void only_columns(f32x2 (&x)[NCH * kV<DT> / 2], const Cols<DT, NCH, MODE>& c, int cols)
{
    constexpr int V = kV<DT>;
    if (MODE != kSingle && c.whole) return;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            float a, b;
            unpack2(x[(k * V + e) / 2], a, b);
            x[(k * V + e) / 2] = pack2(c.is(k, e, cols) ? a : 0.0f, c.is(k, e + 1, cols) ? b : 0.0f);
        }
}

template <int N>
__device__ __forceinline__ float sum_of(const f32x2 (&x)[N])
{
    f32x2 s = x[0], r = x[1];
#pragma unroll
    for (int i = 2; i < N; i += 2) s = add2(s, x[i]), r = add2(r, x[i + 1]);
    return both(add2(s, r));
}
template <int N>
__device__ __forceinline__ float dot_of(const f32x2 (&x)[N], const f32x2 (&y)[N])
{
    f32x2 s = mul2(x[0], y[0]), r = mul2(x[1], y[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) s = fma2(x[i], y[i], s), r = fma2(x[i + 1], y[i + 1], r);
    return both(add2(s, r));
}

// The normalised rows in place of x; mean and rstd of each.
template <int DT, int NCH, int MODE, int R, bool CL>
__device__ __forceinline__ void normalise(f32x2 (&x)[R][NCH * kV<DT> / 2], int kind, float eps, float (&mean)[R], float (&rstd)[R], TeamSum<CL>& team,
                                          const Place& p, const Cols<DT, NCH, MODE>& c, const JoinArgs& a)
{
    float s[R];
#pragma unroll
    for (int q = 0; q < R; ++q) mean[q] = 0.0f;
    if (kind == ZERO_NORM_LAYER) {
#pragma unroll
        for (int q = 0; q < R; ++q) s[q] = sum_of(x[q]);
        team(s, p);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mean[q] = s[q] * a.inv_cols;
            const f32x2 off = pack2(-mean[q], -mean[q]);
#pragma unroll
            for (int i = 0; i < NCH * kV<DT> / 2; ++i) x[q][i] = add2(x[q][i], off);
            only_columns<DT, NCH, MODE>(x[q], c, a.cols);
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) s[q] = dot_of(x[q], x[q]);
    team(s, p);
#pragma unroll
    for (int q = 0; q < R; ++q) {
        rstd[q] = inverse_root(fmaf(s[q], a.inv_cols, eps));
        const f32x2 r = pack2(rstd[q], rstd[q]);
#pragma unroll
        for (int i = 0; i < NCH * kV<DT> / 2; ++i) x[q][i] = mul2(x[q][i], r);
    }
}

__device__ __forceinline__ Place place_of(const JoinArgs& a, bool cl)
{
    Place p;
    p.width = a.width;
    p.team = threadIdx.x / a.width;
    p.t = threadIdx.x - p.team * a.width;
    p.rank = cl ? static_cast<int>(cluster_rank()) : 0;
    p.ctas = cl ? a.ctas : 1;
    // every row of this CTA starts as its first one does
    const int es = a.dtype == ZERO_FP32 ? 4 : 2;
    p.first = static_cast<int>((reinterpret_cast<uintptr_t>(a.lie) + (blockIdx.x / p.ctas % a.apart) * a.stride[kH] * es) % 16) / es;
    return p;
}

template <int DT, int NCH, int R, int DEPTH, int MODE, bool TOK, bool CL>
__global__ void __launch_bounds__(kTeamMax, 1) join_forward(const __grid_constant__ JoinArgs a)
{
    constexpr int N = NCH * kV<DT> / 2, NA = TOK ? 3 : 2;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ TeamShared sh;
    const Place p = place_of(a, CL);
    const int teams = blockDim.x / a.width;
    const Cols<DT, NCH, MODE> c(p, a.cols);
    const Walk<R> walk(a, p, teams);
    TeamSum<CL> team(sh, p);
    const Inputs<DT, NCH, R, NA, MODE, true> in(c, a, walk);
    Places<DT, NCH, MODE> places(a, walk.r0, c);
    float4* stats = p.t == 0 && p.rank == 0 && a.stats_out != nullptr ? reinterpret_cast<float4*>(a.stats_out) + walk.r0 : nullptr;
    const int stage = R * NA * NCH * in.apart;
    unsigned char* mine = ring + threadIdx.x * 16;
    in.clear(mine, DEPTH);
    pdl_wait();
    pdl_launch();
    for (int s = 0; s < DEPTH; ++s) in.issue(mine + s * stage, s, s, places);
    // gate * post's gain and bias; pre's gain and bias
    f32x2 pg[N], pb[N], qg[N], qb[N];
    read_vector<DT, NCH, MODE>(pg, a.post_gain, a.w_dtype, 1.0f, c, a.cols);
    read_vector<DT, NCH, MODE>(pb, a.post_bias, a.w_dtype, 0.0f, c, a.cols);
    if constexpr (!TOK) {
        read_vector<DT, NCH, MODE>(qg, a.gate, a.w_dtype, 1.0f, c, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) pg[i] = mul2(pg[i], qg[i]), pb[i] = mul2(pb[i], qg[i]);
    }
    read_vector<DT, NCH, MODE>(qg, a.pre_gain, a.w_dtype, 1.0f, c, a.cols);
    read_vector<DT, NCH, MODE>(qb, a.pre_bias, a.w_dtype, 0.0f, c, a.cols);
    const f32x2 scale = pack2(a.res_scale, a.res_scale);
    unsigned char *slot = mine, *const end = mine + DEPTH * stage;
    for (int i = 0; i < walk.turns; ++i) {
        cp_async_wait<DEPTH - 1>();
        f32x2 x[R][N];
        float mo[R], ro[R], mh[R], rh[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mo[q] = mh[q] = 0.0f, ro[q] = rh[q] = 1.0f;
            in.read(x[q], 1, q, slot, i, places);
        }
        if (a.post != ZERO_NORM_NONE) normalise<DT, NCH, MODE, R, CL>(x, a.post, a.post_eps, mo, ro, team, p, c, a);
#pragma unroll
        for (int q = 0; q < R; ++q) {
#pragma unroll
            for (int k = 0; k < N; ++k) x[q][k] = fma2(x[q][k], pg[k], pb[k]);
            // what is read late holds no registers over the sums
            f32x2 v[N];
            if constexpr (TOK) {
                in.read(v, 2, q, slot, i, places);
#pragma unroll
                for (int k = 0; k < N; ++k) x[q][k] = mul2(x[q][k], v[k]);
            }
            in.read(v, 0, q, slot, i, places);
#pragma unroll
            for (int k = 0; k < N; ++k) x[q][k] = fma2(v[k], scale, x[q][k]);
            uint4 w[NCH];
            to_words<DT, NCH>(x[q], w);
            if (i < walk.mine[q]) put_row<kH, DT, NCH, MODE>(a.out[0], q, w, c, a, places);
            // pre's norm is that of hout as it is stored
#pragma unroll
            for (int k = 0; k < NCH; ++k) {
                f32x2 u[kV<DT> / 2];
                widen<DT>(w[k], u);
#pragma unroll
                for (int e = 0; e < kV<DT> / 2; ++e) x[q][k * kV<DT> / 2 + e] = u[e];
            }
        }
        in.issue(slot, i + DEPTH, DEPTH, places);
        slot = slot + stage == end ? mine : slot + stage;
        if (a.pre != ZERO_NORM_NONE) {
            normalise<DT, NCH, MODE, R, CL>(x, a.pre, a.pre_eps, mh, rh, team, p, c, a);
#pragma unroll
            for (int q = 0; q < R; ++q) {
#pragma unroll
                for (int k = 0; k < N; ++k) x[q][k] = fma2(x[q][k], qg[k], qb[k]);
                uint4 w[NCH];
                to_words<DT, NCH>(x[q], w);
                if (i < walk.mine[q]) put_row<kY, DT, NCH, MODE>(a.out[1], q, w, c, a, places);
            }
        }
        if (stats != nullptr) {
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (i < walk.mine[q]) stats[q * a.apart] = make_float4(mo[q], ro[q], mh[q], rh[q]);
            stats += walk.step;
        }
        places.template advance<TOK>(a);
    }
    if constexpr (CL) cluster_sync();   // a CTA that ends early takes its shared memory along
}

// A row of a norm's gradient: u = the gradient of the result times the gain, with
// the team's sums of u xhat and u; rstd * (u - E(u) - xhat E(u xhat)), added to d
// or (OVER) in its place.
template <int N, bool OVER>
__device__ __forceinline__ void norm_gradient(f32x2 (&d)[N], const f32x2 (&u)[N], const f32x2 (&xhat)[N], int kind, float rstd, float along, float flat, float inv_cols)
{
    const float c = -inv_cols * rstd;
    along *= c;
    flat = kind == ZERO_NORM_LAYER ? flat * c : 0.0f;
    const f32x2 r = pack2(rstd, rstd), al = pack2(along, along), fl = pack2(flat, flat);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = fma2(u[i], r, fma2(xhat[i], al, OVER ? fl : add2(d[i], fl)));
}

template <int DT, int NCH, int DEPTH, int MODE, bool TOK, bool CL, int TT, bool LAG>
__global__ void __launch_bounds__(TT, 1) join_backward(const __grid_constant__ JoinArgs a)
{
    constexpr int V = kV<DT>, N = NCH * V / 2, NA = TOK ? 5 : 4;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ TeamShared sh;
    const Place p = place_of(a, CL);
    const int teams = blockDim.x / a.width;
    const Cols<DT, NCH, MODE> c(p, a.cols);
    const Walk<1> walk(a, p, teams);
    TeamSum<CL> team(sh, p);
    const Inputs<DT, NCH, 1, NA, MODE, false> in(c, a, walk);   // dhout, dy, hout, o, a gate for every token
    Places<DT, NCH, MODE> places(a, walk.r0, c);
    const int stage = NA * NCH * in.apart;
    unsigned char* mine = ring + threadIdx.x * 16;
    in.clear(mine, DEPTH);
    pdl_wait();
    pdl_launch();
    for (int s = 0; s < DEPTH; ++s) in.issue(mine + s * stage, s, s, places);
    // post's gain (times a gate that all rows share); its bias for each token's gate
    f32x2 pg[N], pb[TOK ? N : 1], qg[N], sum[4][N];
    read_vector<DT, NCH, MODE>(pg, a.post_gain, a.w_dtype, 1.0f, c, a.cols);
    if constexpr (!TOK) {
        read_vector<DT, NCH, MODE>(qg, a.gate, a.w_dtype, 1.0f, c, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) pg[i] = mul2(pg[i], qg[i]);
    } else {
        read_vector<DT, NCH, MODE>(pb, a.post_bias, a.w_dtype, 0.0f, c, a.cols);
    }
    read_vector<DT, NCH, MODE>(qg, a.pre_gain, a.w_dtype, 1.0f, c, a.cols);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) sum[k][i] = 0ull;
    const f32x2 scale = pack2(a.res_scale, a.res_scale);
    const float4* stats = reinterpret_cast<const float4*>(a.stats) + walk.r0;
    const bool post = a.post != ZERO_NORM_NONE, pre = a.pre != ZERO_NORM_NONE;
    const auto statistics = [&](int i) {   // of the row of turn i, the next one to be asked for
        const float4 st = a.stats != nullptr && i < walk.mine[0] ? *stats : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
        stats += walk.step;
        return st;
    };
    // Those of a norm that is not there, and an rms norm's mean, are not the caller's to
    // give.  (Looked at when a turn begins: where they are loaded, the turn before would
    // wait for them, 8192 x 4096 143 us, not 99.)
    const auto of_norms = [&](float4 st) {
        if (a.post != ZERO_NORM_LAYER) st.x = 0.0f;
        if (!post) st.y = 1.0f;
        if (a.pre != ZERO_NORM_LAYER) st.z = 0.0f;
        if (!pre) st.w = 1.0f;
        return st;
    };
    float4 next = statistics(0);
    unsigned char *slot = mine, *const end = mine + DEPTH * stage;
    // LAG: turn i takes pre's gradient of its row and post's of the row before,
    // whose sums share a barrier; a turn more finishes the last one.
    const int turns = walk.turns + (LAG && post ? 1 : 0);
    f32x2 uw[N], xw[N];   // the row before: gate * d * gain, and o normalised
    float rw = 1.0f;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < N; ++k) uw[k] = xw[k] = 0ull;
    for (int i = 0; i < turns; ++i) {
        const float4 st = of_norms(next);
        next = statistics(i + 1);
        cp_async_wait<DEPTH - 1>();
        f32x2 d[N], x[N], u[N];
        uint4 w[NCH];
        if (!LAG) in.read(d, 0, 0, slot, i, places);
        if (pre) {
            in.read(u, 1, 0, slot, i, places);
            in.read(x, 2, 0, slot, i, places);
            const Centred<DT> row(st.z, st.w);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                x[k] = row.xhat(x[k]);
                sum[2][k] = fma2(u[k], x[k], sum[2][k]);
                sum[3][k] = add2(sum[3][k], u[k]);
                u[k] = mul2(u[k], qg[k]);
            }
            s[0] = dot_of(u, x);
            s[1] = sum_of(u);
        }
        if (LAG ? pre || post : pre) {
            if constexpr (LAG) {
                team(s, p);
            } else {
                float v[2] = {s[0], s[1]};
                team(v, p);
                s[0] = v[0], s[1] = v[1];
            }
        }
        if (LAG && post && i > 0) {
            norm_gradient<N, true>(uw, uw, xw, a.post, rw, s[2], s[3], a.inv_cols);
            to_words<DT, NCH>(uw, w);
            if (i - 1 < walk.mine[0]) {
                Places<DT, NCH, MODE> before = places;
                before.at[kO] -= a.step[kO];
                put_row<kO, DT, NCH, MODE>(a.out[1], 0, w, c, a, before);
            }
        }
        if (LAG) in.read(d, 0, 0, slot, i, places);
        if (pre) norm_gradient<N, false>(d, u, x, a.pre, st.w, s[0], s[1], a.inv_cols);
        const bool active = i < walk.mine[0];
#pragma unroll
        for (int k = 0; k < N; ++k) u[k] = mul2(d[k], scale);
        to_words<DT, NCH>(u, w);
        if (active) put_row<kH, DT, NCH, MODE>(a.out[0], 0, w, c, a, places);
        in.read(xw, 3, 0, slot, i, places);
        {
            const Centred<DT> row(st.x, st.y);
#pragma unroll
            for (int k = 0; k < N; ++k) xw[k] = row.xhat(xw[k]);
        }
        if constexpr (TOK) {
            f32x2 g[N];
            in.read(g, 4, 0, slot, i, places);
            if (a.out[2] != nullptr) {
#pragma unroll
                for (int k = 0; k < N; ++k) u[k] = mul2(d[k], fma2(xw[k], pg[k], pb[k]));
                to_words<DT, NCH>(u, w);
                if (active) put_row<kG, DT, NCH, MODE>(a.out[2], 0, w, c, a, places);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) d[k] = mul2(d[k], g[k]);
        }
        in.issue(slot, i + DEPTH, DEPTH, places);
        slot = slot + stage == end ? mine : slot + stage;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            sum[0][k] = fma2(d[k], xw[k], sum[0][k]);
            sum[1][k] = add2(sum[1][k], d[k]);
            uw[k] = mul2(d[k], pg[k]);
        }
        if (post) {
            s[2] = dot_of(uw, xw);
            s[3] = sum_of(uw);
            rw = st.y;
        }
        if (!LAG && post) {
            float v[2] = {s[2], s[3]};
            team(v, p);
            norm_gradient<N, true>(uw, uw, xw, a.post, rw, v[0], v[1], a.inv_cols);
        }
        if (!LAG || !post) {
            to_words<DT, NCH>(uw, w);
            if (active) put_row<kO, DT, NCH, MODE>(a.out[1], 0, w, c, a, places);
        }
        places.template advance<TOK>(a);
    }
    if (a.parts == nullptr) {
        if constexpr (CL) cluster_sync();
        return;
    }
    // the teams' sums in order, then a part of this CTA or cluster
    cp_async_wait<0>();
    float* sums = reinterpret_cast<float*>(ring);
    float* part = a.parts + static_cast<long long>(blockIdx.x / p.ctas) * 4 * a.pitch;
    for (int q = 0; q < 4; ++q) {
        float f[2 * N];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k == q) unpack(sum[k], f);
        if (teams > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) sums[e * blockDim.x + threadIdx.x] = f[e];
            __syncthreads();
        }
        if (p.team != 0) continue;
#pragma unroll
        for (int e = 0; e < 2 * N; ++e) {
            float v = f[e];
            for (int m = 1; m < teams; ++m) v += sums[e * blockDim.x + m * a.width + p.t];
            if (c.is(e / V, e % V, a.cols)) part[q * a.pitch + c.at(e / V, e % V)] = v;
        }
    }
    if constexpr (CL) cluster_sync();
}

// The parts' sums in a fixed order, 32 columns a CTA and sixteen slices of the
// parts side by side; then the vectors' gradients.
__global__ void __launch_bounds__(512) join_finish(const __grid_constant__ JoinArgs a, int parts)
{
    __shared__ float red[16][4][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    pdl_wait();
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i < a.cols) {
#pragma unroll 4
        for (int k = slice; k < parts; k += 16) {
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] += a.parts[(static_cast<long long>(k) * 4 + q) * a.pitch + i];
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) red[slice][q][lane] = s[q];
    __syncthreads();
    if (slice >= 4 || i >= a.cols) return;
    float v[16];
    // warp q adds the slices of sum q, pairwise; warp 0 then needs sum 1 too
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = red[k][slice][lane];
#pragma unroll
    for (int n = 8; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += v[k + n];
    const bool vector = a.gate != nullptr;
    const float gate = vector ? weight_at(a.gate, a.w_dtype, i) : 1.0f;
    if (slice == 2 && a.dpre_gain != nullptr) put_weight(a.dpre_gain, a.w_dtype, i, v[0]);
    if (slice == 3 && a.dpre_bias != nullptr) put_weight(a.dpre_bias, a.w_dtype, i, v[0]);
    if (slice == 0 && a.dpost_gain != nullptr) put_weight(a.dpost_gain, a.w_dtype, i, gate * v[0]);
    if (slice == 1 && a.dpost_bias != nullptr) put_weight(a.dpost_bias, a.w_dtype, i, gate * v[0]);
    if (slice == 0 && vector && a.dgate != nullptr) {
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = red[k][1][lane];
#pragma unroll
        for (int n = 8; n > 0; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) f[k] += f[k + n];
        const float gain = a.post_gain != nullptr ? weight_at(a.post_gain, a.w_dtype, i) : 1.0f;
        const float bias = a.post_bias != nullptr ? weight_at(a.post_bias, a.w_dtype, i) : 0.0f;
        put_weight(a.dgate, a.w_dtype, i, fmaf(gain, v[0], bias * f[0]));
    }
}

// ------------------------------------------------------------------- host
struct Shape {
    int width, teams, ctas, threads;
    long long grid;
    size_t smem;
};

template <int DT, int NCH, int R, int TT>
Shape shape_of(const JoinArgs& a, int mode, int stage_arrays, int depth, int per_sm, int sms)
{
    constexpr int V = kV<DT>;
    Shape s;
    // kAlike: rows may start inside a word
    const int chunks = (a.cols + V - 1 + (mode == kAlike ? V - 1 : 0)) / V;
    const int each = (chunks + NCH - 1) / NCH;   // threads that a row takes
    s.ctas = 1;
    while (each > s.ctas * TT) s.ctas *= 2;
    const int here = (each + s.ctas - 1) / s.ctas;
    s.width = 32;
    if (s.ctas == 1 && here <= 16)
        for (s.width = 1; s.width < here; s.width *= 2) {}
    else
        s.width = (here + 31) / 32 * 32;
    s.teams = s.ctas > 1 ? 1 : TT / s.width;
    // fewer where the rows would not cover the SMs otherwise
    const long long sets = (a.rows + R - 1) / R, spread = (sets + sms - 1) / sms;
    if (s.teams > spread) s.teams = static_cast<int>(spread);
    if (s.teams < 1) s.teams = 1;
    if (s.width < 32) s.teams = (s.teams + 32 / s.width - 1) / (32 / s.width) * (32 / s.width);   // whole warps
    s.threads = s.width * s.teams;
    const int stage = R * stage_arrays * NCH * s.threads * 16, sums = s.threads * NCH * V * 4;
    s.smem = static_cast<size_t>(mode != kSingle ? stage * depth : 0);
    if (s.smem < static_cast<size_t>(sums)) s.smem = sums;
    long long groups = (sets + s.teams - 1) / s.teams;
    const long long most = static_cast<long long>(sms) * per_sm / s.ctas;
    if (groups > most) groups = most;
    if (groups > kJoinMaxParts) groups = kJoinMaxParts;
    groups = groups < a.apart ? a.apart : groups / a.apart * a.apart;
    s.grid = groups * s.ctas;
    return s;
}

constexpr size_t kJoinSmem = 200 * 1024;

template <typename K>
cudaError_t launch_join(K kernel, const JoinArgs& a, const Shape& s, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kJoinSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c;
    std::memset(&c, 0, sizeof(c));
    c.gridDim = dim3(static_cast<unsigned>(s.grid));
    c.blockDim = dim3(s.threads);
    c.dynamicSmemBytes = s.smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = s.ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = s.ctas > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&c, kernel, a);
}

// How the rows of all the arrays lie (`outputs` from `inputs` on in `kinds`); where
// equal rows start equally far into a word but not all rows do, alike ones are
// kApart apart.
template <int DT>
int mode_of(JoinArgs& a, std::initializer_list<int> in, std::initializer_list<int> out)
{
    constexpr int V = kV<DT>;
    a.lie = a.out[0];   // a residual row's
    long long least = a.stride[kH];
    bool alike = true;
    const auto look = [&](const void* p, int kind) {
        if (p == nullptr) return;
        if (a.stride[kind] < least) least = a.stride[kind];
        alike = alike && (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(a.lie)) % 16 == 0 && (a.stride[kind] - a.stride[kH]) % V == 0;
    };
    int n = 0;
    for (int k : in) look(a.in[n++], k);
    n = 0;
    for (int k : out) look(a.out[n++], k);
    a.apart = 1;
    a.edge = static_cast<int>((V + least - 1) / least);   // rows near the arrays' ends, whose words may reach past them
    if (!alike) return kSingle;
    const bool starts = reinterpret_cast<uintptr_t>(a.lie) % 16 == 0 && a.stride[kH] % V == 0;
    if (starts && a.cols % V == 0) return kWhole;
    if (a.stride[kH] % V != 0) a.apart = kApart;
    return kAlike;
}

// what the kernels need of a shape, with the distances from row to row and from
// one turn's rows to the next's in bytes
template <int DT, int R>
void set_shape(JoinArgs& a, const Shape& s)
{
    a.width = s.width;
    a.ctas = s.ctas;
    const long long step = static_cast<long long>(a.apart) * R * (s.grid / s.ctas / a.apart) * s.teams;
    for (int k = 0; k < 4; ++k) {
        a.gap[k] = a.apart * a.stride[k] * dtype_bytes(DT);
        a.step[k] = step * a.stride[k] * dtype_bytes(DT);
    }
}

template <int DT, int NCH, int R, int DEPTH, int MODE, bool TOK>
cudaError_t forward_as(JoinArgs& a, int sms, cudaStream_t st)
{
    const Shape s = shape_of<DT, NCH, R, kTeamMax>(a, MODE, TOK ? 3 : 2, DEPTH, 1, sms);
    set_shape<DT, R>(a, s);
    return s.ctas > 1 ? launch_join(join_forward<DT, NCH, R, DEPTH, MODE, TOK, true>, a, s, st)
                      : launch_join(join_forward<DT, NCH, R, DEPTH, MODE, TOK, false>, a, s, st);
}

template <int DT, int MODE>
cudaError_t forward_of(JoinArgs& a, int sms, cudaStream_t st)
{
    constexpr int W = DT == ZERO_FP32 ? 2 : 1;
    if (a.cols > 4096)   // rows of more than 512 threads' words: one at a time, twice the words
        return a.token_gate ? forward_as<DT, 2 * W, 1, 4 - W, MODE, true>(a, sms, st) : forward_as<DT, 2 * W, 1, 3, MODE, false>(a, sms, st);
    return a.token_gate ? forward_as<DT, W, 2, 4 - W, MODE, true>(a, sms, st) : forward_as<DT, W, 2, 3, MODE, false>(a, sms, st);
}

template <int DT, int NCH, int DEPTH, int MODE, bool TOK, int TT, bool LAG>
cudaError_t backward_as(JoinArgs& a, int sms, cudaStream_t st)
{
    const Shape s = shape_of<DT, NCH, 1, TT>(a, MODE, TOK ? 5 : 4, DEPTH, 1, sms);
    set_shape<DT, 1>(a, s);
    const bool sums = a.dpost_gain != nullptr || a.dpost_bias != nullptr || a.dpre_gain != nullptr || a.dpre_bias != nullptr || a.dgate != nullptr;
    if (!sums) a.parts = nullptr;
    cudaError_t e = cudaSuccess;
    const int parts = a.rows > 0 ? static_cast<int>(s.grid / s.ctas) : 0;
    if (a.rows > 0)
        e = s.ctas > 1 ? launch_join(join_backward<DT, NCH, DEPTH, MODE, TOK, true, TT, LAG>, a, s, st)
                       : launch_join(join_backward<DT, NCH, DEPTH, MODE, TOK, false, TT, LAG>, a, s, st);
    if (e != cudaSuccess || !sums) return e;
    return launch_after(join_finish, dim3((a.cols + 31) / 32), dim3(512), 0, st, a, parts);
}

template <int DT, int MODE>
cudaError_t backward_of(JoinArgs& a, int sms, cudaStream_t st)
{
    constexpr int W = DT == ZERO_FP32 ? 2 : 1, D = DT == ZERO_FP32 ? 3 : 4;
    if (a.cols > 2048)
        return a.token_gate ? backward_as<DT, 2 * W, D - 1, MODE, true, 256, false>(a, sms, st) : backward_as<DT, 2 * W, D, MODE, false, 256, true>(a, sms, st);
    return a.token_gate ? backward_as<DT, W, D - 1, MODE, true, 512, false>(a, sms, st) : backward_as<DT, W, D, MODE, false, 512, false>(a, sms, st);
}

template <int DT>
cudaError_t forward_typed(JoinArgs& a, int sms, cudaStream_t st)
{
    const int mode = mode_of<DT>(a, {kH, kO, kG}, {kH, kY});
    if (mode == kWhole) return forward_of<DT, kWhole>(a, sms, st);
    return mode == kAlike ? forward_of<DT, kAlike>(a, sms, st) : forward_of<DT, kSingle>(a, sms, st);
}

template <int DT>
cudaError_t backward_typed(JoinArgs& a, int sms, cudaStream_t st)
{
    const int mode = a.rows > 0 ? mode_of<DT>(a, {kH, kY, kH, kO, kG}, {kH, kO, kG}) : kSingle;
    if (mode == kWhole) return backward_of<DT, kWhole>(a, sms, st);
    return mode == kAlike ? backward_of<DT, kAlike>(a, sms, st) : backward_of<DT, kSingle>(a, sms, st);
}

}  // namespace

cudaError_t launch_join_forward(JoinArgs a, cudaStream_t st)
{
    if (a.rows == 0) return cudaSuccess;
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    if (a.dtype == ZERO_FP32) return forward_typed<ZERO_FP32>(a, sms, st);
    return a.dtype == ZERO_BF16 ? forward_typed<ZERO_BF16>(a, sms, st) : forward_typed<ZERO_FP16>(a, sms, st);
}

cudaError_t launch_join_backward(JoinArgs a, cudaStream_t st)
{
    const int sms = sms_of_device();
    if (sms == 0) return cudaErrorInvalidDevice;
    if (a.dtype == ZERO_FP32) return backward_typed<ZERO_FP32>(a, sms, st);
    return a.dtype == ZERO_BF16 ? backward_typed<ZERO_BF16>(a, sms, st) : backward_typed<ZERO_FP16>(a, sms, st);
}

}  // namespace zk
