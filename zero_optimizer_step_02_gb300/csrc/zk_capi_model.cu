// zk_capi_model.cu -- the C entry points of the operators around a language
// model's matrix products: argument checks and workspace layout.  Declarations
// and the contract of every entry point are in include/zero.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <new>

#include "zk_capi.h"
#include "zk_ops.h"

// A list of tensors is opaque to callers.
struct zero_tensors {
    zk::TensorList list;
};

namespace {

using zk::as_stream;
using zk::from_cuda;

bool dtype_ok(int dt) { return dt == ZERO_BF16 || dt == ZERO_FP16 || dt == ZERO_FP32; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

zero_status check_elems(const void* p, int es)
{
    if (p == nullptr) return ZERO_ERR_INVALID_ARG;
    return zk::aligned(p, es) ? ZERO_OK : ZERO_ERR_MISALIGNED;
}

// ------------------------------------------------- AdamW over many tensors
zero_status check_tensor(const zero_tensor& t)
{
    if (t.n < 0 || !dtype_ok(t.grad_dtype)) return ZERO_ERR_INVALID_ARG;
    if (t.state_bits != 8 && t.state_bits != 32) return ZERO_ERR_INVALID_ARG;
    if (!(t.lr_scale >= 0.0f) || std::isinf(t.lr_scale) || !(t.wd_scale >= 0.0f) || std::isinf(t.wd_scale))
        return ZERO_ERR_INVALID_ARG;
    if (t.lp != nullptr && t.lp_dtype != ZERO_BF16 && t.lp_dtype != ZERO_FP16) return ZERO_ERR_INVALID_ARG;
    if (t.n > ZERO_MAX_TENSOR_ELEMS) return ZERO_ERR_BOUNDS;
    if (t.n == 0) return ZERO_OK;
    zero_status s;
    const int state = t.state_bits == 8 ? 1 : 4;
    if ((s = check_elems(t.grad, zk::dtype_bytes(t.grad_dtype))) != ZERO_OK) return s;
    if ((s = check_elems(t.master, 4)) != ZERO_OK) return s;
    if ((s = check_elems(t.m, state)) != ZERO_OK || (s = check_elems(t.v, state)) != ZERO_OK) return s;
    if (t.lp != nullptr && !zk::aligned(t.lp, 2)) return ZERO_ERR_MISALIGNED;
    if (t.state_bits == 8 && ((s = check_elems(t.m_scale, 4)) != ZERO_OK || (s = check_elems(t.v_scale, 4)) != ZERO_OK)) return s;
    return ZERO_OK;
}

void add_range(zk::TensorList& list, const void* p, long long bytes, bool written)
{
    if (p == nullptr || bytes == 0) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    list.ranges.push_back({at, at + static_cast<uintptr_t>(bytes), written});
}

void add_ranges(zk::TensorList& list, const zero_tensor& t)
{
    const long long blocks = (t.n + zk::kStateBlock - 1) / zk::kStateBlock, state = t.state_bits == 8 ? 1 : 4;
    add_range(list, t.grad, t.n * zk::dtype_bytes(t.grad_dtype), false);
    add_range(list, t.master, 4 * t.n, true);
    add_range(list, t.m, state * t.n, true);
    add_range(list, t.v, state * t.n, true);
    add_range(list, t.lp, 2 * t.n, true);
    if (t.state_bits == 8) {
        add_range(list, t.m_scale, 4 * blocks, true);
        add_range(list, t.v_scale, 4 * blocks, true);
    }
}

// sorts the ranges; whether one that is written shares a byte with another
bool ranges_clash(zk::TensorList& list)
{
    std::sort(list.ranges.begin(), list.ranges.end(),
              [](const zk::TensorList::Range& a, const zk::TensorList::Range& b) { return a.at < b.at; });
    uintptr_t any = 0, written = 0;
    for (const auto& r : list.ranges) {
        if (r.at < written || (r.written && r.at < any)) return true;
        any = std::max(any, r.end);
        if (r.written) written = std::max(written, r.end);
    }
    return false;
}

// whether [p, p + bytes) shares a byte with any of the sorted ranges
bool meets(const zk::TensorList& list, const void* p, size_t bytes)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), end = at + bytes;
    auto it = std::lower_bound(list.ranges.begin(), list.ranges.end(), end,
                               [](const zk::TensorList::Range& r, uintptr_t x) { return r.at < x; });
    // written ranges share nothing; gradients may share with each other, so the
    // furthest end among the earlier ones was kept with each (zero_tensors_create)
    return it != list.ranges.begin() && std::prev(it)->end > at;
}

zk::TensorEntry entry_of(const zero_tensor& t, int tile0)
{
    zk::TensorEntry e;
    std::memset(&e, 0, sizeof(e));
    e.grad = t.grad;
    e.master = t.master;
    e.m = t.m;
    e.v = t.v;
    e.m_scale = t.m_scale;
    e.v_scale = t.v_scale;
    e.lp = t.lp;
    e.n = t.n;
    e.tile0 = tile0;
    e.lr_scale = t.lr_scale;
    e.wd_scale = t.wd_scale;
    e.grad_dtype = static_cast<unsigned char>(t.grad_dtype);
    e.lp_dtype = static_cast<unsigned char>(t.lp_dtype);
    e.eight = t.state_bits == 8;
    const void* all[] = {t.grad, t.master, t.m, t.v, t.lp};
    e.wide = 1;
    for (const void* p : all)
        if (!zk::aligned(p, 16)) e.wide = 0;
    return e;
}

template <int CAP>
void start(zk::TensorTable<CAP>& t)
{
    std::memset(&t, 0, sizeof(t));
}

void fill(zk::TensorList& list, int n, const zero_tensor* tensors)
{
    const long long most = 1LL << 30;   // tiles of one launch
    const auto in_ring = [](const zk::TensorEntry& e) { return e.wide && e.eight && e.n >= zk::kTensorTile; };
    const auto tiles_of = [](const zero_tensor& t) { return (t.n + zk::kTensorTile - 1) / zk::kTensorTile; };
    int used = 0;
    long long tiles = 0;
    for (int i = 0; i < n; ++i)
        if (tensors[i].n > 0) ++used, tiles += tiles_of(tensors[i]);
    start(list.small);
    if (used <= zk::kTableMin && tiles <= most) {
        for (int i = 0; i < n; ++i) {
            if (tensors[i].n == 0) continue;
            list.small.e[list.small.n] = entry_of(tensors[i], list.small.tiles);
            list.small.ring |= in_ring(list.small.e[list.small.n++]);
            list.small.tiles += static_cast<int>(tiles_of(tensors[i]));
        }
        list.partials = zk::norm_grid(list.small.tiles);
        return;
    }
    for (int i = 0; i < n; ++i) {
        if (tensors[i].n == 0) continue;
        const long long more = tiles_of(tensors[i]);
        if (list.big.empty() || list.big.back().n == zk::kTableMax || list.big.back().tiles + more > most) {
            list.big.emplace_back();
            start(list.big.back());
        }
        zk::TensorTable<zk::kTableMax>& t = list.big.back();
        t.e[t.n] = entry_of(tensors[i], t.tiles);
        t.ring |= in_ring(t.e[t.n++]);
        t.tiles += static_cast<int>(more);
    }
    list.partials = 0;
    for (const auto& t : list.big) list.partials += zk::norm_grid(t.tiles);
}

// ------------------------------------------------------------ residual join
bool kind_ok(int k) { return k == ZERO_NORM_NONE || k == ZERO_NORM_LAYER || k == ZERO_NORM_RMS; }

long long stride_of(long long s, int cols) { return s == 0 ? cols : s; }

zero_status check_join(const zero_residual_norm* d)
{
    if (d == nullptr) return ZERO_ERR_INVALID_ARG;
    if (d->rows < 0 || d->rows > (1LL << 40) || d->cols < 1) return ZERO_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->w_dtype) || !kind_ok(d->post) || !kind_ok(d->pre)) return ZERO_ERR_INVALID_ARG;
    for (float e : {d->post_eps, d->pre_eps})
        if (!(e >= 0.0f) || std::isinf(e)) return ZERO_ERR_INVALID_ARG;
    if (!std::isfinite(d->res_scale)) return ZERO_ERR_INVALID_ARG;
    if (d->cols > ZERO_MAX_RESIDUAL_COLS) return ZERO_ERR_BOUNDS;
    for (long long s : {d->h_stride, d->o_stride, d->y_stride, d->gate_stride}) {
        if (s != 0 && (s < d->cols || s > (1LL << 40))) return ZERO_ERR_INVALID_ARG;
        // an array's extent in bytes is reckoned in 64 bits
        if (d->rows > (1LL << 58) / stride_of(s, d->cols)) return ZERO_ERR_INVALID_ARG;
    }
    return ZERO_OK;
}

// a single row's stride says nothing
long long row_stride(const zero_residual_norm* d, long long s) { return d->rows == 1 ? d->cols : stride_of(s, d->cols); }

zk::JoinArgs join_args(const zero_residual_norm* d, const void* gate)
{
    zk::JoinArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = d->rows;
    a.cols = d->cols;
    a.dtype = d->dtype;
    a.w_dtype = d->w_dtype;
    a.post = d->post;
    a.pre = d->pre;
    a.post_eps = d->post_eps;
    a.pre_eps = d->pre_eps;
    a.res_scale = d->res_scale;
    a.inv_cols = 1.0f / static_cast<float>(d->cols);
    a.token_gate = gate != nullptr && d->gate_stride != 0;
    a.gate = a.token_gate ? nullptr : gate;
    a.pitch = (d->cols + 7) / 8 * 8;
    a.stride[0] = row_stride(d, d->h_stride);
    a.stride[1] = row_stride(d, d->o_stride);
    a.stride[2] = row_stride(d, d->y_stride);
    a.stride[3] = row_stride(d, d->gate_stride);
    return a;
}

// An output that shares bytes with an input without being it (the same start and
// stride), or with another output at all.
bool rows_clash(const zk::JoinArgs& a, std::initializer_list<int> in, std::initializer_list<int> out)
{
    const int es = zk::dtype_bytes(a.dtype);
    const auto clash = [&](const void* x, int kx, const void* y, int ky, bool same) {
        return x != nullptr && y != nullptr && ((!same && x == y) || zk::shares(x, a.stride[kx], y, a.stride[ky], a.rows, a.cols, es));
    };
    int i = 0;
    for (int ko : out) {
        int k = 0;
        for (int ki : in)
            if (clash(a.in[k++], ki, a.out[i], ko, true)) return true;
        k = 0;
        for (int ke : out) {
            if (k == i) break;
            if (clash(a.out[k++], ke, a.out[i], ko, false)) return true;
        }
        ++i;
    }
    return false;
}

struct Bytes {
    const void* p;
    long long n;
};

bool overlap(const Bytes& a, const Bytes& b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && a.n > 0 && b.n > 0 && x < y + static_cast<uintptr_t>(b.n) && y < x + static_cast<uintptr_t>(a.n);
}

// Whether bytes of `b` are bytes of a row of the array at p (between the rows' own
// bytes of a strided array there may be others').
bool meets_rows(const zk::JoinArgs& a, const void* p, int kind, const Bytes& b)
{
    const long long es = zk::dtype_bytes(a.dtype), row = a.cols * es, pitch = a.stride[kind] * es;
    if (a.rows == 0 || !overlap({p, (a.rows - 1) * pitch + row}, b)) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(b.p);
    if (y <= x) return true;   // reaches into the first row
    const long long in = static_cast<long long>((y - x) % static_cast<uintptr_t>(pitch));
    return in < row || (in + b.n > pitch && y - x < static_cast<uintptr_t>((a.rows - 1) * pitch));
}

// Whether one of `written`, beside the rows, meets a row, another of them or one of
// `read`; or a row that is written (all of `out`) one of `read`.
bool lone_clash(const zk::JoinArgs& a, std::initializer_list<int> in, std::initializer_list<int> out, std::initializer_list<Bytes> written,
                std::initializer_list<Bytes> read)
{
    const auto any_meets = [&](const void* p, int kind, std::initializer_list<Bytes> all) {
        for (const Bytes& b : all)
            if (meets_rows(a, p, kind, b)) return true;
        return false;
    };
    int i = 0;
    for (int k : in)
        if (any_meets(a.in[i++], k, written)) return true;
    i = 0;
    for (int k : out) {
        if (any_meets(a.out[i], k, written) || any_meets(a.out[i], k, read)) return true;
        ++i;
    }
    for (const Bytes* x = written.begin(); x != written.end(); ++x) {
        for (const Bytes* y = written.begin(); y != x; ++y)
            if (overlap(*x, *y)) return true;
        for (const Bytes& y : read)
            if (overlap(*x, y)) return true;
    }
    return false;
}

size_t join_parts_bytes(const zero_residual_norm* d)
{
    // at least eight: some launches deal rows out eight apart
    const long long parts = d->rows < 8 ? 8 : d->rows < zk::kJoinMaxParts ? d->rows : zk::kJoinMaxParts;
    return round256(static_cast<size_t>(parts) * 4 * ((d->cols + 7) / 8 * 8) * sizeof(float));
}

// --------------------------------------------------------------- embedding
zero_status check_embedding(const zero_embedding* d)
{
    if (d == nullptr) return ZERO_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->vocab < 1 || d->cols < 1) return ZERO_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->table_dtype)) return ZERO_ERR_INVALID_ARG;
    if (d->id_bits != 32 && d->id_bits != 64) return ZERO_ERR_INVALID_ARG;
    if (d->accumulate != 0 && d->accumulate != 1) return ZERO_ERR_INVALID_ARG;
    if (!std::isfinite(d->scale)) return ZERO_ERR_INVALID_ARG;
    if (d->tokens > ZERO_MAX_TOKENS || d->vocab > ZERO_MAX_VOCAB || d->cols > ZERO_MAX_EMBED_COLS) return ZERO_ERR_BOUNDS;
    for (long long s : {d->table_stride, d->out_stride})
        if (s != 0 && (s < d->cols || s > (1LL << 24))) return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

// The tokens are looked at once for every 2048 rows: no longer than about 0.1 s.
bool sort_too_long(const zero_embedding* d) { return d->tokens > (1LL << 48) / d->vocab; }

zk::EmbedArgs embed_args(const zero_embedding* d, const void* ids, zero_dev_scalars* sc)
{
    zk::EmbedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.ids = ids;
    a.sc = sc;
    a.tokens = d->tokens;
    a.vocab = d->vocab;
    a.padding_id = d->padding_id;
    a.cols = d->cols;
    a.id_bits = d->id_bits;
    a.dtype = d->dtype;
    a.table_dtype = d->table_dtype;
    a.accumulate = d->accumulate;
    a.scale = d->scale;
    a.table_stride = stride_of(d->table_stride, d->cols);
    a.out_stride = stride_of(d->out_stride, d->cols);
    return a;
}

// the arrays of a call: ids, rows [tokens, cols], table [vocab, cols]
void embed_arrays(const zk::EmbedArgs& a, const void* rows, const void* table, Bytes (&all)[3])
{
    const auto extent = [&](long long n, long long stride) { return n == 0 ? 0 : (n - 1) * stride + a.cols; };
    all[0] = {a.ids, a.tokens * a.id_bits / 8};
    all[1] = {rows, extent(a.tokens, a.out_stride) * zk::dtype_bytes(a.dtype)};
    all[2] = {table, extent(a.vocab, a.table_stride) * zk::dtype_bytes(a.table_dtype)};
}

bool has_norm_pass(const zero_hparams* hp) { return hp->max_norm > 0.0f || hp->loss_scaling; }

}  // namespace

extern "C" {

ZERO_API zero_status zero_tensors_create(zero_tensors** out, int n, const zero_tensor* tensors)
{
    if (out == nullptr || n < 1 || tensors == nullptr) return ZERO_ERR_INVALID_ARG;
    if (n > ZERO_MAX_TENSORS) return ZERO_ERR_BOUNDS;
    zero_status s;
    for (int i = 0; i < n; ++i)
        if ((s = check_tensor(tensors[i])) != ZERO_OK) return s;
    zero_tensors* made = nullptr;
    try {
        made = new zero_tensors;
        for (int i = 0; i < n; ++i) add_ranges(made->list, tensors[i]);
        if (ranges_clash(made->list)) {
            delete made;
            return ZERO_ERR_INVALID_ARG;
        }
        // from here on each range's end is the furthest of those before it
        for (size_t i = 1; i < made->list.ranges.size(); ++i)
            made->list.ranges[i].end = std::max(made->list.ranges[i].end, made->list.ranges[i - 1].end);
        fill(made->list, n, tensors);
    } catch (...) {   // out of host memory
        delete made;
        return ZERO_ERR_BOUNDS;
    }
    *out = made;
    return ZERO_OK;
}

ZERO_API void zero_tensors_destroy(zero_tensors* tensors) { delete tensors; }

ZERO_API size_t zero_adamw_tensors_workspace_bytes(const zero_hparams* hp, const zero_tensors* tensors)
{
    if (zk::check_hparams(hp) != ZERO_OK || tensors == nullptr || !has_norm_pass(hp)) return 0;
    return round256(static_cast<size_t>(tensors->list.partials) * sizeof(double));
}

ZERO_API zero_status zero_adamw_tensors(const zero_hparams* hp, const zero_tensors* tensors, zero_dev_scalars* sc,
                                        void* ws, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = zk::check_hparams(hp)) != ZERO_OK) return s;
    if (tensors == nullptr) return ZERO_ERR_INVALID_ARG;
    if ((s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    if (meets(tensors->list, sc, sizeof(zero_dev_scalars))) return ZERO_ERR_INVALID_ARG;
    if (has_norm_pass(hp)) {
        if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
        const size_t bytes = zero_adamw_tensors_workspace_bytes(hp, tensors);
        const uintptr_t w = reinterpret_cast<uintptr_t>(ws), c = reinterpret_cast<uintptr_t>(sc);
        if (meets(tensors->list, ws, bytes) || (w < c + sizeof(zero_dev_scalars) && c < w + bytes)) return ZERO_ERR_INVALID_ARG;
    }
    return from_cuda(zk::launch_adamw(tensors->list, *hp, sc, static_cast<double*>(ws), as_stream(stream)));
}

ZERO_API size_t zero_residual_norm_workspace_bytes(const zero_residual_norm* d)
{
    return check_join(d) != ZERO_OK ? 0 : join_parts_bytes(d);
}

ZERO_API zero_status zero_residual_norm_forward(const zero_residual_norm* d, const void* h, const void* o,
                                                const void* post_gain, const void* post_bias, const void* gate,
                                                void* hout, const void* pre_gain, const void* pre_bias, void* y,
                                                float* stats, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_join(d)) != ZERO_OK) return s;
    if (d->rows == 0) return ZERO_OK;
    const int es = zk::dtype_bytes(d->dtype), ws = zk::dtype_bytes(d->w_dtype);
    zk::JoinArgs a = join_args(d, gate);
    for (const void* p : {h, o, static_cast<const void*>(hout)})
        if ((s = check_elems(p, es)) != ZERO_OK) return s;
    if (d->pre != ZERO_NORM_NONE && (s = check_elems(y, es)) != ZERO_OK) return s;
    if (d->post == ZERO_NORM_NONE) post_gain = post_bias = nullptr;
    if (d->pre == ZERO_NORM_NONE) pre_gain = pre_bias = y = nullptr;
    for (const void* p : {post_gain, post_bias, pre_gain, pre_bias})
        if (!zk::aligned(p, ws)) return ZERO_ERR_MISALIGNED;
    if (!zk::aligned(gate, a.token_gate ? es : ws) || !zk::aligned(stats, 16)) return ZERO_ERR_MISALIGNED;
    a.in[0] = h;
    a.in[1] = o;
    a.in[2] = a.token_gate ? gate : nullptr;
    a.out[0] = hout;
    a.out[1] = y;
    const long long vec = static_cast<long long>(d->cols) * ws;
    if (rows_clash(a, {0, 1, 3}, {0, 2}) ||
        lone_clash(a, {0, 1, 3}, {0, 2}, {{stats, 16 * d->rows}}, {{post_gain, vec}, {post_bias, vec}, {a.gate, vec}, {pre_gain, vec}, {pre_bias, vec}}))
        return ZERO_ERR_INVALID_ARG;
    a.post_gain = post_gain;
    a.post_bias = post_bias;
    a.pre_gain = pre_gain;
    a.pre_bias = pre_bias;
    a.stats_out = stats;
    return from_cuda(zk::launch_join_forward(a, as_stream(stream)));
}

ZERO_API zero_status zero_residual_norm_backward(const zero_residual_norm* d, const void* dy, const void* dhout,
                                                 const void* o, const void* hout, const void* post_gain,
                                                 const void* post_bias, const void* gate, const void* pre_gain,
                                                 const float* stats, void* dh, void* d_o, void* dpost_gain,
                                                 void* dpost_bias, void* dgate, void* dpre_gain, void* dpre_bias,
                                                 void* ws, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_join(d)) != ZERO_OK) return s;
    const int es = zk::dtype_bytes(d->dtype), we = zk::dtype_bytes(d->w_dtype);
    zk::JoinArgs a = join_args(d, gate);
    const bool post = d->post != ZERO_NORM_NONE, pre = d->pre != ZERO_NORM_NONE;
    if (!post) post_gain = post_bias = nullptr, dpost_gain = dpost_bias = nullptr;
    if (!pre) pre_gain = nullptr, dpre_gain = dpre_bias = nullptr, dy = hout = nullptr;
    if (gate == nullptr) dgate = nullptr;
    if (!post && gate == nullptr) o = nullptr;
    if (d->rows > 0) {   // without rows there is nothing to point at
        for (const void* p : {static_cast<const void*>(dh), static_cast<const void*>(d_o)})
            if ((s = check_elems(p, es)) != ZERO_OK) return s;
        if (dhout != nullptr && !zk::aligned(dhout, es)) return ZERO_ERR_MISALIGNED;
        if (!pre && dhout == nullptr) return ZERO_ERR_INVALID_ARG;   // no gradient at all
        if (pre && ((s = check_elems(dy, es)) != ZERO_OK || (s = check_elems(hout, es)) != ZERO_OK)) return s;
        if ((post || gate != nullptr) && (s = check_elems(o, es)) != ZERO_OK) return s;
        if ((post || pre) && (s = zk::check_dev(stats, 16)) != ZERO_OK) return s;
    }
    for (const void* p : {post_gain, post_bias, pre_gain, static_cast<const void*>(dpost_gain), static_cast<const void*>(dpost_bias),
                          static_cast<const void*>(dpre_gain), static_cast<const void*>(dpre_bias)})
        if (!zk::aligned(p, we)) return ZERO_ERR_MISALIGNED;
    if (!zk::aligned(gate, a.token_gate ? es : we) || !zk::aligned(dgate, a.token_gate ? es : we)) return ZERO_ERR_MISALIGNED;
    if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
    a.in[0] = dhout;
    a.in[1] = dy;
    a.in[2] = hout;
    a.in[3] = o;
    a.in[4] = a.token_gate ? gate : nullptr;
    a.out[0] = dh;
    a.out[1] = d_o;
    a.out[2] = a.token_gate ? dgate : nullptr;
    if (d->rows > 0 && rows_clash(a, {0, 2, 0, 1, 3}, {0, 1, 3})) return ZERO_ERR_INVALID_ARG;
    if (d->rows > 0 && (dh == o || (a.token_gate && dh == gate))) return ZERO_ERR_INVALID_ARG;   // written before those are read
    if (a.token_gate) dgate = nullptr;
    const long long vec = static_cast<long long>(d->cols) * we;
    const Bytes stat = {post || pre ? stats : nullptr, 16 * d->rows};
    if (lone_clash(a, {0, 2, 0, 1, 3}, {0, 1, 3},
                   {{dpost_gain, vec}, {dpost_bias, vec}, {dgate, vec}, {dpre_gain, vec}, {dpre_bias, vec},
                    {ws, static_cast<long long>(join_parts_bytes(d))}},
                   {{post_gain, vec}, {post_bias, vec}, {a.gate, vec}, {pre_gain, vec}, stat}))
        return ZERO_ERR_INVALID_ARG;
    a.post_gain = post_gain;
    a.post_bias = post_bias;
    a.pre_gain = pre_gain;
    a.stats = post || pre ? stats : nullptr;
    a.dpost_gain = dpost_gain;
    a.dpost_bias = dpost_bias;
    a.dgate = dgate;
    a.dpre_gain = dpre_gain;
    a.dpre_bias = dpre_bias;
    a.parts = static_cast<float*>(ws);
    return from_cuda(zk::launch_join_backward(a, as_stream(stream)));
}

ZERO_API size_t zero_embedding_workspace_bytes(const zero_embedding* d)
{
    if (check_embedding(d) != ZERO_OK || sort_too_long(d)) return 0;
    size_t at[5];
    zk::embed_layout(d->tokens, d->vocab, d->cols, at);
    return at[4];
}

ZERO_API zero_status zero_embedding_forward(const zero_embedding* d, const void* ids, const void* table, void* out,
                                            zero_dev_scalars* sc, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_embedding(d)) != ZERO_OK) return s;
    if (d->tokens == 0) return ZERO_OK;
    if ((s = check_elems(ids, d->id_bits / 8)) != ZERO_OK) return s;
    if ((s = check_elems(table, zk::dtype_bytes(d->table_dtype))) != ZERO_OK) return s;
    if ((s = check_elems(out, zk::dtype_bytes(d->dtype))) != ZERO_OK) return s;
    if (sc != nullptr && (s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    zk::EmbedArgs a = embed_args(d, ids, sc);
    Bytes all[3];
    embed_arrays(a, out, table, all);
    if (overlap(all[0], all[1]) || overlap(all[1], all[2])) return ZERO_ERR_INVALID_ARG;
    a.table = table;
    a.out = out;
    return from_cuda(zk::launch_embed_forward(a, as_stream(stream)));
}

ZERO_API zero_status zero_embedding_backward(const zero_embedding* d, const void* ids, const void* dout, void* dtable,
                                             void* ws, zero_dev_scalars* sc, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_embedding(d)) != ZERO_OK) return s;
    if (sort_too_long(d)) return ZERO_ERR_BOUNDS;
    if (d->tokens > 0) {   // without tokens there is nothing to point at
        if ((s = check_elems(ids, d->id_bits / 8)) != ZERO_OK) return s;
        if ((s = check_elems(dout, zk::dtype_bytes(d->dtype))) != ZERO_OK) return s;
    }
    if ((s = check_elems(dtable, zk::dtype_bytes(d->table_dtype))) != ZERO_OK) return s;
    if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
    if (sc != nullptr && (s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    zk::EmbedArgs a = embed_args(d, ids, sc);
    Bytes all[3];
    embed_arrays(a, dout, dtable, all);
    const Bytes work = {ws, static_cast<long long>(zero_embedding_workspace_bytes(d))};
    if (overlap(all[0], all[2]) || overlap(all[1], all[2])) return ZERO_ERR_INVALID_ARG;
    for (const Bytes& b : all)
        if (overlap(b, work)) return ZERO_ERR_INVALID_ARG;
    a.dout = dout;
    a.dtable = dtable;
    return from_cuda(zk::launch_embed_backward(a, ws, as_stream(stream)));
}

}  // extern "C"
