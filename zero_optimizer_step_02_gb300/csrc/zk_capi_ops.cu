// zk_capi_ops.cu -- the C entry points of the training operators beside the
// optimizer step: argument checks and workspace layout.  Declarations and the
// contract of every entry point are in include/zero.h.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "zk_capi.h"
#include "zk_ops.h"

namespace {

using zk::as_stream;
using zk::from_cuda;

bool dtype_ok(int dt) { return dt == ZERO_BF16 || dt == ZERO_FP16 || dt == ZERO_FP32; }

zero_status check_elems(const void* p, int dt)
{
    if (p == nullptr) return ZERO_ERR_INVALID_ARG;
    return zk::aligned(p, zk::dtype_bytes(dt)) ? ZERO_OK : ZERO_ERR_MISALIGNED;
}

// ------------------------------------------------------------- layer norm
long long stride_of(long long s, int cols) { return s == 0 ? cols : s; }
// a single row's stride says nothing
long long row_stride(const zero_layernorm* d, long long s) { return d->rows == 1 ? d->cols : stride_of(s, d->cols); }

zero_status check_ln(const zero_layernorm* d)
{
    if (d == nullptr) return ZERO_ERR_INVALID_ARG;
    if (d->rows < 0 || d->rows > (1LL << 40) || d->cols < 1 || d->cols > ZERO_MAX_NORM_COLS) return ZERO_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->w_dtype)) return ZERO_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return ZERO_ERR_INVALID_ARG;
    const long long s[] = {d->x_stride, d->y_stride, d->dy_stride, d->dx_stride};
    for (long long v : s)
        if (v != 0 && (v < d->cols || v > (1LL << 40))) return ZERO_ERR_INVALID_ARG;
    // an array's extent in bytes is reckoned in 64 bits
    for (long long v : s)
        if (d->rows > (1LL << 58) / stride_of(v, d->cols)) return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

// Whether two [rows, cols] row-strided arrays share a byte; exactly the same
// array does not count (in place).  Columns cut side by side from one wide
// buffer interleave without sharing.
bool shares(const void* p, long long ps, const void* q, long long qs, long long rows, int cols, int es)
{
    if (rows == 0 || (p == q && ps == qs)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const uintptr_t na = static_cast<uintptr_t>((rows - 1) * ps + cols) * es, nb = static_cast<uintptr_t>((rows - 1) * qs + cols) * es;
    if (a + na <= b || b + nb <= a) return false;
    if (ps != qs) return true;
    const uintptr_t row = static_cast<uintptr_t>(ps) * es, w = static_cast<uintptr_t>(cols) * es;
    const uintptr_t off = (b > a ? b - a : a - b) % row;
    return off < w || off + w > row;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t ln_parts_bytes(const zero_layernorm* d)
{
    // at least eight: some kernels deal rows out eight apart
    const long long parts = d->rows < 8 ? 8 : d->rows < zk::kLnMaxParts ? d->rows : zk::kLnMaxParts;
    return round256(static_cast<size_t>(parts) * 2 * zk::ln_pitch(d->cols) * sizeof(float));
}

zk::LnArgs ln_args(const zero_layernorm* d)
{
    zk::LnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = d->rows;
    a.cols = d->cols;
    a.dtype = d->dtype;
    a.w_dtype = d->w_dtype;
    a.eps = d->eps;
    a.x_stride = row_stride(d, d->x_stride);
    return a;
}

// --------------------------------------------------- matrix update batches
const float kQuintic[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kDefaultSteps = 5;

long long extent(const zero_matrices* d, long long ld) { return (d->rows - 1) * ld + d->cols; }

// The products keep x, its Gram matrix G and P = b G + c G G in fp16 times 2^12,
// so their entries (bounded by the largest singular value s of x, by s^2 and
// by |b s^2 + c s^4|) must stay below 16.  x starts with every singular value
// in [0, 1].  A step's polynomial is continuous and keeps 0, so it takes the
// interval of singular values (signs included) to an interval, from its least
// to its largest value at the ends and where it turns: the reachable values
// after each step exactly, with none missed between samples.
bool schedule_fits(int steps, const float* coefs)
{
    double lo = 0.0, hi = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double a = coefs[3 * k], b = coefs[3 * k + 1], c = coefs[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        const double g = (hi > -lo ? hi : -lo) * (hi > -lo ? hi : -lo);   // s^2 fills [0, g]
        const auto p = [&](double q) { return q * (b + c * q); };
        if (!(g <= 15.0) || !(std::fabs(p(g)) <= 15.0)) return false;
        const double top = -b / (2.0 * c);                                // where p turns
        if (top > 0.0 && top < g && !(std::fabs(p(top)) <= 15.0)) return false;
        const auto f = [&](double s) { return s * (a + p(s * s)); };
        double least = std::fmin(f(lo), f(hi)), most = std::fmax(f(lo), f(hi));
        const auto turn = [&](double q) {   // f' = a + 3 b q + 5 c q^2 is 0 at s^2 = q
            if (!(q > 0.0 && q < g)) return;
            for (double s : {-std::sqrt(q), std::sqrt(q)})
                if (s > lo && s < hi) least = std::fmin(least, f(s)), most = std::fmax(most, f(s));
        };
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (c == 0.0) {
            if (b != 0.0) turn(-a / (3.0 * b));
        } else if (d >= 0.0) {
            const double u = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));   // the roots without cancellation
            turn(u / (5.0 * c));
            if (u != 0.0) turn(a / u);
        }
        lo = std::fmin(least, 0.0);
        hi = std::fmax(most, 0.0);
    }
    return std::isfinite(lo) && std::isfinite(hi);
}

zero_status check_matrices(const zero_matrices* d)
{
    if (d == nullptr) return ZERO_ERR_INVALID_ARG;
    if (d->rows < 1 || d->cols < 1 || d->batch < 1) return ZERO_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->out_dtype)) return ZERO_ERR_INVALID_ARG;
    if (d->steps < 0 || d->steps > ZERO_MAX_NS_STEPS || (d->coefs != nullptr && d->steps == 0)) return ZERO_ERR_INVALID_ARG;
    if (!(d->eps >= 1e-30f) || std::isinf(d->eps)) return ZERO_ERR_INVALID_ARG;
    if (d->products != 0 && d->products != 1 && d->products != 3) return ZERO_ERR_INVALID_ARG;
    if (d->rows > ZERO_MAX_MATRIX_DIM || d->cols > ZERO_MAX_MATRIX_DIM || d->batch > 65535) return ZERO_ERR_BOUNDS;
    if (static_cast<long long>(d->rows) * d->cols > ZERO_MAX_MATRIX_ELEMS) return ZERO_ERR_BOUNDS;
    // every kernel numbers its tiles in 32 bits
    const long long tiles = ((d->rows + 127LL) / 128) * ((d->cols + 63LL) / 64);
    const long long side = (((d->rows < d->cols ? d->rows : d->cols) + 127LL) / 128) + 1;
    if ((tiles > side * side ? tiles : side * side) * d->batch > (1LL << 30)) return ZERO_ERR_BOUNDS;
    const long long ld[] = {d->in_ld, d->out_ld}, st[] = {d->in_stride, d->out_stride};
    for (int i = 0; i < 2; ++i) {
        if (ld[i] != 0 && (ld[i] < d->cols || ld[i] > (1LL << 32))) return ZERO_ERR_INVALID_ARG;
        if (st[i] != 0 && (st[i] < extent(d, stride_of(ld[i], d->cols)) || st[i] > (1LL << 40))) return ZERO_ERR_INVALID_ARG;
    }
    if (d->coefs != nullptr && !schedule_fits(d->steps, d->coefs)) return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

// products = 0: one product where the result is rounded to bf16, whose own
// rounding is as large as that product's error; else three.  A short side under
// kFewRows takes three in any case: the operands' roundings then hardly average
// out (2 x 3: 7e-3 off, 64 x 64: 1.8e-3, 768 x 768: 1.2e-3), and the products
// are too short to matter beside the launches.
constexpr int kFewRows = 256;
int products_of(const zero_matrices* d, bool muon)
{
    if ((d->rows < d->cols ? d->rows : d->cols) < kFewRows) return 3;
    if (d->products != 0) return d->products;
    return !muon && d->out_dtype == ZERO_BF16 ? 1 : 3;
}

void set_schedule(zk::NsArgs& a, const zero_matrices* d)
{
    a.rows = d->rows;
    a.cols = d->cols;
    a.batch = d->batch;
    a.steps = d->steps == 0 ? kDefaultSteps : d->steps;
    for (int i = 0; i < a.steps; ++i)
        for (int k = 0; k < 3; ++k) a.coef[i][k] = d->coefs != nullptr ? d->coefs[3 * i + k] : kQuintic[k];
    a.eps = d->eps;
    a.in_dtype = d->dtype;
}

bool overlap(const void* p, const void* q, size_t np, size_t nq)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

}  // namespace

extern "C" {

ZERO_API size_t zero_orthogonalize_workspace_bytes(const zero_matrices* d)
{
    if (check_matrices(d) != ZERO_OK) return 0;
    return zk::ns_workspace_bytes(d->rows, d->cols, d->batch, products_of(d, false), false);
}

ZERO_API size_t zero_muon_workspace_bytes(const zero_matrices* d)
{
    if (check_matrices(d) != ZERO_OK) return 0;
    return zk::ns_workspace_bytes(d->rows, d->cols, d->batch, products_of(d, true), true);
}

ZERO_API zero_status zero_orthogonalize(const zero_matrices* d, const void* g, void* out, void* ws,
                                        zero_dev_scalars* sc, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_matrices(d)) != ZERO_OK) return s;
    if ((s = check_elems(g, d->dtype)) != ZERO_OK || (s = check_elems(out, d->out_dtype)) != ZERO_OK) return s;
    if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
    if (sc != nullptr && (s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    zk::NsArgs a;
    std::memset(&a, 0, sizeof(a));
    set_schedule(a, d);
    a.products = products_of(d, false);
    a.in = g;
    a.in_ld = stride_of(d->in_ld, d->cols);
    a.in_stride = d->in_stride != 0 ? d->in_stride : d->rows * a.in_ld;
    a.out = out;
    a.out_dtype = d->out_dtype;
    a.out_ld = stride_of(d->out_ld, d->cols);
    a.out_stride = d->out_stride != 0 ? d->out_stride : d->rows * a.out_ld;
    const size_t ni = static_cast<size_t>((d->batch - 1) * a.in_stride + extent(d, a.in_ld)) * zk::dtype_bytes(d->dtype);
    const size_t no = static_cast<size_t>((d->batch - 1) * a.out_stride + extent(d, a.out_ld)) * zk::dtype_bytes(d->out_dtype);
    const size_t nw = zk::ns_workspace_bytes(d->rows, d->cols, d->batch, a.products, false);
    if (overlap(g, ws, ni, nw) || overlap(out, ws, no, nw)) return ZERO_ERR_INVALID_ARG;
    // a matrix is read whole before its result is written, but the matrices of a
    // batch are under way side by side: each result may lie on its own input
    // only, or between the inputs' rows
    if (d->batch > 1 && overlap(g, out, ni, no)) {
        if (zk::dtype_bytes(d->dtype) != zk::dtype_bytes(d->out_dtype) || a.in_ld != a.out_ld || a.in_stride != a.out_stride)
            return ZERO_ERR_INVALID_ARG;
        const long long all = (d->batch - 1) * (a.in_stride / a.in_ld) + d->rows;
        if (g != out && (a.in_stride % a.in_ld != 0 || shares(g, a.in_ld, out, a.out_ld, all, d->cols, zk::dtype_bytes(d->dtype))))
            return ZERO_ERR_INVALID_ARG;
    }
    a.ws = ws;
    a.sc = sc;
    return from_cuda(zk::launch_ns(a, as_stream(stream)));
}

ZERO_API zero_status zero_muon_step(const zero_matrices* d, const zero_muon_hparams* hp, int n_d,
                                    const void* const* rank_grads, float* momentum, float* master, void* lp_out,
                                    void* ws, zero_dev_scalars* sc, void* stream)
{
    ZK_CALL_RANGE();
    return zero_muon_step_ex(d, hp, nullptr, n_d, rank_grads, momentum, master, lp_out, ws, sc, stream);
}

ZERO_API zero_status zero_muon_step_ex(const zero_matrices* d, const zero_muon_hparams* hp, const zero_muon_opts* opts,
                                       int n_d, const void* const* rank_grads, float* momentum, float* master,
                                       void* lp_out, void* ws, zero_dev_scalars* sc, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_matrices(d)) != ZERO_OK) return s;
    if (hp == nullptr || rank_grads == nullptr) return ZERO_ERR_INVALID_ARG;
    if (n_d < 1 || n_d > ZERO_MAX_RANKS) return ZERO_ERR_INVALID_ARG;
    // the flat parameter space: whole rows, one index for every array
    if (d->dtype == ZERO_FP32 || d->out_dtype == ZERO_FP32) return ZERO_ERR_INVALID_ARG;
    if ((d->in_ld != 0 && d->in_ld != d->cols) || (d->out_ld != 0 && d->out_ld != d->cols)) return ZERO_ERR_INVALID_ARG;
    const long long elems = static_cast<long long>(d->rows) * d->cols;
    const long long stride = d->in_stride != 0 ? d->in_stride : elems;
    if (d->out_stride != 0 && d->out_stride != stride) return ZERO_ERR_INVALID_ARG;
    if (d->batch > 1 && stride % 8 != 0) return ZERO_ERR_MISALIGNED;
    const float v[] = {hp->lr, hp->momentum, hp->weight_decay, hp->rms_scale, hp->loss_scale};
    for (float x : v)
        if (!std::isfinite(x) || x < 0.0f) return ZERO_ERR_INVALID_ARG;
    if (hp->momentum >= 1.0f) return ZERO_ERR_INVALID_ARG;
    const int loss_scaling = opts != nullptr ? opts->loss_scaling : 0, clipping = opts != nullptr ? opts->clipping : 0;
    for (int f : {hp->nesterov, loss_scaling, clipping})
        if (f != 0 && f != 1) return ZERO_ERR_INVALID_ARG;
    if ((loss_scaling || clipping) && sc == nullptr) return ZERO_ERR_INVALID_ARG;
    for (int r = 0; r < n_d; ++r)
        if ((s = zk::check_dev(rank_grads[r])) != ZERO_OK) return s;
    if ((s = zk::check_dev(momentum)) != ZERO_OK || (s = zk::check_dev(master)) != ZERO_OK) return s;
    if (lp_out != nullptr && (s = zk::check_dev(lp_out)) != ZERO_OK) return s;
    if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
    if (sc != nullptr && (s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    const int products = products_of(d, true);
    const size_t n = static_cast<size_t>((d->batch - 1) * stride + elems);
    const void* arr[] = {momentum, master, lp_out, ws};
    const size_t len[] = {4 * n, 4 * n, lp_out != nullptr ? 2 * n : 0,
                          zk::ns_workspace_bytes(d->rows, d->cols, d->batch, products, true)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (len[i] != 0 && len[j] != 0 && overlap(arr[i], arr[j], len[i], len[j])) return ZERO_ERR_INVALID_ARG;
        for (int r = 0; r < n_d; ++r)
            if (len[i] != 0 && overlap(arr[i], rank_grads[r], len[i], 2 * n)) return ZERO_ERR_INVALID_ARG;
    }
    zk::NsArgs a;
    std::memset(&a, 0, sizeof(a));
    set_schedule(a, d);
    a.products = products;
    a.ranks = rank_grads;
    a.n_d = n_d;
    a.divisor = static_cast<float>(n_d) * (hp->loss_scale > 0.0f ? hp->loss_scale : 1.0f);
    a.mu = hp->momentum;
    a.nesterov = hp->nesterov;
    a.loss_scaling = loss_scaling;
    a.clipping = clipping;
    a.momentum = momentum;
    a.master = master;
    a.lp = lp_out;
    a.lp_dtype = d->out_dtype;
    a.flat_stride = stride;
    const double ratio = static_cast<double>(d->rows) / d->cols;
    const double longest = d->rows > d->cols ? d->rows : d->cols;
    const double scale = hp->rms_scale > 0.0f ? hp->rms_scale * std::sqrt(longest) : std::sqrt(ratio > 1.0 ? ratio : 1.0);
    a.decay = static_cast<float>(1.0 - static_cast<double>(hp->lr) * hp->weight_decay);
    a.step = static_cast<float>(hp->lr * scale);
    a.ws = ws;
    a.sc = sc;
    return from_cuda(zk::launch_ns(a, as_stream(stream)));
}

ZERO_API zero_status zero_debug_matrix_plan(const zero_matrices* d, int muon, int sms, zero_matrix_plan* out)
{
    zero_status s;
    if ((s = check_matrices(d)) != ZERO_OK) return s;
    if (out == nullptr || sms < 2 || (muon != 0 && muon != 1)) return ZERO_ERR_INVALID_ARG;
    zk::ns_plan(d->rows, d->cols, d->batch, products_of(d, muon != 0), sms, out);
    return ZERO_OK;
}

ZERO_API zero_status zero_debug_matmul_timeout(void* scratch, zero_dev_scalars* sc, long long timeout_ns, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = zk::check_dev(scratch, 256)) != ZERO_OK) return s;
    if ((s = zk::check_dev(sc, 256)) != ZERO_OK) return s;
    if (timeout_ns < 1 || timeout_ns > 10000000000LL) return ZERO_ERR_INVALID_ARG;
    return from_cuda(zk::launch_mm_starved(scratch, sc, static_cast<unsigned long long>(timeout_ns), as_stream(stream)));
}

ZERO_API size_t zero_layernorm_workspace_bytes(const zero_layernorm* d)
{
    if (check_ln(d) != ZERO_OK) return 0;
    const size_t means = d->cols >= zk::kLnWide ? round256(static_cast<size_t>(d->rows) * 2 * sizeof(float)) : 0;
    return 256 + ln_parts_bytes(d) + means;
}

ZERO_API zero_status zero_layernorm_forward(const zero_layernorm* d, const void* x, const void* gain, const void* bias,
                                            void* y, float* mean, float* rstd, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_ln(d)) != ZERO_OK) return s;
    if (d->rows == 0) return ZERO_OK;
    if ((s = check_elems(x, d->dtype)) != ZERO_OK || (s = check_elems(y, d->dtype)) != ZERO_OK) return s;
    if (gain != nullptr && (s = check_elems(gain, d->w_dtype)) != ZERO_OK) return s;
    if (bias != nullptr && (s = check_elems(bias, d->w_dtype)) != ZERO_OK) return s;
    if (!zk::aligned(mean, 4) || !zk::aligned(rstd, 4)) return ZERO_ERR_MISALIGNED;
    zk::LnArgs a = ln_args(d);
    a.out_stride = row_stride(d, d->y_stride);
    if (shares(x, a.x_stride, y, a.out_stride, d->rows, d->cols, zk::dtype_bytes(d->dtype))) return ZERO_ERR_INVALID_ARG;
    a.x = x;
    a.gain = gain;
    a.bias = bias;
    a.out = y;
    a.mean_out = mean;
    a.rstd_out = rstd;
    return from_cuda(zk::launch_ln_forward(a, as_stream(stream)));
}

ZERO_API zero_status zero_layernorm_backward(const zero_layernorm* d, const void* dy, const void* x, const void* gain,
                                             const float* mean, const float* rstd, void* dx, void* dgain, void* dbias,
                                             void* ws, void* stream)
{
    ZK_CALL_RANGE();
    zero_status s;
    if ((s = check_ln(d)) != ZERO_OK) return s;
    if (d->rows > 0) {   // without rows there is nothing to point at
        const void* acts[] = {dy, x, dx};
        for (const void* p : acts)
            if ((s = check_elems(p, d->dtype)) != ZERO_OK) return s;
        if ((s = check_elems(mean, ZERO_FP32)) != ZERO_OK || (s = check_elems(rstd, ZERO_FP32)) != ZERO_OK) return s;
    }
    if (gain != nullptr && (s = check_elems(gain, d->w_dtype)) != ZERO_OK) return s;
    if (dgain != nullptr && (s = check_elems(dgain, d->w_dtype)) != ZERO_OK) return s;
    if (dbias != nullptr && (s = check_elems(dbias, d->w_dtype)) != ZERO_OK) return s;
    if ((s = zk::check_dev(ws, 256)) != ZERO_OK) return s;
    zk::LnArgs a = ln_args(d);
    a.dy_stride = row_stride(d, d->dy_stride);
    a.out_stride = row_stride(d, d->dx_stride);
    const int es = zk::dtype_bytes(d->dtype);
    if (shares(x, a.x_stride, dx, a.out_stride, d->rows, d->cols, es) ||
        shares(dy, a.dy_stride, dx, a.out_stride, d->rows, d->cols, es))
        return ZERO_ERR_INVALID_ARG;
    if (dgain != nullptr && (dgain == dbias || shares(dgain, d->cols, dbias, d->cols, 1, d->cols, zk::dtype_bytes(d->w_dtype))))
        return ZERO_ERR_INVALID_ARG;
    a.x = x;
    a.dy = dy;
    a.gain = gain;
    a.mean = mean;
    a.rstd = rstd;
    a.out = dx;
    a.dgain = dgain;
    a.dbias = dbias;
    a.pitch = zk::ln_pitch(d->cols);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    a.rowsums = reinterpret_cast<float*>(static_cast<char*>(ws) + 256 + ln_parts_bytes(d));
    return from_cuda(zk::launch_ln_backward(a, as_stream(stream)));
}

}  // extern "C"
