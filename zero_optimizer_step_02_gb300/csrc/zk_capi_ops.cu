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

zero_status check_ln(const zero_layernorm* d)
{
    if (d == nullptr) return ZERO_ERR_INVALID_ARG;
    if (d->rows < 0 || d->rows > (1LL << 40) || d->cols < 1 || d->cols > ZERO_MAX_NORM_COLS) return ZERO_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->w_dtype)) return ZERO_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return ZERO_ERR_INVALID_ARG;
    const long long s[] = {d->x_stride, d->y_stride, d->dy_stride, d->dx_stride};
    for (long long v : s)
        if (v != 0 && (v < d->cols || v > (1LL << 40))) return ZERO_ERR_INVALID_ARG;
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
    const long long parts = d->rows < zk::kLnMaxParts ? d->rows : zk::kLnMaxParts;
    return round256(static_cast<size_t>(parts) * 2 * d->cols * sizeof(float));
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
    a.x_stride = stride_of(d->x_stride, d->cols);
    return a;
}

}  // namespace

extern "C" {

ZERO_API size_t zero_layernorm_workspace_bytes(const zero_layernorm* d)
{
    if (check_ln(d) != ZERO_OK) return 0;
    return 256 + ln_parts_bytes(d) + round256(static_cast<size_t>(d->rows) * 2 * sizeof(float));
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
    a.out_stride = stride_of(d->y_stride, d->cols);
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
    a.dy_stride = stride_of(d->dy_stride, d->cols);
    a.out_stride = stride_of(d->dx_stride, d->cols);
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
    a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    a.rowsums = reinterpret_cast<float*>(static_cast<char*>(ws) + 256 + ln_parts_bytes(d));
    return from_cuda(zk::launch_ln_backward(a, as_stream(stream)));
}

}  // extern "C"
