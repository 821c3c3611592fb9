// zk_tensors.cu -- the AdamW step over many tensors at once.
//
// The tensors' addresses travel in the launch's parameters (up to kTableMax of
// them; a longer list takes several launches), so a call neither copies nor
// allocates, and a captured graph holds what it needs.  All tensors together
// are cut into tiles of kTensorTile elements; every CTA takes an equal,
// contiguous range of them.  A warp works on 256 elements at a time, the block
// of an 8-bit state, so that nothing but its largest values crosses lanes:
//   p <- p (1 - lr wd)
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g g,  r = sqrt(v)
//   p <- p - (lr s / (1 - b1^t)) m / (r + eps s),  s = sqrt(1 - b2^t)
// each operation one IEEE rounding in this order, as in the step's Adam.
//
// What a call cannot do without, at a copy's rate, and what it takes (us; bf16
// gradients and 16-bit weights):
//   105M parameters of 12 layers, 32-bit states   435.7   461; clipped 521: the
//       norm pass reads the gradients once more (31 of it at a copy's rate, 60 in all,
//       as it adds squares up with their rounding errors, in packed fp32)
//   436M parameters, 8-bit states                1032.9   1230: some 70 instructions an
//       element pair leave 1 in 6 of the copy's rate unused: IEEE's roots, and the
//       codes' thresholds, roundings and packing
//   300 odd fp32 tensors                          133.5   152
//   10 tensors of 1.4M parameters                   2.2   7.3: one launch
#include <cuda_fp8.h>

#include "zk_common.cuh"
#include "zk_launch.h"
#include "zk_ops.h"

namespace zk {

namespace {

constexpr int kThreadsT = 256;
static_assert(kTensorTile == kThreadsT / 32 * kStateBlock, "a warp's share of a tile is one state block");

constexpr uint32_t kTurnStep = 0xC13FA9A9u, kTurnElem = 0x91E10DA5u;   // in 2^-32

struct Consts {
    float b1, b2, omb1, omb2, bc1, sbc2, eps, coef, divisor;
    float factor;    // of the gradient, without a division: 0 where that takes one
    uint32_t turn;   // this step's part of the 8-bit states' thresholds
    float lift;      // the 8-bit states' divisors and dividends times this: 1, or what makes a subnormal eps a normal number
};

// The step's constants (one thread).
__device__ __forceinline__ void step_consts(const AdamwArgs& a, Consts* out)
{
    StepConsts c = {};
    set_divisor(c, 1, a.hp.loss_scaling ? a.sc->loss_scale : 1.0f);
    Consts k;
    const double b1t = __dmul_rn(a.sc->beta1_pow, static_cast<double>(a.hp.beta1));
    const double b2t = __dmul_rn(a.sc->beta2_pow, static_cast<double>(a.hp.beta2));
    k.bc1 = __double2float_rn(__dsub_rn(1.0, b1t));
    k.sbc2 = __fsqrt_rn(__double2float_rn(__dsub_rn(1.0, b2t)));
    k.b1 = a.hp.beta1;
    k.b2 = a.hp.beta2;
    k.omb1 = __fsub_rn(1.0f, a.hp.beta1);
    k.omb2 = __fsub_rn(1.0f, a.hp.beta2);
    k.eps = __fmul_rn(a.hp.eps, k.sbc2);
    k.coef = a.clip ? a.sc->clip_coef : 1.0f;   // of the norm pass
    k.divisor = c.divisor;
    // g / 1 * coef, or g / 2^k, in one product, which rounds as the two do
    k.factor = c.divisor == 1.0f ? k.coef : c.div_pow2 && k.coef == 1.0f ? c.inv_divisor : 0.0f;
    // the near reciprocal takes a subnormal for 0: 0 / eps would be NaN
    k.lift = k.eps > 0.0f && k.eps < 1.17549435e-38f ? 4294967296.0f : 1.0f;
    k.turn = static_cast<uint32_t>(a.sc->t) * static_cast<uint32_t>(a.sc->t) * kTurnStep;
    *out = k;
}

// ------------------------------------------------------------- 8-bit states
// Codes are e4m3 values; the block's largest magnitude is 448, its scale
// largest * (1 / 448) in fp32.  r = sqrt(v) is held in place of v: its range is half
// as wide in the exponent, and it is what divides.  A positive r keeps at least
// the smallest code: a zero under a momentum that survived its own rounding
// would divide by eps alone.  Blocks whose largest magnitude is under 2^-100
// stand for zeros; one that is not finite makes the scale NaN, and so every
// value of the block.
//
// Rounding to nearest would hold a moment in place: codes lie up to 1/8 apart,
// and a decay by b1 >= 0.95, or any by b2, moves it by less than half of that.
// So a value between two codes takes the upper one when its place between them
// plus a threshold reaches 1.  The threshold of an element moves over its
// neighbours by 0.5698 and with the step by 0.7549 t^2 (mod 1; the two are the
// plane's most even lattice): over the steps the roundings' mean is the value
// (0.1 % over 512 steps of a moment that stands still; with 0.7549 t, whose
// thresholds keep step with the decay, 2 %).  No random state, and the same
// inputs give the same codes.
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Min = 0.001953125f;     // 2^-9
constexpr float kE4m3Normal = 0.015625f;     // 2^-6
constexpr float kBlockSmall = 7.8886090522101181e-31f;   // 2^-100

// the values of two codes, times the scale (one rounding)
__device__ __forceinline__ f32x2 decode2(uint32_t w, f32x2 scale)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return mul2(pack2(f.x, f.y), scale);
}

__device__ __forceinline__ uint32_t encode2(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// q, z >= 0 down to a code or up to the next: the 20 mantissa bits that e4m3 has
// not are added to the threshold, and cut.  Under 2^-6 codes lie as far apart as
// from there to 2^-5, so there it is done.
__device__ __forceinline__ void turn_to_codes(float& q, float& z, uint32_t turn)
{
    const f32x2 under = pack2(q < kE4m3Normal ? kE4m3Normal : 0.0f, z < kE4m3Normal ? kE4m3Normal : 0.0f);
    float a, b;
    unpack2(add2(pack2(q, z), under), a, b);
    a = __uint_as_float((__float_as_uint(a) + turn) & 0xFFF00000u);
    b = __uint_as_float((__float_as_uint(b) + turn) & 0xFFF00000u);
    unpack2(sub2(pack2(a, b), under), q, z);
}

__device__ __forceinline__ float reciprocal_near(float x)   // 1 ulp
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The scales of a block's two moments and the factors of their codes, from the
// largest magnitudes: both reciprocals in one division, half of the warp each.
// `scale` is the momentum's in lane 0, the root's in lane 16.
struct Scales {
    float scale, mi, ri;
};
__device__ __forceinline__ Scales block_scales(float mtop, float rtop, int lane)
{
    // as integers, magnitudes keep their order, with a NaN above them all
    const uint32_t mb = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mtop)), rb = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(rtop));
    const uint32_t bits = lane < 16 ? mb : rb;
    const float top = __uint_as_float(bits);
    float scale = __fmul_rn(top, 1.0f / kE4m3Max), inv = __fmul_rn(kE4m3Max, __fdiv_rn(1.0f, top));
    if (top < kBlockSmall) scale = inv = 0.0f;
    if (bits >= 0x7F800000u) scale = __uint_as_float(0x7FC00000u), inv = 0.0f;
    return Scales{scale, __shfl_sync(0xFFFFFFFFu, inv, 0), __shfl_sync(0xFFFFFFFFu, inv, 16)};
}

// ------------------------------------------------------------ one warp's 256
// WIDE: lane l holds elements 8l .. 8l+7 in 16-byte words (every base 16-byte
// aligned, 256 elements there); else element e of lane l is 32 e + l, which
// keeps a warp's accesses together at any alignment.
template <bool WIDE>
__device__ __forceinline__ int elem_of(int e, int lane) { return WIDE ? 8 * lane + e : 32 * e + lane; }

template <bool WIDE>
__device__ __forceinline__ void load_f32(const float* p, int lane, int n, float (&x)[8])
{
    if constexpr (WIDE) {
        const float4 a = reinterpret_cast<const float4*>(p)[2 * lane], b = reinterpret_cast<const float4*>(p)[2 * lane + 1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 32 * e + lane < n ? p[32 * e + lane] : 0.0f;
    }
}

template <bool WIDE>
__device__ __forceinline__ void store_f32(float* p, int lane, int n, const float (&x)[8])
{
    if constexpr (WIDE) {
        reinterpret_cast<float4*>(p)[2 * lane] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[2 * lane + 1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e + lane < n) p[32 * e + lane] = x[e];
    }
}

template <int DT>
__device__ __forceinline__ void widen8(uint4 w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = Lp<DT>::lo(u[k]);
        x[2 * k + 1] = Lp<DT>::hi(u[k]);
    }
}

template <bool WIDE, int DT>
__device__ __forceinline__ void load_lp(const void* p, int lane, int n, float (&x)[8])
{
    if constexpr (WIDE) {
        widen8<DT>(reinterpret_cast<const uint4*>(p)[lane], x);
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 32 * e + lane < n ? Lp<DT>::widen(q[32 * e + lane]) : 0.0f;
    }
}

template <bool WIDE>
__device__ __forceinline__ void load_grad(const void* g, int dt, int lane, int n, float (&x)[8])
{
    if (dt == ZERO_BF16) load_lp<WIDE, ZERO_BF16>(g, lane, n, x);
    else if (dt == ZERO_FP16) load_lp<WIDE, ZERO_FP16>(g, lane, n, x);
    else load_f32<WIDE>(static_cast<const float*>(g), lane, n, x);
}

template <bool WIDE, int DT>
__device__ __forceinline__ void store_lp(void* p, int lane, int n, const float (&x)[8])
{
    if constexpr (WIDE) {
        reinterpret_cast<uint4*>(p)[lane] = make_uint4(Lp<DT>::narrow2(x[0], x[1]), Lp<DT>::narrow2(x[2], x[3]),
                                                       Lp<DT>::narrow2(x[4], x[5]), Lp<DT>::narrow2(x[6], x[7]));
    } else {
        uint16_t* q = static_cast<uint16_t*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e + lane < n) q[32 * e + lane] = Lp<DT>::narrow(x[e]);
    }
}

// eight codes of a lane, two to a 16-bit word
template <bool WIDE>
__device__ __forceinline__ void load_codes(const unsigned char* p, int lane, int n, uint32_t (&c)[4])
{
    if constexpr (WIDE) {
        const uint2 w = reinterpret_cast<const uint2*>(p)[lane];
        c[0] = w.x & 0xFFFFu;
        c[1] = w.x >> 16;
        c[2] = w.y & 0xFFFFu;
        c[3] = w.y >> 16;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = 64 * k + lane;
            c[k] = (i < n ? p[i] : 0u) | (i + 32 < n ? static_cast<uint32_t>(p[i + 32]) << 8 : 0u);
        }
    }
}

template <bool WIDE>
__device__ __forceinline__ void store_codes(unsigned char* p, int lane, int n, const uint32_t (&c)[4])
{
    if constexpr (WIDE) {
        reinterpret_cast<uint2*>(p)[lane] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = 64 * k + lane;
            if (i < n) p[i] = static_cast<unsigned char>(c[k]);
            if (i + 32 < n) p[i + 32] = static_cast<unsigned char>(c[k] >> 8);
        }
    }
}

// this tensor's own constants
struct Rates {
    float step, decay;
};

__device__ __forceinline__ Rates rates_of(const AdamwArgs& a, const Consts& c, const TensorEntry& e)
{
    const float lr = __fmul_rn(a.hp.lr, e.lr_scale), wd = __fmul_rn(a.hp.weight_decay, e.wd_scale);
    return Rates{__fdiv_rn(__fmul_rn(lr, c.sbc2), c.bc1), __fsub_rn(1.0f, __fmul_rn(lr, wd))};
}

// What a lane holds of a block: eight elements' gradients, weights and moments (in
// 8 bits their codes and the block's scales).
template <bool EIGHT>
struct Held {
    float g[8], p[8], m[8], v[8];
};
template <>
struct Held<true> {
    float g[8], p[8];
    uint32_t mc[4], rc[4];
    float ms, rs;
};

// n <= 256 elements from element `at` (a multiple of 256) of a tensor
template <bool WIDE, bool EIGHT>
__device__ __forceinline__ void load(Held<EIGHT>& h, const TensorEntry& t, long long at, int n, int lane)
{
    const int gb = t.grad_dtype == ZERO_FP32 ? 4 : 2;
    load_grad<WIDE>(static_cast<const char*>(t.grad) + at * gb, t.grad_dtype, lane, n, h.g);
    load_f32<WIDE>(t.master + at, lane, n, h.p);
    if constexpr (EIGHT) {
        load_codes<WIDE>(static_cast<const unsigned char*>(t.m) + at, lane, n, h.mc);
        load_codes<WIDE>(static_cast<const unsigned char*>(t.v) + at, lane, n, h.rc);
        h.ms = t.m_scale[at / kStateBlock];
        h.rs = t.v_scale[at / kStateBlock];
    } else {
        load_f32<WIDE>(static_cast<const float*>(t.m) + at, lane, n, h.m);
        load_f32<WIDE>(static_cast<const float*>(t.v) + at, lane, n, h.v);
    }
}

// the gradients unscaled and clipped
__device__ __forceinline__ void unscale(float (&g)[8], const Consts& c)
{
    if (c.factor != 0.0f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], c.factor);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(__fdiv_rn(g[e], c.divisor), c.coef);
    }
}

template <bool WIDE>
__device__ __forceinline__ void store_weights(const TensorEntry& t, long long at, int n, int lane, const float (&p)[8])
{
    store_f32<WIDE>(t.master + at, lane, n, p);
    if (t.lp != nullptr) {
        if (t.lp_dtype == ZERO_BF16) store_lp<WIDE, ZERO_BF16>(static_cast<uint16_t*>(t.lp) + at, lane, n, p);
        else store_lp<WIDE, ZERO_FP16>(static_cast<uint16_t*>(t.lp) + at, lane, n, p);
    }
}

template <bool WIDE>
__device__ __forceinline__ void update(Held<false>& h, const TensorEntry& t, long long at, int n, const Consts& c, const Rates& r, int lane)
{
    unscale(h.g, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = h.g[e];
        h.p[e] = __fmul_rn(h.p[e], r.decay);   // by 1 without decay
        h.m[e] = __fadd_rn(__fmul_rn(c.b1, h.m[e]), __fmul_rn(c.omb1, x));
        h.v[e] = __fadd_rn(__fmul_rn(c.b2, h.v[e]), __fmul_rn(c.omb2, __fmul_rn(x, x)));
        h.p[e] = __fsub_rn(h.p[e], __fmul_rn(r.step, __fdiv_rn(h.m[e], __fadd_rn(__fsqrt_rn(h.v[e]), c.eps))));
    }
    store_weights<WIDE>(t, at, n, lane, h.p);
    store_f32<WIDE>(static_cast<float*>(t.m) + at, lane, n, h.m);
    store_f32<WIDE>(static_cast<float*>(t.v) + at, lane, n, h.v);
}

// With 8-bit states the arithmetic is what a call waits for, not memory: products
// on pairs (each rounded, and never added as pairs, which would fuse them), and for
// the weights, which no code depends on, fused operations and a near reciprocal.
// The moments take the operations above in their order, so that a code is what
// they say and not a neighbour that a rounding leads to.
template <bool WIDE>
__device__ __forceinline__ void update(Held<true>& h, const TensorEntry& t, long long at, int n, const Consts& c, const Rates& r, int lane)
{
    unscale(h.g, c);
    const f32x2 ms = pack2(h.ms, h.ms), rs = pack2(h.rs, h.rs), b1 = pack2(c.b1, c.b1), b2 = pack2(c.b2, c.b2);
    const f32x2 omb1 = pack2(c.omb1, c.omb1), omb2 = pack2(c.omb2, c.omb2);
    const float eps1 = __fmul_rn(c.eps, c.lift), step1 = -__fmul_rn(r.step, c.lift);
    const f32x2 eps = pack2(eps1, eps1), step = pack2(step1, step1), lift = pack2(c.lift, c.lift), decay = pack2(r.decay, r.decay);
    float m[8], root[8], mtop = 0.0f, rtop = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x2 x = pack2(h.g[2 * k], h.g[2 * k + 1]);
        float a0, a1, b0, b1_;
        unpack2(mul2(b1, decode2(h.mc[k], ms)), a0, a1);
        unpack2(mul2(omb1, x), b0, b1_);
        m[2 * k] = a0 = __fadd_rn(a0, b0), m[2 * k + 1] = a1 = __fadd_rn(a1, b1_);
        mtop = max_or_nan(mtop, max_or_nan(fabsf(a0), fabsf(a1)));
        const f32x2 momentum = pack2(a0, a1), was = decode2(h.rc[k], rs);
        unpack2(mul2(b2, mul2(was, was)), a0, a1);
        unpack2(mul2(omb2, mul2(x, x)), b0, b1_);
        root[2 * k] = a0 = __fsqrt_rn(__fadd_rn(a0, b0)), root[2 * k + 1] = a1 = __fsqrt_rn(__fadd_rn(a1, b1_));
        rtop = max_or_nan(rtop, max_or_nan(a0, a1));
        unpack2(fma2(pack2(a0, a1), lift, eps), a0, a1);
        const f32x2 inv = pack2(reciprocal_near(a0), reciprocal_near(a1));
        unpack2(fma2(mul2(momentum, step), inv, mul2(pack2(h.p[2 * k], h.p[2 * k + 1]), decay)), h.p[2 * k], h.p[2 * k + 1]);
    }
    store_weights<WIDE>(t, at, n, lane, h.p);
    const Scales s = block_scales(mtop, rtop, lane);
    const uint32_t turn0 = c.turn + (static_cast<uint32_t>(at) + static_cast<uint32_t>(elem_of<WIDE>(0, lane))) * kTurnElem;
    uint32_t mc[4], rc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float q[2], z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t turn = (turn0 + static_cast<uint32_t>(elem_of<WIDE>(2 * k + e, 0)) * kTurnElem) >> 12;
            const float x = m[2 * k + e], y = root[2 * k + e];
            q[e] = __fmul_rn(fabsf(x), s.mi);
            z[e] = __fmul_rn(y, s.ri);
            turn_to_codes(q[e], z[e], turn);
            q[e] = copysignf(q[e], x);
            z[e] = y > 0.0f ? fmaxf(z[e], kE4m3Min) : 0.0f;
        }
        mc[k] = encode2(q[0], q[1]);
        rc[k] = encode2(z[0], z[1]);
    }
    if (!(s.mi > 0.0f)) mc[0] = mc[1] = mc[2] = mc[3] = 0u;
    if (!(s.ri > 0.0f)) rc[0] = rc[1] = rc[2] = rc[3] = 0u;
    store_codes<WIDE>(static_cast<unsigned char*>(t.m) + at, lane, n, mc);
    store_codes<WIDE>(static_cast<unsigned char*>(t.v) + at, lane, n, rc);
    if (lane == 0) t.m_scale[at / kStateBlock] = s.scale;
    if (lane == 16) t.v_scale[at / kStateBlock] = s.scale;
}

template <bool WIDE, bool EIGHT>
__device__ __forceinline__ void step(const TensorEntry& t, long long at, int n, const Consts& c, const Rates& r, int lane)
{
    Held<EIGHT> h;
    load<WIDE, EIGHT>(h, t, at, n, lane);
    update<WIDE>(h, t, at, n, c, r, lane);
}

// Whole tiles with 8-bit states come through a ring in shared memory, by bulk
// copies: a tile has fewer bytes than one with 32-bit states, and its arithmetic
// takes as long as the memory, so that what 24 warps an SM ask for at a time does
// not cover the latency (436M parameters 1617 us by direct loads, 1230 through the
// ring; with 32-bit states direct loads reach 95 to 97 % of a copy's rate).
constexpr int kRing = 3;
constexpr int kRingStage = kTensorTile * (4 + 4 + 1 + 1);   // fp32 gradients, weights, codes
struct Ring {
    uint64_t full[kRing];
    uint32_t asked[kRing];   // how often
    int abort;
    int stage;               // the next to be read
    uint32_t phase;
};

__device__ __forceinline__ void ask(const TensorEntry& t, long long at, unsigned char* ring, Ring& sh, int stage)
{
    const uint32_t gb = t.grad_dtype == ZERO_FP32 ? 4 : 2;
    unsigned char* to = ring + stage * kRingStage;
    uint64_t* bar = &sh.full[stage];
    ++sh.asked[stage];
    mbar_arrive_expect_tx(bar, kTensorTile * (gb + 6));
    bulk_load(to, static_cast<const char*>(t.grad) + at * gb, kTensorTile * gb, bar);
    bulk_load(to + kTensorTile * 4, t.master + at, kTensorTile * 4, bar);
    bulk_load(to + kTensorTile * 8, static_cast<const unsigned char*>(t.m) + at, kTensorTile, bar);
    bulk_load(to + kTensorTile * 9, static_cast<const unsigned char*>(t.v) + at, kTensorTile, bar);
}

// `tiles` whole tiles from element `first` (a multiple of the tile) on, by the CTA.
// False: a copy did not come.
__device__ __forceinline__ bool step_ring(const TensorEntry& t, long long first, int tiles, unsigned char* ring, Ring& sh, const Consts& c, const Rates& r, int warp, int lane)
{
    int stage = sh.stage;
    uint32_t phase = sh.phase;
    if (threadIdx.x == 0) {
        fence_proxy_async_smem();   // after the last tensor's reads
        for (int i = 0; i < kRing && i < tiles; ++i) ask(t, first + static_cast<long long>(i) * kTensorTile, ring, sh, (stage + i) % kRing);
    }
    long long at = first + warp * kStateBlock;
    float ms = t.m_scale[at / kStateBlock], rs = t.v_scale[at / kStateBlock];
    for (int i = 0; i < tiles; ++i, at += kTensorTile) {
        Held<true> h;
        h.ms = ms, h.rs = rs;
        if (i + 1 < tiles) {
            ms = t.m_scale[at / kStateBlock + kTensorTile / kStateBlock];
            rs = t.v_scale[at / kStateBlock + kTensorTile / kStateBlock];
        }
        if (!mbar_wait_bounded(&sh.full[stage], phase, &sh.abort, kDefaultTimeoutNs)) atomicExch(&sh.abort, 1);
        const unsigned char* from = ring + stage * kRingStage;
        const int block = warp * kStateBlock;
        load_grad<true>(from + block * (t.grad_dtype == ZERO_FP32 ? 4 : 2), t.grad_dtype, lane, kStateBlock, h.g);
        load_f32<true>(reinterpret_cast<const float*>(from + kTensorTile * 4) + block, lane, kStateBlock, h.p);
        load_codes<true>(from + kTensorTile * 8 + block, lane, kStateBlock, h.mc);
        load_codes<true>(from + kTensorTile * 9 + block, lane, kStateBlock, h.rc);
        __syncthreads();   // the stage is read
        if (*reinterpret_cast<volatile int*>(&sh.abort)) return false;
        if (threadIdx.x == 0 && i + kRing < tiles) {
            fence_proxy_async_smem();
            ask(t, first + static_cast<long long>(i + kRing) * kTensorTile, ring, sh, stage);
        }
        if (++stage == kRing) stage = 0, phase ^= 1u;
        update<true>(h, t, at, kStateBlock, c, r, lane);
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.stage = stage, sh.phase = phase;
    __syncthreads();
    return true;
}

// the tensor that holds a tile: the last one whose first tile is not past it
// (empty tensors share their first tile with the next one)
template <int CAP>
__device__ __forceinline__ int tensor_of(const TensorTable<CAP>& t, int tile)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.e[mid].tile0 <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsT, 3)
k_adamw(const __grid_constant__ TensorTable<CAP> t, const __grid_constant__ AdamwArgs a)
{
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ Consts shc;
    __shared__ Ring shr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&shr.full[i], 1), shr.asked[i] = 0u;
        shr.abort = shr.stage = 0;
        shr.phase = 0u;
        fence_barrier_init();
    }
    // with the flag set by the norm pass the step is skipped
    const bool skip = a.hp.loss_scaling && *reinterpret_cast<volatile int*>(&a.sc->nonfinite) != 0;
    if (threadIdx.x == 0) step_consts(a, &shc);
    __syncthreads();
    if (!skip) {
        const Consts c = shc;
        const int first = static_cast<int>(static_cast<long long>(t.tiles) * blockIdx.x / gridDim.x);
        const int last = static_cast<int>(static_cast<long long>(t.tiles) * (blockIdx.x + 1) / gridDim.x);
        int i = first < last ? tensor_of(t, first) : 0;
        Rates r = rates_of(a, c, t.e[i]);
        for (int tile = first; tile < last; ++tile) {
            bool moved = false;
            while (i + 1 < t.n && t.e[i + 1].tile0 <= tile) ++i, moved = true;
            const TensorEntry& e = t.e[i];
            if (moved) r = rates_of(a, c, e);
            if (e.wide && e.eight) {
                // the whole tiles of this tensor in the CTA's range
                const int whole = static_cast<int>(e.n / kTensorTile) - (tile - e.tile0), run = whole < last - tile ? whole : last - tile;
                if (run > 0) {
                    if (!step_ring(e, static_cast<long long>(tile - e.tile0) * kTensorTile, run, ring, shr, c, r, warp, lane)) break;
                    tile += run - 1;
                    continue;
                }
            }
            const long long at = static_cast<long long>(tile - e.tile0) * kTensorTile + warp * kStateBlock;
            const long long left = e.n - at;
            if (left <= 0) continue;
            if (e.wide && !e.eight && left >= kStateBlock) {
                step<true, false>(e, at, kStateBlock, c, r, lane);
            } else {
                const int n = left < kStateBlock ? static_cast<int>(left) : kStateBlock;
                if (e.eight) step<false, true>(e, at, n, c, r, lane);
                else step<false, false>(e, at, n, c, r, lane);
            }
        }
    }
    if (threadIdx.x == 0 && *reinterpret_cast<volatile int*>(&shr.abort)) {
        atomicOr(&a.sc->status, ZERO_DEV_TIMEOUT);
        // copies still under way have to land before the CTA's memory goes
        for (int i = 0; i < kRing; ++i)
            if (shr.asked[i] != 0u) mbar_wait_bounded(&shr.full[i], (shr.asked[i] - 1u) & 1u, nullptr, kDefaultTimeoutNs);
    }
    if (a.commit && threadIdx.x == 0) {
        // the last CTA to take a ticket commits the step scalars: every CTA
        // read them before taking its own (no CTA waits for another)
        __threadfence();
        const unsigned done = atomicAdd(&a.sc->ctas_done, 1u);
        if (done == gridDim.x - 1) {
            __threadfence();
            commit_scalars(a.hp, a.sc);
            a.sc->ctas_done = 0u;
        }
    }
}

// Squared norm of every unscaled gradient: one fp64 partial sum a CTA (see
// sq_accumulate), which the last CTA of the last launch adds up in order for the
// clip coefficient; under loss scaling the non-finite flag.  Squares and a lane's
// sums are fp32, which a finite gradient from 1.8e19 on leaves: a warp whose lanes
// then hold an infinity or a NaN (the rounding errors' sum keeps one to the end)
// reads its share once more and adds it up in fp64, whose range no list of fp32
// values leaves.
constexpr int kNormAhead = 4;   // tiles under way

struct Squares {
    f32x2 hi, lo;
    float inv, divisor;   // inv 0: the divisor is not a power of two
    bool bad;

    __device__ __forceinline__ float unscaled(float x) const { return inv != 0.0f ? __fmul_rn(x, inv) : __fdiv_rn(x, divisor); }
    __device__ __forceinline__ void take(float x, float y)
    {
        x = unscaled(x), y = unscaled(y);
        bad |= !is_finite_f32(x) | !is_finite_f32(y);
        sq_accumulate2(x, y, hi, lo);
    }
    // one warp's blocks of kNormAhead whole tiles; p: the lane's first words
    template <int DT>
    __device__ __forceinline__ void tiles(const uint4* p)
    {
        constexpr int kWords = DT == ZERO_FP32 ? 2 : 1, kTileWords = kTensorTile * (DT == ZERO_FP32 ? 4 : 2) / 16;
#pragma unroll
        for (int k0 = 0; k0 < kNormAhead; k0 += 4 / kWords) {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = p[(k0 + k / kWords) * kTileWords + k % kWords];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                if constexpr (DT == ZERO_FP32) {
                    take(__uint_as_float(u[0]), __uint_as_float(u[1]));
                    take(__uint_as_float(u[2]), __uint_as_float(u[3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) take(Lp<DT>::lo(u[e]), Lp<DT>::hi(u[e]));
                }
            }
        }
    }
};

// A lane's part of the squared norm of tiles [first, last), in fp64.
template <int CAP>
__device__ __noinline__ double squares_in_fp64(const TensorTable<CAP>& t, int first, int last, const Squares& sq)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double part = 0.0;
    int i = tensor_of(t, first);
    for (int tile = first; tile < last; ++tile) {
        while (i + 1 < t.n && t.e[i + 1].tile0 <= tile) ++i;
        const TensorEntry& e = t.e[i];
        const long long at = static_cast<long long>(tile - e.tile0) * kTensorTile + warp * kStateBlock, left = e.n - at;
        if (left <= 0) continue;
        float g[8];
        load_grad<false>(static_cast<const char*>(e.grad) + at * (e.grad_dtype == ZERO_FP32 ? 4 : 2), e.grad_dtype, lane,
                         left < kStateBlock ? static_cast<int>(left) : kStateBlock, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double x = sq.unscaled(g[k]);
            part = __dadd_rn(part, __dmul_rn(x, x));
        }
    }
    return part;
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsT, 6)
k_tensors_norm(const __grid_constant__ TensorTable<CAP> t, const __grid_constant__ AdamwArgs a, double* partials)
{
    __shared__ double red[kThreadsT / 32];
    __shared__ int last_one;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    StepConsts c = {};
    set_divisor(c, 1, a.hp.loss_scaling ? a.sc->loss_scale : 1.0f);
    const int first = static_cast<int>(static_cast<long long>(t.tiles) * blockIdx.x / gridDim.x);
    const int last = static_cast<int>(static_cast<long long>(t.tiles) * (blockIdx.x + 1) / gridDim.x);
    Squares sq = {0ull, 0ull, c.inv_divisor, c.divisor, false};
    int i = first < last ? tensor_of(t, first) : 0;
    for (int tile = first; tile < last;) {
        while (i + 1 < t.n && t.e[i + 1].tile0 <= tile) ++i;
        const TensorEntry& e = t.e[i];
        const int es = e.grad_dtype == ZERO_FP32 ? 4 : 2;
        const long long tile_of = tile - e.tile0, at = tile_of * kTensorTile + warp * kStateBlock;
        const char* src = static_cast<const char*>(e.grad) + at * es;
        const long long whole = e.n / kTensorTile - tile_of;   // tiles with nothing missing
        if (e.wide && whole >= kNormAhead && last - tile >= kNormAhead) {
            if (e.grad_dtype == ZERO_BF16) sq.tiles<ZERO_BF16>(reinterpret_cast<const uint4*>(src) + lane);
            else if (e.grad_dtype == ZERO_FP16) sq.tiles<ZERO_FP16>(reinterpret_cast<const uint4*>(src) + lane);
            else sq.tiles<ZERO_FP32>(reinterpret_cast<const uint4*>(src) + 2 * lane);
            tile += kNormAhead;
            continue;
        }
        ++tile;
        const long long left = e.n - at;
        if (left <= 0) continue;
        float g[8];
        load_grad<false>(src, e.grad_dtype, lane, left < kStateBlock ? static_cast<int>(left) : kStateBlock, g);
#pragma unroll
        for (int k = 0; k < 8; k += 2) sq.take(g[k], g[k + 1]);
    }
    float h0, h1, l0, l1;
    unpack2(sq.hi, h0, h1);
    unpack2(sq.lo, l0, l1);
    const bool bad = sq.bad;
    double part = __dadd_rn(__dadd_rn(static_cast<double>(h0), static_cast<double>(l0)), __dadd_rn(static_cast<double>(h1), static_cast<double>(l1)));
    const bool left_range = !(is_finite_f32(h0) && is_finite_f32(h1) && is_finite_f32(l0) && is_finite_f32(l1));
    // (with a non-finite gradient under loss scaling the step is skipped, whatever the norm)
    if (a.clip && __any_sync(0xFFFFFFFFu, left_range) && !(a.hp.loss_scaling && __any_sync(0xFFFFFFFFu, bad)))
        part = squares_in_fp64(t, first, last, sq);
    part = warp_sum_f64(part);
    if (lane == 0) red[warp] = part;
    if (__syncthreads_or(bad) && a.hp.loss_scaling && threadIdx.x == 0) atomicExch(&a.sc->nonfinite, 1);
    if (!a.clip) return;
    if (threadIdx.x == 0) {
        double tot = 0.0;
        for (int w = 0; w < kThreadsT / 32; ++w) tot = __dadd_rn(tot, red[w]);
        partials[blockIdx.x] = tot;
        last_one = 0;
        if (a.finalize) {
            __threadfence();
            last_one = atomicAdd(&a.sc->ctas_done, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (last_one && warp == 0) {
        __threadfence();
        double all = 0.0;
        for (int k = lane; k < a.n_partials; k += 32) all = __dadd_rn(all, __ldcg(a.partials + k));
        all = warp_sum_f64(all);
        if (lane == 0) {
            a.sc->sqnorm = all;
            // max_norm over a norm that is not a number is not 1
            a.sc->clip_coef = isnan(all) ? __uint_as_float(0x7FC00000u) : clip_coefficient(a.hp.max_norm, all);
            a.sc->ctas_done = 0u;
        }
    }
}

template <int CAP>
cudaError_t launch_table(const TensorTable<CAP>& t, AdamwArgs a, double* partials, int grid, bool norm, cudaStream_t st)
{
    count_launch();
    if (norm) {
        k_tensors_norm<CAP><<<grid, kThreadsT, 0, st>>>(t, a, partials);
        return cudaGetLastError();
    }
    const int smem = t.ring ? kRing * kRingStage : 0;
    const cudaError_t e = cudaFuncSetAttribute(k_adamw<CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * kRingStage);
    if (e != cudaSuccess) return e;
    k_adamw<CAP><<<grid, kThreadsT, smem, st>>>(t, a);
    return cudaGetLastError();
}

}  // namespace

// CTAs of the norm pass over `tiles` tiles, the same on every device (each leaves a
// partial sum)
int norm_grid(int tiles) { return tiles < 1 ? 1 : tiles < kNormCtas ? tiles : kNormCtas; }

namespace {

// CTAs of the step: several times as many as run at a time.  Those far from their
// memory take half as long again as the others (with equal shares an SM was busy for
// 292 to 458 K clocks), and an SM that is done early takes the next: 436M parameters
// with 8-bit states 1357 us with 456 CTAs, 1230 with 15048 (14 tiles each), 1209 with
// 3648 (56 each).  Shorter shares wait for the step's constants too often; those of
// 32-bit states, which have no ring to fill meanwhile, are twice as long (105M
// parameters 461 us, 457 with 456 CTAs).  Whole multiples: 1839 CTAs, where 456 run at
// a time, leave the last 15 a turn to themselves (504 us).
int step_grid(int tiles, bool ring)
{
    const int turns = tiles / ((ring ? 1 : 2) * kTilesEach * kStepCtas);
    return tiles < kStepCtas ? (tiles < 1 ? 1 : tiles) : kStepCtas * (turns < 1 ? 1 : turns);
}

}  // namespace

cudaError_t launch_adamw(const TensorList& list, const zero_hparams& hp, zero_dev_scalars* sc, double* partials, cudaStream_t st)
{
    AdamwArgs a = {};
    a.hp = hp;
    a.sc = sc;
    a.partials = partials;
    a.clip = hp.max_norm > 0.0f;
    const bool pass = a.clip || hp.loss_scaling;
    for (int norm = pass ? 1 : 0; norm >= 0; --norm) {
        int at = 0;
        for (size_t k = 0; k < list.launches(); ++k) {
            const bool small = list.big.empty();
            const int tiles = small ? list.small.tiles : list.big[k].tiles, grid = norm != 0 ? norm_grid(tiles) : step_grid(tiles, (small ? list.small.ring : list.big[k].ring) != 0);
            a.n_partials = list.partials;
            a.finalize = a.commit = k + 1 == list.launches();
            const cudaError_t e = small ? launch_table(list.small, a, partials + at, grid, norm != 0, st)
                                        : launch_table(list.big[k], a, partials + at, grid, norm != 0, st);
            if (e != cudaSuccess) return e;
            at += grid;
        }
    }
    return cudaSuccess;
}

}  // namespace zk
