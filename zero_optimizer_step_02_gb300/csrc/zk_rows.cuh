// zk_rows.cuh -- rows of [rows, cols] arrays in 16-byte words: what the norms'
// kernels share.  Elements in whichever type, words that hold a part of a row,
// asynchronous copies into shared memory.
#pragma once

#include "zk_common.cuh"

namespace zk {

template <int DT>
struct El;
template <>
struct El<ZERO_BF16> {
    using T = uint16_t;
    __device__ static __forceinline__ float up(T v) { return Lp<ZERO_BF16>::widen(v); }
    __device__ static __forceinline__ T down(float v) { return Lp<ZERO_BF16>::narrow(v); }
};
template <>
struct El<ZERO_FP16> {
    using T = uint16_t;
    __device__ static __forceinline__ float up(T v) { return Lp<ZERO_FP16>::widen(v); }
    __device__ static __forceinline__ T down(float v) { return Lp<ZERO_FP16>::narrow(v); }
};
template <>
struct El<ZERO_FP32> {
    using T = float;
    __device__ static __forceinline__ float up(T v) { return v; }
    __device__ static __forceinline__ T down(float v) { return v; }
};

// a weight vector's element in whichever type it has
__device__ __forceinline__ float weight_at(const void* w, int dt, long long i)
{
    if (dt == ZERO_FP32) return static_cast<const float*>(w)[i];
    const uint16_t h = static_cast<const uint16_t*>(w)[i];
    return dt == ZERO_BF16 ? Lp<ZERO_BF16>::widen(h) : Lp<ZERO_FP16>::widen(h);
}
__device__ __forceinline__ void put_weight(void* w, int dt, long long i, float v)
{
    if (dt == ZERO_FP32)
        static_cast<float*>(w)[i] = v;
    else
        static_cast<uint16_t*>(w)[i] = dt == ZERO_BF16 ? Lp<ZERO_BF16>::narrow(v) : Lp<ZERO_FP16>::narrow(v);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// 1 / sqrt(v) to an ulp or so: the approximate root and a Newton step (a root
// and a division in every thread were a seventh of the forward kernel's
// instructions).  0, infinity and NaN as they come.
__device__ __forceinline__ float inverse_root(float v)
{
    const float y = rsqrtf(v), e = fmaf(-v * y, y, 1.0f);
    return is_finite_f32(e) ? fmaf(0.5f * y, e, y) : y;
}

template <int DT>
constexpr int kV = DT == ZERO_FP32 ? 4 : 8;

__device__ __forceinline__ void cp_async16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// the compiler forgets that it has this chunk's values widened already
__device__ __forceinline__ void forget(uint4& w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

template <int DT>
__device__ __forceinline__ void widen(const uint4& w, float (&v)[kV<DT>])
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    if constexpr (DT == ZERO_FP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = Lp<DT>::lo(a[i]), v[2 * i + 1] = Lp<DT>::hi(a[i]);
    }
}

// the same as register pairs, for the packed fp32 operations
template <int DT>
__device__ __forceinline__ void widen(const uint4& w, f32x2 (&v)[kV<DT> / 2])
{
    float f[kV<DT>];
    widen<DT>(w, f);
#pragma unroll
    for (int i = 0; i < kV<DT> / 2; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void unpack(const f32x2 (&p)[N], float (&v)[2 * N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) unpack2(p[i], v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ float both(f32x2 v)
{
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

// xhat of a row with this mean and 1 / std.  |xhat| <= sqrt(cols), and an x that
// is not the mean differs from it by 2^-25 of it or more: where |mean| * rstd
// passes 2^40, every x is the mean and xhat is 0, however large mean * rstd (an
// overflow would make it NaN).  rstd NaN or infinite: as they come.
template <int DT>
struct Centred {
    f32x2 rs, by;
    __device__ __forceinline__ Centred(float mean, float rstd)
    {
        const float nm = -mean * rstd;
        const bool flat = fabsf(nm) > 1.099511627776e12f && is_finite_f32(rstd);
        const float r = flat ? 0.0f : rstd, b = DT == ZERO_FP32 ? mean : flat ? 0.0f : nm;
        rs = pack2(r, r);
        by = pack2(b, b);
    }
    __device__ __forceinline__ f32x2 xhat(f32x2 x) const
    {
        if constexpr (DT == ZERO_FP32)
            return mul2(sub2(x, by), rs);
        else
            return fma2(x, rs, by);
    }
};

// a chunk without the columns before 0 and from `cols` on (zeros there); c: its first
template <int DT>
__device__ __forceinline__ uint4 masked(const uint4& w, int c, int cols)
{
    if (c >= 0 && c + kV<DT> <= cols) return w;
    uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == ZERO_FP32) {
            if (c + i < 0 || c + i >= cols) a[i] = 0;
        } else {
            if (c + 2 * i < 0 || c + 2 * i >= cols) a[i] &= 0xFFFF0000u;
            if (c + 2 * i + 1 < 0 || c + 2 * i + 1 >= cols) a[i] &= 0xFFFFu;
        }
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
}

template <int DT>
__device__ __forceinline__ uint4 narrowed(const float (&v)[kV<DT>])
{
    if constexpr (DT == ZERO_FP32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        return make_uint4(Lp<DT>::narrow2(v[0], v[1]), Lp<DT>::narrow2(v[2], v[3]), Lp<DT>::narrow2(v[4], v[5]),
                          Lp<DT>::narrow2(v[6], v[7]));
}

// A [rows, cols] array read row by row.
template <int DT>
struct RowSource {
    using T = typename El<DT>::T;
    const T* base;
    long long stride;
    uintptr_t lo, hi;   // the bytes from the first row's first to the last row's last element

    __device__ __forceinline__ RowSource(const void* p, long long s, long long rows, int cols)
        : base(static_cast<const T*>(p)), stride(s), lo(reinterpret_cast<uintptr_t>(p)),
          hi(lo + static_cast<uintptr_t>((rows - 1) * s + cols) * sizeof(T))
    {
    }
    __device__ __forceinline__ uintptr_t row(long long r) const { return reinterpret_cast<uintptr_t>(base + r * stride); }

    // The aligned word at `at`, which holds elements of the row [from, to), into
    // *dst: whole if it lies inside the array (as it does unless `ends`), else the
    // row's elements alone.
    __device__ __forceinline__ void copy_word(uint4* dst, uintptr_t at, uintptr_t from, uintptr_t to, bool ends) const
    {
        if (!ends || (at >= lo && at + 16 <= hi)) {
            cp_async16(dst, reinterpret_cast<const void*>(at));
            return;
        }
        T* d = reinterpret_cast<T*>(dst);
        for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) {
            const uintptr_t q = at + e * sizeof(T);
            if (q >= from && q < to) d[e] = *reinterpret_cast<const T*>(q);
        }
    }

    // columns c .. of the row at q, four bytes each (fp32)
    __device__ __forceinline__ void copy_fours(uint4* dst, const T* q, int c, int cols) const
    {
#pragma unroll
        for (int e = 0; e < kV<DT>; ++e)
            if (c + e >= 0 && c + e < cols) cp_async4(reinterpret_cast<uint32_t*>(dst) + e, q + c + e);
    }

    // The same if the word holds any of the row's elements (one that does not
    // may lie in memory that is not there).
    __device__ __forceinline__ void copy_if_any(uint4* dst, uintptr_t at, uintptr_t from, uintptr_t to, bool ends) const
    {
        if (at + 16 > from && at < to) copy_word(dst, at, from, to, ends);
    }
};

// V results from column c on of the row that starts at `row` (kAlike: c + row's
// offset is a whole word; a row's first and last words are written in part)
template <int DT>
__device__ __forceinline__ void put_word(uintptr_t row, int c, int cols, const uint4& w)
{
    using T = typename El<DT>::T;
    T* p = reinterpret_cast<T*>(row) + c;
    if (c >= 0 && c + kV<DT> <= cols) {
        __stcs(reinterpret_cast<uint4*>(p), w);
        return;
    }
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < kV<DT>; ++e) {
        if (c + e < 0 || c + e >= cols) continue;
        if constexpr (sizeof(T) == 4)
            reinterpret_cast<uint32_t*>(p)[e] = a[e];
        else
            reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(a[e / 2] >> (16 * (e & 1)));
    }
}

inline int sms_of_device()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

}  // namespace zk
