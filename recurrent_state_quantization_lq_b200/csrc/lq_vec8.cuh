// Eight consecutive channels of a row in one thread: packed loads, widening to
// FP32 and rounding stores (BF16 or FP32 rows).
#pragma once

#include "lq_common.cuh"

namespace lq {

// Eight values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 w;
};
template <>
struct Raw8<float> {
    float4 lo, hi;
};

__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16> &r) { r.w = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero8(Raw8<float> &r) { r.lo = r.hi = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16> &r, float *f) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8<float> &r, float *f) {
    f[0] = r.lo.x; f[1] = r.lo.y; f[2] = r.lo.z; f[3] = r.lo.w;
    f[4] = r.hi.x; f[5] = r.hi.y; f[6] = r.hi.z; f[7] = r.hi.w;
}

// The same as four pairs.
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float2 *f) {
    float x[8];
    widen8(r, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// The first n (1..8) channels of a row; the rest are zero.  VEC: p is 16-byte
// aligned and n whole pieces of 16 bytes (8 BF16 channels; 4 or 8 FP32).
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, Raw8<__nv_bfloat16> &r) {
    if constexpr (VEC) {
        r.w = __ldg(reinterpret_cast<const uint4 *>(p));
    } else {
        const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 2] |= (uint32_t)__ldg(h + i) << (16 * (i & 1));
        r.w = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int n, Raw8<float> &r) {
    if constexpr (VEC) {
        r.lo = __ldg(reinterpret_cast<const float4 *>(p));
        r.hi = n > 4 ? __ldg(reinterpret_cast<const float4 *>(p) + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? __ldg(p + i) : 0.0f;
        r.lo = make_float4(f[0], f[1], f[2], f[3]);
        r.hi = make_float4(f[4], f[5], f[6], f[7]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int n, const float *f) {
    if constexpr (VEC) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(f[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int n, const float *f) {
    if constexpr (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        if (n > 4) reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = f[i];
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T *p, int n, const float2 *f) {
    const float x[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    store8<VEC>(p, n, x);
}

// Two FP32 operations in one instruction (sm_100a's packed pairs); each half
// rounds as the scalar operation does.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// Lanes that share a row of d channels, eight each: a power of two, 1..32.
__host__ __device__ constexpr int row_lanes(int d) {
    int l = 1;
    while (8 * l < d) l *= 2;
    return l;
}

}  // namespace lq
