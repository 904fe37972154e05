// Rows of channels in pieces of eight (16 bytes of bf16), and their 8-bit codes with a scale: what the
// RMS norm and the quantisation share.
#pragma once
#include <cuda_fp8.h>

#include "gdr_common.cuh"

namespace gdr {
namespace {

// eight consecutive channels, and as loaded
struct Eight {
    float v[8];
};
__device__ __forceinline__ float2 two(const Eight& e, int q) { return make_float2(e.v[2 * q], e.v[2 * q + 1]); }
__device__ __forceinline__ void set_two(Eight& e, int q, float2 f) {
    e.v[2 * q] = f.x;
    e.v[2 * q + 1] = f.y;
}
// two bf16, by a shift and a mask (the conversion function takes three instructions)
__device__ __forceinline__ float2 widen_pair(uint32_t r) { return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)); }
template <class T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ Eight widen() const {
        Eight e;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen_pair(w[i]);
            e.v[2 * i] = f.x;
            e.v[2 * i + 1] = f.y;
        }
        return e;
    }
};
template <> struct RawOf<float> {
    float4 a, b;
    __device__ __forceinline__ Eight widen() const { return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
// `n` channels of a row from p on; `wide`: rows are whole numbers of aligned pieces, else pairs
__device__ __forceinline__ RawOf<__nv_bfloat16> ld8(const __nv_bfloat16* p, int n, bool wide) {
    if (wide) return {__ldcs(reinterpret_cast<const uint4*>(p))};
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    return {make_uint4(__ldcs(q), n > 2 ? __ldcs(q + 1) : 0u, n > 4 ? __ldcs(q + 2) : 0u, n > 6 ? __ldcs(q + 3) : 0u)};
}
__device__ __forceinline__ RawOf<float> ld8(const float* p, int n, bool wide) {
    if (wide) return {__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1)};
    const float2* q = reinterpret_cast<const float2*>(p);
    const float2 none = make_float2(0.f, 0.f), f0 = __ldcs(q), f1 = n > 2 ? __ldcs(q + 1) : none, f2 = n > 4 ? __ldcs(q + 2) : none,
                 f3 = n > 6 ? __ldcs(q + 3) : none;
    return {make_float4(f0.x, f0.y, f1.x, f1.y), make_float4(f2.x, f2.y, f3.x, f3.y)};
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const Eight& e) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                                              pack_bf16(e.v[6], e.v[7]));
}
__device__ __forceinline__ void st8(float* p, const Eight& e) {
    reinterpret_cast<float4*>(p)[0] = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}
// pairs
template <class T> __device__ __forceinline__ float2 ld2(const T* p);
template <> __device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) { return unpack_bf16(__ldcs(reinterpret_cast<const uint32_t*>(p))); }
template <> __device__ __forceinline__ float2 ld2(const float* p) { return __ldcs(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ void st2(__nv_bfloat16* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = pack_bf16(v.x, v.y); }
__device__ __forceinline__ void st2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
template <class T>
__device__ __forceinline__ void st8n(T* p, const Eight& e, int n, bool wide) {
    if (wide) {
        st8(p, e);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        if (i < n) st2(p + i, make_float2(e.v[i], e.v[i + 1]));
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// The scale of values up to m: m / 448, 1 where all are zero.  Where m / 448 rounds to zero it is the
// smallest float32, so that zeros stay zero.
__device__ __forceinline__ float scale_of(float m) { return m > 0.f ? fmaxf(m / 448.f, 1.4e-45f) : 1.f; }
// The codes of y / scale.  A product with 1 / scale (two steps of the last place off at most) is within
// 3 2^-23 of the quotient, so that products to either side by 2^-21 have the quotient's code unless a tie
// lies between them: then (some 10^-5 of the values), or where 1 / scale is far from the normal numbers,
// the division itself decides.  (In the norm, dividing every value of 32768 x 2048 takes 98 us, this 85, the product
// alone, which takes the other code next to a tie and is infinite for scales below 2^-128, 81.)
__device__ __forceinline__ void codes_of(const Eight& y, float scale, uint32_t (&h)[4]) {
    const float inv = __fdividef(1.f, scale), under = inv * (1.f - 0x1p-21f), over = inv * (1.f + 0x1p-21f);
    uint32_t differ = scale > 0x1p-120f && scale < 0x1p120f ? 0 : 1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 a = __fmul2_rn(two(y, q), make_float2(under, under)), b = __fmul2_rn(two(y, q), make_float2(over, over));
        h[q] = e4m3x2(a.x, a.y);
        differ |= h[q] ^ e4m3x2(b.x, b.y);
    }
    if (differ) {
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = e4m3x2(y.v[2 * q] / scale, y.v[2 * q + 1] / scale);
    }
}

}  // namespace
}  // namespace gdr
