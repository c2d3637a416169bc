// Shared by the kernels of libarcserve: element types, e4m3 conversions and
// host-side launch helpers.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "arc_sample.h"

namespace arcs {

constexpr int kScaleExp = 32;  // page scales written here lie in [2^-32, 2^32]

template <int DT>
struct Half;  // the 16-bit element types

template <>
struct Half<ARC_BF16> {
    using T = __nv_bfloat16;
    __device__ __forceinline__ static float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ __forceinline__ static uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float to_float(T x) { return __bfloat162float(x); }
    __device__ __forceinline__ static T from_float(float x) { return __float2bfloat16_rn(x); }
};

template <>
struct Half<ARC_F16> {
    using T = __half;
    __device__ __forceinline__ static float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    __device__ __forceinline__ static uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float to_float(T x) { return __half2float(x); }
    __device__ __forceinline__ static T from_float(float x) { return __float2half_rn(x); }
};

// Eight consecutive 16-bit elements: one 16-byte load where the address allows
// it (`vec`), else eight element loads.
template <int DT>
__device__ __forceinline__ void load8(const void* p, bool vec, float (&x)[8]) {
    if (vec) {
        const uint4 v = *static_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Half<DT>::unpack(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        const typename Half<DT>::T* e = static_cast<const typename Half<DT>::T*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = Half<DT>::to_float(e[i]);
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, bool vec, const float (&x)[8]) {
    if (vec) {
        *static_cast<uint4*>(p) = make_uint4(Half<DT>::pack(x[0], x[1]), Half<DT>::pack(x[2], x[3]),
                                             Half<DT>::pack(x[4], x[5]), Half<DT>::pack(x[6], x[7]));
    } else {
        typename Half<DT>::T* e = static_cast<typename Half<DT>::T*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = Half<DT>::from_float(x[i]);
    }
}

// Two e4m3 codes, `a` in the low byte: nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The four e4m3 codes of w as two f16x2 (exact), the lower two first.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Least e in [-32, 32] with amax <= 448 * 2^e; 448 = 1.75 * 2^8, so the
// exponent of amax counts one more when its mantissa passes 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>((b + 0x1FFFFFu) >> 23) - 127 - 8;
    return e < -kScaleExp ? -kScaleExp : (e > kScaleExp ? kScaleExp : e);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e for |e| <= 126.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace arcs
