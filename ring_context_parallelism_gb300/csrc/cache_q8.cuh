// cache_q8.cuh -- the 8-bit form of a paged cache: codes in e4m3, and for every token and
// KV head one byte e that gives the scale 2^(e - 127) (zero where e is 0).
//
// A power of two as the scale costs nothing in a format with an exponent of its own: every
// normal code keeps its four significant bits, and scaling rounds nothing.  The scale
// written is the least one that brings the row's largest value to at most 448, the
// largest code, and at least 2^-126.
#pragma once

#include <cuda_fp8.h>

#include "cache_simt.cuh"

namespace ra {

__device__ __forceinline__ float scale_of(unsigned e) { return __uint_as_float(e << 23); }

// The scale byte of a row whose values have the largest magnitude with these bits (that of a NaN is above infinity's).
__device__ __forceinline__ unsigned scale_byte(unsigned largest) {
    const int e = static_cast<int>(largest >> 23) - 8 + ((largest & 0x7fffffu) > 0x600000u ? 1 : 0);
    return static_cast<unsigned>(max(e, 1));
}

// Four values times `inverse` as codes, the first in the lowest byte: to the nearest, ties to even, an infinity to 448.
__device__ __forceinline__ uint32_t codes4(const float* x, float inverse) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inverse, x[1] * inverse), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inverse, x[3] * inverse), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

__device__ __forceinline__ void values4(uint32_t codes, float* x) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> (16 * j)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

// Eight consecutive elements.
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = lds4(p), b = lds4(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    store4(p, make_float4(x[0], x[1], x[2], x[3]));
    store4(p + 4, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}

}  // namespace ra
