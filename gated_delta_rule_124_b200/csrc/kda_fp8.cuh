// 8-bit values with a scale per block of 128 (internal to libkda): e4m3 codes
// y8 = round(x * f) with f = 448 / amax and the fp32 scale amax / 448 that gives x
// back, amax the block's largest magnitude.  f and x * f are fp32 numbers, so that a
// value that lies exactly between two codes may take either (2 in 10,000 of normally
// distributed bf16 values do not take the even one).  One rounding to 4 significant
// bits, at most half a step (2^-4 of the value) off down to amax * 2^-15, where e4m3's
// subnormal numbers begin.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

constexpr float kFp8Max = 448.f;
// Blocks whose values are all smaller are scaled as if one were this large, so
// that neither 448 / amax nor the scale leaves the normal fp32 range (a block
// of zeros included).
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100

// What to multiply by for a block's maximum, and its scale.
__device__ __forceinline__ float fp8_factor(float amax) { return kFp8Max / fmaxf(amax, kAmaxFloor); }
__device__ __forceinline__ float fp8_scale(float amax) { return fmaxf(amax, kAmaxFloor) / kFp8Max; }

__device__ __forceinline__ uint32_t fp8x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
    return fp8x2(a, b) | fp8x2(c, d) << 16;
}

// Eight consecutive elements of a row, from a 16-byte boundary, as they lie in
// memory (a load in flight holds no more registers than its bytes).
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
__device__ __forceinline__ void store_vec8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_vec8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ float max_abs8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}
// The largest value over 16 consecutive lanes (a block of 128 columns, eight a lane).
__device__ __forceinline__ float max16(float m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float f) {
    return make_uint2(fp8x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                      fp8x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
}

}  // namespace kda
