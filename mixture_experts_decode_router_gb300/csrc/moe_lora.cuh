// moe_lora.cuh -- what the adapters' kernels (moe_lora.cu, moe_lora_tc.cu) share: v's parts, and
// elements of base and out.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

// v as a sum of `kParts` 16-bit numbers; an infinity (or what rounds to one) and a NaN have one part.
template <bool kBf16, int kParts> __device__ __forceinline__ void split(float v, uint16_t (&part)[kParts]) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        float f;
        if constexpr (kBf16) {
            const __nv_bfloat16 b = __float2bfloat16_rn(v);
            part[i] = __bfloat16_as_ushort(b);
            f = __bfloat162float(b);
        } else {
            const __half b = __float2half_rn(v);
            part[i] = __half_as_ushort(b);
            f = __half2float(b);
        }
        v = fabsf(f) < INFINITY ? v - f : 0.f;
    }
}

// Single elements.
template <int kType> __device__ __forceinline__ uint32_t load_bits(const void* p, int64_t at) {
    if constexpr (kType == MOE_F32) return reinterpret_cast<const uint32_t*>(p)[at];
    else return reinterpret_cast<const uint16_t*>(p)[at];
}
template <int kType> __device__ __forceinline__ float of_bits(uint32_t u) {
    if constexpr (kType == MOE_F32) return __uint_as_float(u);
    else if constexpr (kType == MOE_BF16) return bf16_lo(u);
    else return __half2float(__ushort_as_half((uint16_t)u));
}
template <int kType> __device__ __forceinline__ float load_one(const void* p, int64_t at) { return of_bits<kType>(load_bits<kType>(p, at)); }
template <int kType> __device__ __forceinline__ void store_bits(void* p, int64_t at, uint32_t u) {
    if constexpr (kType == MOE_F32) reinterpret_cast<uint32_t*>(p)[at] = u;
    else reinterpret_cast<uint16_t*>(p)[at] = (uint16_t)u;
}
template <int kType> __device__ __forceinline__ void store_one(void* p, int64_t at, float v) {
    if constexpr (kType == MOE_F32) reinterpret_cast<float*>(p)[at] = v;
    else reinterpret_cast<uint16_t*>(p)[at] = kType == MOE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
// Four elements of a row of base or out, `step` apart, as far as there are (`left`, counted from the first).
// Neighbouring ones (step 1) are four elements aligned together.
template <int kType> __device__ __forceinline__ void load4_of(const void* p, int64_t at, int step, int left, float (&v)[4]) {
    if (step == 1 && left >= 4) {
        if constexpr (kType == MOE_F32) {
            const float4 q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
            v[0] = of_bits<kType>(q.x & 0xffffu); v[1] = of_bits<kType>(q.x >> 16);
            v[2] = of_bits<kType>(q.y & 0xffffu); v[3] = of_bits<kType>(q.y >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i * step < left ? load_one<kType>(p, at + i * step) : 0.f;
    }
}
__device__ __forceinline__ void load4(int type, const void* p, int64_t at, int step, int left, float (&v)[4]) {
    if (type == MOE_F32) load4_of<MOE_F32>(p, at, step, left, v);
    else if (type == MOE_BF16) load4_of<MOE_BF16>(p, at, step, left, v);
    else load4_of<MOE_F16>(p, at, step, left, v);
}
template <int kType> __device__ __forceinline__ void store4_of(void* p, int64_t at, int step, int left, const float (&v)[4]) {
    if (step == 1 && left >= 4) {
        if constexpr (kType == MOE_F32) {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            uint16_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) store_one<kType>(u, i, v[i]);
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) = make_uint2(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * step < left) store_one<kType>(p, at + i * step, v[i]);
    }
}
__device__ __forceinline__ void store4(int type, void* p, int64_t at, int step, int left, const float (&v)[4]) {
    if (type == MOE_F32) store4_of<MOE_F32>(p, at, step, left, v);
    else if (type == MOE_BF16) store4_of<MOE_BF16>(p, at, step, left, v);
    else store4_of<MOE_F16>(p, at, step, left, v);
}

// The 16 bytes of four elements (fp32) or eight.
template <int kType> __device__ __forceinline__ void add_raw(const uint4& was, float* y) {
    const uint32_t u[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == MOE_F32) {
            y[i] += __uint_as_float(u[i]);
        } else if constexpr (kType == MOE_BF16) {
            y[2 * i] += bf16_lo(u[i]);
            y[2 * i + 1] += bf16_hi(u[i]);
        } else {
            const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            y[2 * i] += q.x;
            y[2 * i + 1] += q.y;
        }
    }
}
// The same from single elements.
template <int kType> __device__ __forceinline__ uint4 gather_raw(const void* p, int64_t at) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = kType == MOE_F32 ? load_bits<kType>(p, at + i) : load_bits<kType>(p, at + 2 * i) | load_bits<kType>(p, at + 2 * i + 1) << 16;
    return make_uint4(u[0], u[1], u[2], u[3]);
}
template <int kType> __device__ __forceinline__ uint4 pack_raw(const float* y) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == MOE_F32) {
            u[i] = __float_as_uint(y[i]);
        } else if constexpr (kType == MOE_BF16) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&q);
        } else {
            const __half2 q = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&q);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace moe
