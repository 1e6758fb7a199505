// Rows of f32, f16 or bf16 values whose type is known at run time: four values
// at a time in f32, and back with one rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/plm.h"

namespace plm {

__host__ __device__ __forceinline__ int type_bytes(int type) { return type == PLM_F32 ? 4 : 2; }

// Whether four values of a row are one aligned access: pointer and stride.
inline bool four_aligned(const void* p, long long stride, int type) {
    return (uintptr_t)p % (4 * type_bytes(type)) == 0 && stride % 4 == 0;
}

__device__ __forceinline__ float value_at(const void* p, int type, long long i) {
    if (type == PLM_F32) return static_cast<const float*>(p)[i];
    if (type == PLM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void value_put(void* p, int type, long long i, float v) {
    if (type == PLM_F32) static_cast<float*>(p)[i] = v;
    else if (type == PLM_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float value_rounded(float v, int type) {
    return type == PLM_F32 ? v : type == PLM_F16 ? __half2float(__float2half_rn(v)) : __bfloat162float(__float2bfloat16_rn(v));
}

// Values i .. i + 3, of which the first n are there (the others give 0); four:
// one access (four_aligned, i a multiple of 4, n 4 or none).
__device__ __forceinline__ float4 load_four(const void* p, int type, long long i, int n, bool four) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n <= 0) return v;
    if (four) {
        if (type == PLM_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        if (type == PLM_F16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
            return make_float4(a.x, a.y, b.x, b.y);
        }
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xFFFF0000u));
    }
    v.x = value_at(p, type, i);
    if (n > 1) v.y = value_at(p, type, i + 1);
    if (n > 2) v.z = value_at(p, type, i + 2);
    if (n > 3) v.w = value_at(p, type, i + 3);
    return v;
}
__device__ __forceinline__ void store_four(void* p, int type, long long i, int n, bool four, float4 v) {
    if (n <= 0) return;
    if (four) {
        if (type == PLM_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
        } else if (type == PLM_F16) {
            const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
        return;
    }
    value_put(p, type, i, v.x);
    if (n > 1) value_put(p, type, i + 1, v.y);
    if (n > 2) value_put(p, type, i + 2, v.z);
    if (n > 3) value_put(p, type, i + 3, v.w);
}

}  // namespace plm
