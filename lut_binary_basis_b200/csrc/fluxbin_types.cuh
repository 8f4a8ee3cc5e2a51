// Conversions between fp32 and the types of the 8-bit operators' arrays, and
// 16-byte pieces of rows that start off a 16-byte boundary.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace fluxbin {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The 16 bytes that start `by` bytes (below 16, a multiple of 2) into w[K..K+7].
template <int K>
__device__ __forceinline__ uint4 shifted(const uint32_t* w, uint32_t by) {
    uint32_t x[6], y[5], r[4];
#pragma unroll
    for (int k = 0; k < 6; ++k) x[k] = (by & 8u) ? w[K + k + 2] : w[K + k];
#pragma unroll
    for (int k = 0; k < 5; ++k) y[k] = (by & 4u) ? x[k + 1] : x[k];
    const uint32_t sel = (by & 2u) ? 0x5432u : 0x3210u;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __byte_perm(y[k], y[k + 1], sel);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void put(uint32_t* w, const uint4& v) {
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
}

}  // namespace fluxbin
