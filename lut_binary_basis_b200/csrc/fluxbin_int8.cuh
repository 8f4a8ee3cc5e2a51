// 8-bit integer product with a scale for each token and each channel (sm_100a):
//
//   y[t][m] (+)= sx[t] * sw[m] * sum_n xq[t][n] * wq[m][n]
//
// The sum is an exact 32-bit integer (|sum| <= 128^2 N < 2^31 for
// N <= 131071), so neither tiling nor splitting changes a result; it is
// rounded to fp32 once, multiplied by the two scales and rounded to y's type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fluxbin_types.cuh"

namespace fluxbin {

struct Int8Args {
    const int8_t* w;      // [M][ldw]
    const float* sw;      // [M]
    const int8_t* x;      // [T][ldx]
    const float* sx;      // [T]
    void* y;              // [T][ldy]
    int64_t ldw, ldx, ldy;
    int32_t M, N, T;
    uint32_t flags;
    int32_t vec4;         // rows of y allow accesses of four elements
};

constexpr uint32_t kInt8Accumulate = 1u, kInt8YFp32 = 2u, kInt8Early = 4u, kInt8Bf16 = 256u;

__device__ __forceinline__ float int8_value(int acc, float sx, float sw) {
    // no contraction with the accumulation's addition: the same bits in every kernel
    return __fmul_rn((float)acc, __fmul_rn(sx, sw));
}

// The product of no input features: y (+)= 0 * scales.
template <typename Y, bool ACC>
__global__ void __launch_bounds__(256) fluxbin_int8_empty_kernel(const Int8Args p) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (int64_t)p.T * p.M) return;
    const int64_t t = i / p.M, m = i % p.M;
    Y* y = static_cast<Y*>(p.y) + t * p.ldy + m;
    const float v = int8_value(0, p.sx[t], p.sw[m]);
    *y = from_f32<Y>(ACC ? to_f32(*y) + v : v);
}

}  // namespace fluxbin
