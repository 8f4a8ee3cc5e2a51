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
};

constexpr uint32_t kInt8Accumulate = 1u, kInt8YFp32 = 2u, kInt8Early = 4u, kInt8Bf16 = 256u;

// y = v or y += v, in y's type (the sum of an accumulation is taken in fp32
// and rounded once).
__device__ __forceinline__ void int8_store(const Int8Args& p, int64_t t, int m, float v) {
    const int64_t o = t * p.ldy + m;
    if (p.flags & kInt8YFp32) {
        float* y = static_cast<float*>(p.y) + o;
        *y = (p.flags & kInt8Accumulate) ? *y + v : v;
    } else if (p.flags & kInt8Bf16) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
        *y = __float2bfloat16_rn((p.flags & kInt8Accumulate) ? __bfloat162float(*y) + v : v);
    } else {
        __half* y = static_cast<__half*>(p.y) + o;
        *y = __float2half_rn((p.flags & kInt8Accumulate) ? __half2float(*y) + v : v);
    }
}

// Four codes n .. n+3 of a row of N (zeros past its end; the bytes after it
// are not read).
__device__ __forceinline__ int int8_load4(const int8_t* row, int n, int N) {
    if (n + 4 <= N) return *reinterpret_cast<const int*>(row + n);
    int v = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (n + i < N) v |= (int)(uint8_t)row[n + i] << (8 * i);
    return v;
}

constexpr int kInt8Tile = 64, kInt8TileK = 64;

// 64 tokens x 64 channels a CTA, 256 threads of 4 x 4 sums.
__global__ void __launch_bounds__(256) fluxbin_int8_kernel(const Int8Args p) {
    __shared__ int xs[kInt8TileK / 4][kInt8Tile + 1];
    __shared__ int ws[kInt8TileK / 4][kInt8Tile + 1];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int m0 = blockIdx.x * kInt8Tile;
    const int t0 = blockIdx.y * kInt8Tile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.N; k0 += kInt8TileK) {
        for (int i = threadIdx.x; i < kInt8Tile * kInt8TileK / 4; i += 256) {
            const int r = i / (kInt8TileK / 4), c = i % (kInt8TileK / 4);
            xs[c][r] = t0 + r < p.T ? int8_load4(p.x + (t0 + r) * p.ldx, k0 + 4 * c, p.N) : 0;
            ws[c][r] = m0 + r < p.M ? int8_load4(p.w + (m0 + r) * p.ldw, k0 + 4 * c, p.N) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kInt8TileK / 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[c][ty + 16 * i], ws[c][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty + 16 * i, m = m0 + tx + 16 * j;
            if (t < p.T && m < p.M) int8_store(p, t, m, (float)acc[i][j] * (p.sx[t] * p.sw[m]));
        }
}

}  // namespace fluxbin
