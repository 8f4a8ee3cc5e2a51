// Row-wise 8-bit quantisation (sm_100a): the operators that produce the
// left operand of the 8-bit integer product.
//
// A row v of N values becomes codes and one scale,
//     a = max_n |v_n|,   q_n = rint(v_n * (127 / a)),   s = a / 127,
// (round to nearest even, codes in -127..127), v_n ~ q_n s.  The row is
//   quant     v = x
//   silu_mul  v = g / (1 + exp(-g)) * u
//   rmsnorm   v = h' (.) gamma * r,  h' = h + delta rounded to h's type,
//             r = 1 / sqrt(mean(h'^2) + eps)
// In rmsnorm r > 0 is a factor of the whole row, so it cancels in v / a: the
// codes come from w = h' (.) gamma alone and r only enters the scale,
// s = max|w| * r / 127.  One pass over the row then gives both reductions (the
// sum of squares and the maximum) and the codes need no second one; for
// 16-bit h' and gamma the products w are exact in fp32, so the codes do not
// depend on the order in which the squares are summed.
//
// A row of zeros gets codes 0 and scale 0.  A row that has no finite scale (a
// NaN or an infinity in it, a sum of squares beyond fp32) gets codes 0 and
// scale NaN: every product with it is NaN, nothing is hidden.  The maximum is
// taken over the bit patterns of |v| as integers, whose order is that of the
// values with NaN above infinity, so a NaN is never lost in it.
//
// Bound: memory (one read of each input, one write of each output).  A row is
// owned by blockDim.x threads and stays in their registers between the
// reductions and the codes (VPT vectors of 8 elements a thread); rows of more
// than 32,768 elements are read twice (VPT = 0).  Rows that allow 16-byte
// accesses take them (VEC); others are read element by element with
// consecutive threads on consecutive elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fluxbin_types.cuh"

namespace fluxbin {

constexpr int kQuantQuant = 0, kQuantSilu = 1, kQuantNorm = 2;

struct QuantArgs {
    const void* a;        // x, gate or h: [T][lda]
    const void* b;        // up, or delta (NULL: none): [T][ldb]
    const void* gamma;    // rmsnorm: [N]
    void* h_out;          // rmsnorm: [T][ldo] or NULL
    int8_t* q;            // [T][ldq]
    float* scale;         // [T]
    int64_t lda, ldb, ldo, ldq;
    int32_t T, N;
    float eps;
};

// 8 consecutive elements at a 16-byte boundary.
template <typename T>
struct alignas(16) Vec8 {
    T v[8];
};

// Element j of a thread's chunk i: 8 consecutive elements (VEC), or elements
// one row of threads apart.
template <bool VEC>
__device__ __forceinline__ int quant_index(int i, int j, int tpr) {
    return VEC ? (i * tpr + (int)threadIdx.x) * 8 + j : (i * 8 + j) * tpr + (int)threadIdx.x;
}

template <bool VEC, typename T>
__device__ __forceinline__ void quant_load(const T* row, int i, int tpr, int N, float (&f)[8]) {
    if constexpr (VEC) {
        const int n = quant_index<true>(i, 0, tpr);
        Vec8<T> x;
        if (n < N) {
            x = *reinterpret_cast<const Vec8<T>*>(row + n);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x.v[j] = from_f32<T>(0.f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = to_f32(x.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = quant_index<false>(i, j, tpr);
            f[j] = n < N ? to_f32(row[n]) : 0.f;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void quant_store(T* row, int i, int tpr, int N, const float (&f)[8]) {
    if constexpr (VEC) {
        const int n = quant_index<true>(i, 0, tpr);
        Vec8<T> x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x.v[j] = from_f32<T>(f[j]);
        if (n < N) *reinterpret_cast<Vec8<T>*>(row + n) = x;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = quant_index<false>(i, j, tpr);
            if (n < N) row[n] = from_f32<T>(f[j]);
        }
    }
}

__device__ __forceinline__ float silu_mul(float g, float u) {
    // exp(-g) overflows to infinity below g = -88 and its reciprocal is then
    // 0: silu's own limit.  The approximate exponential and reciprocal are
    // within a few 2^-23 of the value, far below half a step of 8 bits.
    float rc;
    asm("rcp.approx.f32 %0, %1;" : "=f"(rc) : "f"(1.f + __expf(-g)));
    return g * rc * u;
}

// The row's values before the common factor (chunk i).  rmsnorm: adds the
// residual, writes h' (FIRST) and sums its squares; a second pass reads h'
// back when it was written (h_out may be h itself).
template <int KIND, typename E, typename H, bool VEC, bool FIRST>
__device__ __forceinline__ void quant_values(const QuantArgs& p, int64_t t, int i, int tpr, float (&f)[8], float& ss) {
    if constexpr (KIND == kQuantQuant) {
        quant_load<VEC>(static_cast<const E*>(p.a) + t * p.lda, i, tpr, p.N, f);
    } else if constexpr (KIND == kQuantSilu) {
        float u[8];
        quant_load<VEC>(static_cast<const E*>(p.a) + t * p.lda, i, tpr, p.N, f);
        quant_load<VEC>(static_cast<const E*>(p.b) + t * p.ldb, i, tpr, p.N, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = silu_mul(f[j], u[j]);
    } else {
        float g[8];
        if (FIRST || !p.h_out) {
            quant_load<VEC>(static_cast<const H*>(p.a) + t * p.lda, i, tpr, p.N, f);
            if (p.b) {
                float d[8];
                quant_load<VEC>(static_cast<const E*>(p.b) + t * p.ldb, i, tpr, p.N, d);
                // rounded once to the stream's own type: the norm and every
                // later reader of the stream see the same h'
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = to_f32(from_f32<H>(f[j] + d[j]));
            }
            if (FIRST && p.h_out) quant_store<VEC>(static_cast<H*>(p.h_out) + t * p.ldo, i, tpr, p.N, f);
        } else {
            quant_load<VEC>(static_cast<const H*>(p.h_out) + t * p.ldo, i, tpr, p.N, f);
        }
        quant_load<VEC>(static_cast<const E*>(p.gamma), i, tpr, p.N, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (FIRST) ss = fmaf(f[j], f[j], ss);
            f[j] *= g[j];
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void quant_codes(const QuantArgs& p, int64_t t, int i, int tpr, const float (&f)[8],
                                            float pre, float inv) {
    int8_t* row = p.q + t * p.ldq;
    int c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = max(-127, min(127, __float2int_rn(f[j] * pre * inv)));
    if constexpr (VEC) {
        const int n = quant_index<true>(i, 0, tpr);
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = (uint32_t)(c[4 * k] & 255) | ((uint32_t)(c[4 * k + 1] & 255) << 8) |
                   ((uint32_t)(c[4 * k + 2] & 255) << 16) | ((uint32_t)(c[4 * k + 3] & 255) << 24);
        if (n < p.N) *reinterpret_cast<uint2*>(row + n) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = quant_index<false>(i, j, tpr);
            if (n < p.N) row[n] = (int8_t)c[j];
        }
    }
}

// blockDim = (threads of a row, rows of the CTA); threads of a row a multiple of 32.
template <int KIND, typename E, typename H, int VPT, bool VEC>
__global__ void fluxbin_quant_kernel(const QuantArgs p) {
    __shared__ float s_sum[32];
    __shared__ unsigned int s_max[32];
    const int tpr = (int)blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool live = t < p.T;

    float ss = 0.f;
    unsigned int mx = 0u;
    float f[VPT ? VPT : 1][8];
    const int chunks = (p.N + 8 * tpr - 1) / (8 * tpr);
    if (live) {
        if constexpr (VPT > 0) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                quant_values<KIND, E, H, VEC, true>(p, t, i, tpr, f[i], ss);
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(f[i][j]) & 0x7fffffffu);
            }
        } else {
            for (int i = 0; i < chunks; ++i) {
                quant_values<KIND, E, H, VEC, true>(p, t, i, tpr, f[0], ss);
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(f[0][j]) & 0x7fffffffu);
            }
        }
    }
    // the row's maximum and sum: within the warps, then over the row's warps
    // (the same order in every thread)
    mx = __reduce_max_sync(0xffffffffu, mx);
    if constexpr (KIND == kQuantNorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const int wpr = tpr / 32;
    if (wpr > 1) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, w0 = (int)threadIdx.y * wpr;
        if (lane == 0) {
            s_max[w0 + w] = mx;
            s_sum[w0 + w] = ss;
        }
        __syncthreads();
        mx = __reduce_max_sync(0xffffffffu, lane < wpr ? s_max[w0 + lane] : 0u);
        if constexpr (KIND == kQuantNorm) {
            ss = lane < wpr ? s_sum[w0 + lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
    }
    if (!live) return;
    const float amax = __uint_as_float(mx);
    float factor = 1.f;
    if constexpr (KIND == kQuantNorm) {
        factor = 1.f / sqrtf(ss / (float)p.N + p.eps);
        if (!(ss < INFINITY)) factor = NAN;
    }
    float s = amax * factor / 127.f;
    const bool finite = fabsf(s) < INFINITY;
    if (!finite) s = NAN;
    if (threadIdx.x == 0) p.scale[t] = s;
    // 127 / amax, the row scaled up first where the quotient would overflow
    const float pre = amax < 0x1p-100f ? 0x1p100f : 1.f;
    const float inv = (finite && mx != 0u) ? 127.f / (amax * pre) : 0.f;
    if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!finite) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = 0.f;   // a NaN or infinite value has no code
            }
            quant_codes<VEC>(p, t, i, tpr, f[i], pre, inv);
        }
    } else {
        for (int i = 0; i < chunks; ++i) {
            quant_values<KIND, E, H, VEC, false>(p, t, i, tpr, f[0], ss);
            if (!finite) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[0][j] = 0.f;
            }
            quant_codes<VEC>(p, t, i, tpr, f[0], pre, inv);
        }
    }
}

}  // namespace fluxbin
