// The 8-bit integer product for a few tokens and a layer that one wave of the
// GPU holds (sm_100a).
//
// Such a call is over in a few microseconds, most of them latency: there is
// no time to set up a ring, tensor memory and a cluster.  A CTA owns 16
// channels and streams them straight into registers; its 8 warps take the
// 64-byte segments of K in turn, so that together they read 512 contiguous
// bytes of a row at a time, and add their sums through shared memory.
//
// The products run on mma.sync (m16n8k32, 32-bit integer sums): the 16
// channels are its rows, 8 tokens (of up to 16: NT = 2) its columns.  Its operands leave the
// order of K free as long as both agree, so a lane takes 16 consecutive codes
// of a row (one 16-byte load) as the codes of two instructions.  The tensor
// rate does not matter here: 2 instructions per KB of weights.
//
// Bound: latency (1x4096x4096 3.8 us, 67% of the measured copy rate, with
// FLUXBIN_FLAG_EARLY_WEIGHTS; 4.7 without).  Eight segments in flight a warp and
// eight warps: four segments 4.6 to 5.2, four warps 5.2.
#pragma once

#include "fluxbin_int8.cuh"

namespace fluxbin {

constexpr int kMvRows = 16, kMvWarps = 8, kMvTokens = 8;   // tokens of one instruction
constexpr int kMvSegment = 64;           // codes of K a warp takes at a time
constexpr int kMvBatch = 8;              // segments in flight per warp

// 16 codes from n on of a row of N (zeros past its end, whose bytes are not
// read).  STREAM: read once, so not kept in L1; not an invariant load, for the
// preceding kernel may have written the row after this one started.
template <bool STREAM>
__device__ __forceinline__ uint4 mv_load(const int8_t* row, int n, int N) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n + 16 <= N) {
        if (STREAM)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(row + n) : "memory");
        else
            v = *reinterpret_cast<const uint4*>(row + n);
    } else if (n < N) {
        // whole words, then the bytes of the last one (every load before its use)
        uint32_t w[4], b[3];
        const int words = (N - n) / 4, bytes = (N - n) % 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = k < words ? *reinterpret_cast<const uint32_t*>(row + n + 4 * k) : 0u;
#pragma unroll
        for (int k = 0; k < 3; ++k) b[k] = k < bytes ? (uint32_t)(uint8_t)row[n + 4 * words + k] : 0u;
        const uint32_t last = b[0] | (b[1] << 8) | (b[2] << 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] |= k == words ? last : 0u;
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

__device__ __forceinline__ void mv_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename Y, bool ACC, int NT>
__global__ void __launch_bounds__(32 * kMvWarps, 2) fluxbin_int8_mv_kernel(const Int8Args p) {
    __shared__ int part[kMvWarps][NT * kMvTokens][kMvRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;         // row (and row + 8) or token; 16 codes of a segment
    const int m0 = blockIdx.x * kMvRows;
    asm volatile("griddepcontrol.launch_dependents;");
    const bool early = (p.flags & kInt8Early) != 0;
    // rows past the last one repeat it; their sums are not written
    const int8_t* w0 = p.w + (int64_t)min(m0 + g, p.M - 1) * p.ldw;
    const int8_t* w1 = p.w + (int64_t)min(m0 + g + 8, p.M - 1) * p.ldw;
    if (!early) {
        // into L2 only: that may run ahead of the preceding kernel even if
        // that one writes the weights
        if (q == 0) {
#pragma unroll
            for (int i = 0; i < kMvBatch; ++i) {
                const int n = (warp + i * kMvWarps) * kMvSegment;
                if (n < p.N) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 + n));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 + n));
                }
            }
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    const int segments = (p.N + kMvSegment - 1) / kMvSegment;

    int c[NT][4] = {};
    bool waited = !early;
    for (int s0 = warp; s0 < segments; s0 += kMvWarps * kMvBatch) {
        uint4 a[kMvBatch], b[kMvBatch];
#pragma unroll
        for (int i = 0; i < kMvBatch; ++i) {
            const int n = (s0 + i * kMvWarps) * kMvSegment + 16 * q;
            a[i] = mv_load<true>(w0, n, p.N);
            b[i] = mv_load<true>(w1, n, p.N);
        }
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
        }
#pragma unroll
        for (int h = 0; h < NT; ++h) {
            const int t = h * kMvTokens + g;
            const int8_t* x0 = p.x + (int64_t)min(t, p.T - 1) * p.ldx;
            uint4 x[kMvBatch];
#pragma unroll
            for (int i = 0; i < kMvBatch; ++i) {
                const int n = (s0 + i * kMvWarps) * kMvSegment + 16 * q;
                x[i] = t < p.T ? mv_load<false>(x0, n, p.N) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kMvBatch; ++i) {
                mv_mma(c[h], a[i].x, b[i].x, a[i].y, b[i].y, x[i].x, x[i].y);
                mv_mma(c[h], a[i].z, b[i].z, a[i].w, b[i].w, x[i].z, x[i].w);
            }
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    // sums: rows g and g + 8, tokens 2 q and 2 q + 1 of every eight
#pragma unroll
    for (int h = 0; h < NT; ++h) {
        int(*to)[kMvRows] = &part[warp][h * kMvTokens + 2 * q];
        to[0][g] = c[h][0];
        to[1][g] = c[h][1];
        to[0][g + 8] = c[h][2];
        to[1][g + 8] = c[h][3];
    }
    __syncthreads();
    const int t = tid / kMvRows, m = m0 + tid % kMvRows;
    if (t >= p.T || m >= p.M) return;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kMvWarps; ++w) sum += part[w][t][tid % kMvRows];
    Y* y = static_cast<Y*>(p.y) + t * p.ldy + m;
    const float v = int8_value(sum, p.sx[t], p.sw[m]);
    *y = from_f32<Y>(ACC ? to_f32(*y) + v : v);
}

}  // namespace fluxbin
