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
// Bound: memory (one read of each input, one write of each output).  A row
// stays in its threads' registers between the reductions and the codes: VPT
// vectors of 8 consecutive elements a thread, blockDim.x threads a CTA and,
// for rows that one CTA does not hold, the CTAs of a cluster, which exchange
// their maxima and sums through distributed shared memory.  Rows that start
// off a 16-byte boundary are read with aligned 16-byte loads that are shifted
// into place, and written with 16-byte stores put together from two
// neighbouring threads' elements (an SM gets a store away every 13 to 20
// clocks, however narrow it is); only the ends of such a row go element by
// element.
// A CTA also asks L2 for the inputs of a row that will start later, so that
// memory stays busy while the resident CTAs compute and store.
// Measured (B200, a graph of calls on rotated inputs): norm with residual
// 2048x8192 fp16 20 us, 89% of the measured copy rate, 2047x4099 22 (41%);
// quant 4096x8192 17.0 (91%), 4096x8191 33 (47%); gate 2048x11008 22.3 (78%),
// 2048x28672 52 (87%), 2048x28671 100 (45%).
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
    int32_t parts;        // CTAs (of one cluster) that share a row
    int32_t ahead;        // rows from here to the one whose inputs this CTA asks L2 for (0: none)
};

// --- pairs of fp32 (one instruction for both) -------------------------------

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max_abs(float m, uint64_t ab) {
    const float2 f = unpair(ab);
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(f.x)), "f"(fabsf(f.y)));
    return r;
}

// --- eight elements of a row ------------------------------------------------

// Their bits, two 16-bit values or one fp32 a word.
template <typename T>
struct Raw {
    static constexpr int kWords = 8 * sizeof(T) / 4;
    uint32_t w[kWords];
};

// Elements n .. n+7 of a row of N (zeros past its end).  VEC: the row's
// length is a multiple of 8 and it starts at a 16-byte boundary.
template <bool VEC, typename T>
__device__ __forceinline__ Raw<T> quant_load(const T* row, int n, int N) {
    constexpr int U = Raw<T>::kWords / 4;                       // 16-byte units of the eight elements
    Raw<T> x;
    if constexpr (VEC) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (n < N) v = reinterpret_cast<const uint4*>(row + n)[u];
            put(x.w + 4 * u, v);
        }
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + n);
        const uint32_t off = (uint32_t)at & 15u;                // the same for the whole row
        const int before = (int)(off / sizeof(T)), after = off ? (int)((16u - off) / sizeof(T)) : 0;
        if (n >= before && n + 8 + after <= N) {
            // whole aligned units, all of them within the row
            const uint4* from = reinterpret_cast<const uint4*>(at - off);
            uint32_t w[4 * U + 4];
#pragma unroll
            for (int u = 0; u < U; ++u) put(w + 4 * u, from[u]);
            put(w + 4 * U, off ? from[U] : make_uint4(0, 0, 0, 0));
            put(x.w, shifted<0>(w, off));
            if constexpr (U == 2) put(x.w + 4, shifted<4>(w, off));
        } else {
            uint32_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = 0u;
                if (n + j < N) {
                    if constexpr (U == 1) e[j] = *reinterpret_cast<const unsigned short*>(row + n + j);
                    else e[j] = *reinterpret_cast<const uint32_t*>(row + n + j);
                }
            }
#pragma unroll
            for (int k = 0; k < 4 * U; ++k)
                x.w[k] = U == 1 ? __byte_perm(e[(2 * k) % 8], e[(2 * k + 1) % 8], 0x5410) : e[k % 8];
        }
    }
    return x;
}

template <typename T>
__device__ __forceinline__ void put_element(T* at, const Raw<T>& x, int j) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<unsigned short*>(at) = (unsigned short)(x.w[j / 2] >> (16 * (j % 2)));
    else *reinterpret_cast<uint32_t*>(at) = x.w[j % Raw<T>::kWords];
}

// Writes them.  All 32 lanes take part: lane l has the eight elements after
// lane l-1's.
template <bool VEC, typename T>
__device__ __forceinline__ void quant_store(T* row, int n, int N, const Raw<T>& x) {
    constexpr int U = Raw<T>::kWords / 4;
    if constexpr (VEC) {
        if (n < N) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                reinterpret_cast<uint4*>(row + n)[u] =
                    make_uint4(x.w[4 * u], x.w[4 * u + 1], x.w[4 * u + 2], x.w[4 * u + 3]);
        }
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + n);
        const uint32_t off = (uint32_t)at & 15u;
        uint32_t w[4 * U + 4];                                  // own words, then the next lane's first unit
#pragma unroll
        for (int k = 0; k < 4 * U; ++k) w[k] = x.w[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * U + k] = __shfl_down_sync(0xffffffffu, x.w[k], 1);
        const int lane = threadIdx.x & 31;
        if (off == 0u) {
            if (n + 8 <= N) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    reinterpret_cast<uint4*>(at)[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n + j < N) put_element(row + n + j, x, j);
            }
            return;
        }
        // aligned units from 16 - off bytes into the own elements on; the
        // last one ends with the next lane's first `head` elements
        const int head = (int)((16u - off) / sizeof(T));
        uint4* to = reinterpret_cast<uint4*>(at + 16u - off);
        const bool join = lane < 31 && n + 8 + head <= N;
        if constexpr (U == 2) {
            if (n + 8 <= N) to[0] = shifted<0>(w, 16u - off);
        }
        if (join) to[U - 1] = shifted<4 * U - 4>(w, 16u - off);
        // what no unit covers: the head where the lane before has not joined
        // it, the rest where this lane has not joined
        const bool own_head = lane == 0 || n + head > N;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int per = (int)(16 / sizeof(T));              // elements of a unit
            const bool in_head = j < head;
            const bool in_first = U == 2 && !in_head && j < head + per && n + 8 <= N;
            const bool covered = in_head ? !own_head : (in_first || join);
            if (!covered && n + j < N) put_element(row + n + j, x, j);
        }
    }
}

// Two elements as fp32.
__device__ __forceinline__ uint64_t widen(const Raw<__half>& x, int k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x.w[k]));
    return pair(f.x, f.y);
}
__device__ __forceinline__ uint64_t widen(const Raw<__nv_bfloat16>& x, int k) {
    return pair(__uint_as_float(x.w[k] << 16), __uint_as_float(x.w[k] & 0xffff0000u));
}
__device__ __forceinline__ uint64_t widen(const Raw<float>& x, int k) {
    return pair(__uint_as_float(x.w[2 * k]), __uint_as_float(x.w[2 * k + 1]));
}

// h + delta rounded once to h's type: the norm and every later reader of the
// stream see the same h'.  (The 16-bit additions round the exact sum.)
__device__ __forceinline__ void add_delta(Raw<__half>& h, const Raw<__half>& d) {
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("add.rn.f16x2 %0, %0, %1;" : "+r"(h.w[k]) : "r"(d.w[k]));
}
__device__ __forceinline__ void add_delta(Raw<__nv_bfloat16>& h, const Raw<__nv_bfloat16>& d) {
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(h.w[k]) : "r"(d.w[k]));
}
template <typename E>
__device__ __forceinline__ void add_delta(Raw<float>& h, const Raw<E>& d) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpair(add2(widen(h, k), widen(d, k)));
        h.w[2 * k] = __float_as_uint(f.x);
        h.w[2 * k + 1] = __float_as_uint(f.y);
    }
}

// g / (1 + exp(-g)) of two gates, as g/4 divided by (1 + exp(-g)) / 4: the
// approximate reciprocal gives 0 from 2^126 on, so that without the factor gates
// below -87.33 would be lost, with it those below -88.72, where exp(-g) itself
// leaves fp32 and the value is 0.  (g/4 is exact: a bf16 has no bit below 2^-133.)
// The exponent's constant and product are rounded, which the exponential turns
// into a relative error of up to |g| units of 2^-23; the approximate
// exponential, the sum, the reciprocal and the product add a few: below 100
// units, 2^-16, and half a step of 8 bits is 2^-8 of the row's maximum.
// Flushing subnormals saves the instructions that would scale them.
__device__ __forceinline__ uint64_t silu(uint64_t g) {
    const uint64_t quarter = pair(0.25f, 0.25f);
    const float2 x = unpair(mul2(g, pair(-1.4426950408889634f, -1.4426950408889634f)));
    float2 e, rc;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    const float2 s = unpair(fma2(pair(e.x, e.y), quarter, quarter));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc.x) : "f"(s.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc.y) : "f"(s.y));
    return mul2(mul2(g, quarter), pair(rc.x, rc.y));
}

// A chunk's inputs.
template <int KIND, typename E, typename H>
struct QuantIn {
    Raw<H> a;
    Raw<E> b;
};

template <int KIND, typename E, typename H, bool VEC>
__device__ __forceinline__ void quant_inputs(const QuantArgs& p, int64_t t, int n, QuantIn<KIND, E, H>& x) {
    x.a = quant_load<VEC>(static_cast<const H*>(p.a) + t * p.lda, n, p.N);
    if (KIND == kQuantSilu || (KIND == kQuantNorm && p.b))
        x.b = quant_load<VEC>(static_cast<const E*>(p.b) + t * p.ldb, n, p.N);
}

// Asks L2 for elements n .. n+count-1 of a row of N, as far as they are whole
// 16-byte units.
template <typename T>
__device__ __forceinline__ void quant_prefetch(const T* row, int n, int count, int N) {
    const int c = min(count, N - n);
    if (c <= 0) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + n), from = (at + 15u) & ~(uintptr_t)15u;
    const uintptr_t end = (at + (uintptr_t)c * sizeof(T)) & ~(uintptr_t)15u;
    if (from < end)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(end - from)) : "memory");
}

// Asks for the inputs of the row `ahead` rows on, which a CTA that has not
// started yet will read (one thread).
template <int KIND, typename E, typename H>
__device__ __forceinline__ void quant_prefetch_ahead(const QuantArgs& p, int64_t t, int n, int count) {
    if (threadIdx.x != 0 || p.ahead == 0 || t + p.ahead >= p.T) return;
    t += p.ahead;
    quant_prefetch(static_cast<const H*>(p.a) + t * p.lda, n, count, p.N);
    if (KIND == kQuantSilu || (KIND == kQuantNorm && p.b))
        quant_prefetch(static_cast<const E*>(p.b) + t * p.ldb, n, count, p.N);
}

// The row's values before its common factor; their largest magnitude, and for
// rmsnorm h' (written) and the sum of its squares.
template <int KIND, typename E, typename H, bool VEC>
__device__ __forceinline__ void quant_values(const QuantArgs& p, int64_t t, int n, QuantIn<KIND, E, H>& x,
                                             uint64_t (&v)[4], uint64_t& ss, float& mx) {
    if constexpr (KIND == kQuantNorm) {
        const Raw<E> g = quant_load<VEC>(static_cast<const E*>(p.gamma), n, p.N);
        if (p.b) add_delta(x.a, x.b);
        if (p.h_out) quant_store<VEC>(static_cast<H*>(p.h_out) + t * p.ldo, n, p.N, x.a);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t h = widen(x.a, k);
            ss = fma2(h, h, ss);
            v[k] = mul2(h, widen(g, k));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = widen(x.a, k);
            if constexpr (KIND == kQuantSilu) v[k] = mul2(silu(v[k]), widen(x.b, k));
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) mx = max_abs(mx, v[k]);
}

// A row's scale, from the bits of its largest magnitude and its common factor.
struct QuantScale {
    float s, pre, inv;
    bool finite;
};
__device__ __forceinline__ QuantScale quant_scale(unsigned int mx, float factor) {
    const float amax = __uint_as_float(mx);
    QuantScale c;
    c.s = amax * factor / 127.f;
    c.finite = fabsf(c.s) < INFINITY;
    if (!c.finite) c.s = NAN;
    // 127 / amax, the row scaled up first where the quotient would overflow
    c.pre = amax < 0x1p-100f ? 0x1p100f : 1.f;
    c.inv = (c.finite && mx != 0u) ? 127.f / (amax * c.pre) : 0.f;
    return c;
}

// Codes of a chunk: v * pre * inv is at most 127 (1 + 2^-22) in magnitude, so
// adding 1.5 * 2^23 rounds it to the nearest integer (ties to even) and leaves
// that integer, modulo 2^8, in the low byte.  (The addition is a scalar one:
// a paired multiplication and a paired addition were seen to be contracted
// into one rounding, which moves ties.)
__device__ __forceinline__ void quant_codes(const QuantArgs& p, int64_t t, int n, uint64_t (&v)[4], float pre,
                                            float inv, bool finite) {
    const uint64_t inv2 = pair(inv, inv);
    constexpr float kMagic = 12582912.f;
    if (pre != 1.f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], pair(pre, pre));
    }
    uint32_t c[4];   // two codes each, in the low bytes
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpair(mul2(v[k], inv2));
        c[k] = __byte_perm(__float_as_uint(__fadd_rn(f.x, kMagic)), __float_as_uint(__fadd_rn(f.y, kMagic)), 0x0040);
    }
    uint32_t w[2] = {__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410)};
    if (!finite) w[0] = w[1] = 0u;   // a NaN or an infinity has no code
    int8_t* at = p.q + t * p.ldq + n;
    if (n + 8 <= p.N) {
        *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (n + j < p.N) at[j] = (int8_t)(w[j / 4] >> (8 * (j % 4)));
    }
}

// Threads that a CTA of the kernel with VPT chunks a thread may have (what its
// registers allow).
__host__ __device__ constexpr int quant_max_threads(int vpt) { return vpt <= 1 ? 1024 : vpt == 2 ? 768 : 512; }

constexpr int kGateMaxThreads = 1024, kGateMaxVpt = 4;
constexpr int kGateMaxSmem = 226 * 1024;   // two rows of both inputs
constexpr int kQuantMaxParts = 8;   // a portable cluster: 8 * 512 threads * 4 * 8 elements hold the longest row

// blockDim = (threads of a row, rows of the CTA); threads of a row a multiple
// of 32; one row per cluster where p.parts > 1.  (Named one CTA per SM as the
// least, the compiler gives the plain quantiser a few registers more: 4096x8192
// 19.7 -> 18.9 us; the norm lost by it, 21.1 -> 22.2.)
template <int KIND, typename E, typename H, int VPT, bool VEC>
__global__ void __launch_bounds__(quant_max_threads(VPT), KIND == kQuantQuant ? 1 : 0)
    fluxbin_quant_kernel(const QuantArgs p) {
    __shared__ float s_sum[32];
    __shared__ unsigned int s_max[32];
    __shared__ float s_part_sum[kQuantMaxParts];
    __shared__ unsigned int s_part_max[kQuantMaxParts];
    const int tpr = (int)blockDim.x, parts = p.parts;
    const int rank = (int)(blockIdx.x % (unsigned)parts);
    const int64_t t = (int64_t)(blockIdx.x / (unsigned)parts) * blockDim.y + threadIdx.y;
    const int n0 = (rank * VPT * tpr + (int)threadIdx.x) * 8;   // chunk i at n0 + 8 i tpr
    asm volatile("griddepcontrol.launch_dependents;");
    // the others of the cluster have started once this barrier is passed (below)
    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool live = t < p.T;

    uint64_t ss2 = 0ull;
    float mxf = 0.f;
    uint64_t v[VPT][4];
    if (live) {
        // what is asked for ahead comes after the own loads, but in the gate
        // before them: there it costs registers after them (2048x28672 63.8
        // against 66.5 us; norm of a 32-bit 2048x8192 31.4 against 30.4)
        if (KIND == kQuantSilu) quant_prefetch_ahead<KIND, E, H>(p, t, n0, 8 * VPT * tpr);
        // every load before the first store
        QuantIn<KIND, E, H> x[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) quant_inputs<KIND, E, H, VEC>(p, t, n0 + 8 * i * tpr, x[i]);
        if (KIND != kQuantSilu) quant_prefetch_ahead<KIND, E, H>(p, t, n0, 8 * VPT * tpr);
#pragma unroll
        for (int i = 0; i < VPT; ++i) quant_values<KIND, E, H, VEC>(p, t, n0 + 8 * i * tpr, x[i], v[i], ss2, mxf);
    }
    float ss = unpair(ss2).x + unpair(ss2).y;
    // the row's maximum and sum: within the warps, over the CTA's warps, over
    // the cluster's CTAs (the same order in every thread)
    unsigned int mx = __reduce_max_sync(0xffffffffu, __float_as_uint(mxf) & 0x7fffffffu);
    if constexpr (KIND == kQuantNorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const int wpr = tpr / 32, lane = threadIdx.x & 31;
    if (wpr > 1) {
        const int w = threadIdx.x >> 5, w0 = (int)threadIdx.y * wpr;
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
    if (parts > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if ((int)threadIdx.x < parts) {
            uint32_t am, as;
            asm("mapa.shared::cluster.u32 %0, %1, %2;"
                : "=r"(am) : "r"((uint32_t)__cvta_generic_to_shared(s_part_max + rank)), "r"((int)threadIdx.x));
            asm("mapa.shared::cluster.u32 %0, %1, %2;"
                : "=r"(as) : "r"((uint32_t)__cvta_generic_to_shared(s_part_sum + rank)), "r"((int)threadIdx.x));
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(am), "r"(mx) : "memory");
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(as), "r"(__float_as_uint(ss)) : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        ss = 0.f;
        for (int r = 0; r < parts; ++r) {
            mx = max(mx, s_part_max[r]);
            ss += s_part_sum[r];
        }
    }
    if (!live) return;
    float factor = 1.f;
    if constexpr (KIND == kQuantNorm) {
        factor = 1.f / sqrtf(ss / (float)p.N + p.eps);
        if (!(ss < INFINITY)) factor = NAN;
    }
    const QuantScale c = quant_scale(mx, factor);
    if (threadIdx.x == 0 && rank == 0) p.scale[t] = c.s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) quant_codes(p, t, n0 + 8 * i * tpr, v[i], c.pre, c.inv, c.finite);
}

// The gate for many rows: a CTA takes every gridDim.x-th row, and copies the
// next one into shared memory while it works on the current one, so that memory
// does not wait for the exponentials and the stores (2048x28672 64 -> 52 us, of
// 45 that memory takes; the exponential's and the reciprocal's unit is busy for
// 26).  Each thread copies what it
// reads itself (no barrier but the reduction's); the buffer that it copies into
// was read a row ago, before that row's reduction.
template <typename E, int VPT>
__global__ void __launch_bounds__(kGateMaxThreads, 1) fluxbin_gate_rows_kernel(const QuantArgs p) {
    extern __shared__ __align__(16) uint4 gate_rows[];          // [2][gate, up][N / 8]
    __shared__ unsigned int s_max[2][32];
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31, vecs = p.N / 8;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const auto request = [&](int64_t t, int s) {
        if (t < p.T) {
            const E* g = static_cast<const E*>(p.a) + t * p.lda;
            const E* u = static_cast<const E*>(p.b) + t * p.ldb;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i * nt + tid;
                if (c < vecs) {
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(gate_rows + 2 * s * vecs + c);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(g + 8 * c) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * vecs), "l"(u + 8 * c) : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int64_t t = blockIdx.x;
    int s = 0;
    request(t, s);
    for (; t < p.T; t += gridDim.x, s ^= 1) {
        request(t + gridDim.x, s ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const uint4* in = gate_rows + 2 * s * vecs;
        uint64_t v[VPT][4], ss = 0ull;
        float mxf = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            QuantIn<kQuantSilu, E, E> x;
            const int c = i * nt + tid;
            put(x.a.w, c < vecs ? in[c] : make_uint4(0, 0, 0, 0));
            put(x.b.w, c < vecs ? in[vecs + c] : make_uint4(0, 0, 0, 0));
            quant_values<kQuantSilu, E, E, true>(p, t, 0, x, v[i], ss, mxf);
        }
        unsigned int mx = __reduce_max_sync(0xffffffffu, __float_as_uint(mxf) & 0x7fffffffu);
        if (lane == 0) s_max[s][tid >> 5] = mx;
        __syncthreads();
        mx = __reduce_max_sync(0xffffffffu, lane < nt / 32 ? s_max[s][lane] : 0u);
        const QuantScale c = quant_scale(mx, 1.f);
        if (tid == 0) p.scale[t] = c.s;
#pragma unroll
        for (int i = 0; i < VPT; ++i) quant_codes(p, t, (i * nt + tid) * 8, v[i], c.pre, c.inv, c.finite);
    }
}

}  // namespace fluxbin
