// The 8-bit integer product on the fifth-generation tensor cores (sm_100a).
//
//   acc[m][t] = sum_n wq[m][n] xq[t][n],  y[t][m] (+)= acc * (sx[t] * sw[m])
//
// The weights are the matrix instruction's A operand (128 channels a tile,
// along the tensor memory's lanes) and the tokens its B operand: a tile of `bn`
// tokens, a multiple of 16 up to 256, fits the batch at hand without wasting
// operand loads on padding.  Both are K-major rows of codes,
// copied by TMA with the 128-byte swizzle, 128 codes of K a stage; rows and
// codes beyond the arrays' ends arrive as zeros.
//
// Split of K: with few tiles the stages of a tile are shared out over the
// CTAs of a cluster.  Every CTA leaves its partial sums in its own shared
// memory, and each then adds its share of the tokens over all of them through
// distributed shared memory: integer sums, so the split changes no bit.  (That
// memory yields 8 to 16 bytes per clock and SM: 2.5 us of 333x4096x11008's 18.
// Sending the sums with st.async instead took longer, 21.)  A CTA releases its tensor memory before it waits for the others (none holds
// tensor memory while it waits for one that may be waiting for some).
//
// Roles: one thread of warp 0 issues the copies, one of warp 1 the matrix
// instructions; a ring of stages with full and empty mbarriers lies between
// them.  All eight warps then empty the accumulators.  Every wait is bounded:
// one that gives up sets bit 0 of the device error word, and the CTA's sums
// are replaced by NaN outputs.
//
// Bound: for few tokens by HBM (1x28672x8192 38.0 us, 95% of the measured copy
// rate), below that by the latency of one wave and the clusters' meeting
// (128x4096x4096 9.0 us), then by the products (333x4096x11008: a stage takes
// 460 clocks, 352 of them products).
#pragma once

#include <cuda.h>

#include "fluxbin_int8.cuh"
#include "fluxbin_tc.cuh"

namespace fluxbin {

constexpr int kI8Rows = 128;                     // channels of a tile
constexpr int kI8K = 128;                        // codes of K a stage (one swizzle row)
constexpr int kI8MaxBn = 256;
constexpr int kI8MaxStages = 12;
constexpr int kI8MaxSplits = 8;                  // a portable cluster
constexpr uint32_t kI8SpinLimit = 1u << 22;      // polls (each may suspend for microseconds) before a wait fails
constexpr uint32_t kI8TestSpinLimit = 64u;

struct Int8TcArgs {
    Int8Args p;
    int32_t bn;           // tokens of a tile
    int32_t kblocks;      // stages of K
    int32_t splits;       // CTAs (of one cluster) that share a tile
    int32_t stages;       // ring length
    int32_t tiles_t;      // token tiles
    uint32_t tmem_cols;
    uint32_t spin_limit;
    int32_t test_stall;   // test hook: no copy is issued
    int32_t bulk;         // y's rows can be written by TMA: 1 whole tiles, 2 a ragged last tile too
    unsigned int* err;
};

constexpr int kI8Threads = 256;
constexpr int kI8OutBox = 16;                    // tokens of y written by one bulk copy
// Token scales behind the barriers, then the ring (1024-byte atoms).
constexpr int kI8SxOff = 1024;
constexpr int kI8RingOff = 2048;
__host__ __device__ constexpr int int8_stage_bytes(int bn) { return kI8Rows * kI8K + bn * kI8K; }

// Instruction descriptor of the 8-bit integer kind: 32-bit integer
// accumulator, signed A and B, both K-major.
__device__ __forceinline__ uint32_t int8_idesc(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One thread of a converged warp, the same one every time.  A branch on it,
// unlike one on the lane number, is known to be taken by a single thread: the
// matrix instructions' descriptors then stay in uniform registers (the pair
// kernel at 4096 x 8192 x 8192: 305,000 -> 263,000 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void int8_mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}

__device__ __forceinline__ void int8_tma(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// The same box into L2 only.  L2 is where all writes meet: a prefetch may run
// ahead of the preceding kernel even if that one writes the weights.
__device__ __forceinline__ void int8_prefetch(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void int8_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void int8_ld16(uint32_t taddr, int (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ void int8_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t dsmem_addr(uint32_t addr, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ int ld_dsmem(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int4 ld_dsmem4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Four consecutive channels m .. m+3 (fewer at the end of M) of token t.
template <typename Y, bool ACC>
__device__ __forceinline__ void int8_store4(const Int8Args& p, int64_t t, int m, float sx, const float (&sw)[4],
                                            const int4& acc, bool ok) {
    Y* y = static_cast<Y*>(p.y) + t * p.ldy + m;
    const int n = p.M - m < 4 ? p.M - m : 4;
    const int v4[4] = {acc.x, acc.y, acc.z, acc.w};
    struct alignas(4 * sizeof(Y)) Quad { Y v[4]; } o;
    const bool vec = p.vec4 && n == 4;
    if (ACC) {
        if (vec) {
            o = *reinterpret_cast<const Quad*>(y);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[i] = i < n ? y[i] : from_f32<Y>(0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = int8_value(v4[i], sx, sw[i]);
        if (!ok) v = __int_as_float(0x7fc00000);
        if (ACC) v += to_f32(o.v[i]);
        o.v[i] = from_f32<Y>(v);
    }
    if (vec) {
        *reinterpret_cast<Quad*>(y) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) y[i] = o.v[i];
    }
}

// `rows` tokens of a tile of y, [rows][128 channels] of Y at byte offset `buf`
// of the shared memory, out to y (tokens from t0, channels from m0 on) or in
// from it, by THREADS threads (e: this one's number): 16 bytes a lane, the
// pieces of rows that start off a 16-byte boundary shifted into place, the ends
// of a row element by element; U rows of a thread at a time, every load before
// the first store.
template <typename Y, int THREADS, int U>
__device__ __forceinline__ void int8_rows_out(const Int8Args& p, uint32_t buf, int64_t t0, int rows, int m0, int e) {
    constexpr int kLanes = kI8Rows * (int)sizeof(Y) / 16, kPer = 16 / (int)sizeof(Y), kStep = THREADS / kLanes;
    const int l = e % kLanes, nv = p.M - m0 < kI8Rows ? p.M - m0 : kI8Rows;
    if (t0 + rows > p.T) rows = (int)(p.T - t0);
    for (int j0 = e / kLanes; j0 < rows; j0 += U * kStep) {
        uint4 piece[U];
        Y end[U];
        int end_at[U], piece_at[U];                                  // elements of the row, -1: none
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kStep;
            const Y* y = static_cast<const Y*>(p.y) + (t0 + j) * p.ldy + m0;
            const uint32_t row = buf + (uint32_t)(j * kI8Rows * (int)sizeof(Y));
            const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(y) & 15u;
            const int head = off ? (int)((16u - off) / sizeof(Y)) : 0;   // elements before the first boundary
            const int whole = nv > head ? (nv - head) / kPer : 0;        // pieces
            piece_at[u] = j < rows && l < whole ? head + l * kPer : -1;
            if (piece_at[u] >= 0) {
                uint32_t w[8];
                put(w, smem_at<const uint4>(row + 16u * l));
                put(w + 4, off ? smem_at<const uint4>(row + 16u * l + 16u) : make_uint4(0, 0, 0, 0));
                piece[u] = shifted<0>(w, off ? 16u - off : 0u);
            }
            const int el = l < head ? l : whole * kPer + l;              // what no piece covers: below 16 elements
            end_at[u] = j < rows && el < nv ? el : -1;
            if (end_at[u] >= 0) end[u] = smem_at<const Y>(row + (uint32_t)(el * (int)sizeof(Y)));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Y* y = static_cast<Y*>(p.y) + (t0 + j0 + u * kStep) * p.ldy + m0;
            if (piece_at[u] >= 0) *reinterpret_cast<uint4*>(y + piece_at[u]) = piece[u];
            if (end_at[u] >= 0) y[end_at[u]] = end[u];
        }
    }
}
template <typename Y, int THREADS, int U>
__device__ __forceinline__ void int8_rows_in(const Int8Args& p, uint32_t buf, int64_t t0, int rows, int m0, int e) {
    constexpr int kLanes = kI8Rows * (int)sizeof(Y) / 16, kPer = 16 / (int)sizeof(Y), kStep = THREADS / kLanes;
    const int l = e % kLanes, nv = p.M - m0 < kI8Rows ? p.M - m0 : kI8Rows;
    if (t0 + rows > p.T) rows = (int)(p.T - t0);
    for (int j0 = e / kLanes; j0 < rows; j0 += U * kStep) {
        uint4 lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kStep;
            const Y* y = static_cast<const Y*>(p.y) + (t0 + j) * p.ldy + m0 + l * kPer;
            const uintptr_t at = reinterpret_cast<uintptr_t>(y);
            const uint32_t off = (uint32_t)at & 15u;
            const int before = (int)(off / sizeof(Y)), after = off ? (int)((16u - off) / sizeof(Y)) : 0;
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (j < rows) {
                if (m0 + l * kPer >= before && m0 + (l + 1) * kPer + after <= p.M) {
                    lo[u] = *reinterpret_cast<const uint4*>(at - off);
                    if (off) hi[u] = *reinterpret_cast<const uint4*>(at - off + 16);
                } else {
                    // the ends of the row; put where the shift below takes them from
                    alignas(16) Y el[2 * kPer];
#pragma unroll
                    for (int k = 0; k < 2 * kPer; ++k) {
                        const int c = k - before;
                        el[k] = c >= 0 && c < kPer && l * kPer + c < nv ? y[c] : from_f32<Y>(0.f);
                    }
                    lo[u] = *reinterpret_cast<const uint4*>(el);
                    hi[u] = *reinterpret_cast<const uint4*>(el + kPer);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kStep;
            const Y* y = static_cast<const Y*>(p.y) + (t0 + j) * p.ldy + m0 + l * kPer;
            uint32_t w[8];
            put(w, lo[u]);
            put(w + 4, hi[u]);
            if (j < rows)
                smem_at<uint4>(buf + (uint32_t)(j * kI8Rows * (int)sizeof(Y)) + 16u * l) =
                    shifted<0>(w, (uint32_t)reinterpret_cast<uintptr_t>(y) & 15u);
        }
    }
}

// The 128 channels from m0 on of a token of y into L2, ahead of an accumulation.
template <typename Y>
__device__ __forceinline__ void int8_prefetch_row(const Int8Args& p, int64_t t, int m0) {
    const int n = (p.M - m0 < kI8Rows ? p.M - m0 : kI8Rows) * (int)sizeof(Y);
    const char* row = reinterpret_cast<const char*>(static_cast<const Y*>(p.y) + t * p.ldy + m0);
    for (int o = 0; o < n; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + o));
    if (n > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + n - 1));
}

__device__ __forceinline__ int4 add4(const int4& a, const int4& b) {
    return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Tokens c, c + 8, .. below c1 of a split tile: the sums of `splits` <= MAX
// CTAs, U tokens at a time, scaled and written.  Nothing read from another CTA
// is left unused, so all of it has arrived when this returns: the lanes past
// the end of M read from this CTA (`rank`).
template <typename Y, bool ACC, int MAX, int U>
__device__ __forceinline__ void int8_sum_split(const Int8Args& p, uint32_t ring, int splits, int rank, int64_t t0,
                                               int c, int c1, int m0, int mq, const float (&sw4)[4], int failed) {
    constexpr int kWarps = kI8Threads / 32;
    uint32_t peer[MAX];
#pragma unroll
    for (int r = 0; r < MAX; ++r) peer[r] = dsmem_addr(ring + (uint32_t)(mq * 4), r < splits && m0 + mq < p.M ? r : rank);
    for (; c < c1; c += U * kWarps) {
        int4 part[U][MAX];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < MAX; ++r)
                if (r < splits && c + u * kWarps < c1)
                    part[u][r] = ld_dsmem4(peer[r] + (uint32_t)((c + u * kWarps) * kI8Rows * 4));
        const bool ok = !__any_sync(0xffffffffu, failed != 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cu = c + u * kWarps;
            if (cu >= c1 || m0 + mq >= p.M) continue;
            int4 v = part[u][0];
#pragma unroll
            for (int r = 1; r < MAX; ++r)
                if (r < splits) v = add4(v, part[u][r]);
            int8_store4<Y, ACC>(p, t0 + cu, m0 + mq, smem_at<const float>((uint32_t)(kI8SxOff + 4 * cu)), sw4, v, ok);
        }
    }
}

template <typename Y, bool ACC>
__global__ void __launch_bounds__(kI8Threads)
    fluxbin_int8_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                           const __grid_constant__ CUtensorMap map_y, const __grid_constant__ Int8TcArgs a) {
    const Int8Args& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sb = smem_base();
    const uint32_t full0 = sb, empty0 = sb + 8 * kI8MaxStages, done = sb + 16 * kI8MaxStages;
    constexpr uint32_t kSlot = 16 * kI8MaxStages + 8, kFailed = kSlot + 4;
    const uint32_t ring = sb + kI8RingOff;
    const uint32_t stage_bytes = (uint32_t)int8_stage_bytes(a.bn);

    const int rank = (int)(blockIdx.x % (unsigned)a.splits);
    const unsigned tile = blockIdx.x / (unsigned)a.splits;
    const int tile_t = (int)(tile % (unsigned)a.tiles_t), tile_m = (int)(tile / (unsigned)a.tiles_t);
    const int kb0 = (int)((int64_t)a.kblocks * rank / a.splits), kb1 = (int)((int64_t)a.kblocks * (rank + 1) / a.splits);
    const int nk = kb1 - kb0;
    const int m0 = tile_m * kI8Rows;

    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + kSlot),
                     "r"(a.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc_mbar_init(full0 + 8 * s, 1);
            tc_mbar_init(empty0 + 8 * s, 1);
        }
        tc_mbar_init(done, 1);
        smem_at<uint32_t>(kFailed) = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = smem_at<const uint32_t>(kSlot);
    const bool aligned = (sb & 1023u) == 0;

    if (warp == 0 && aligned) {
        // ---- copies ----
        if (elect_one()) {
            bool ok = true;
            const bool early = (p.flags & kInt8Early) != 0;
            const int ahead = nk < a.stages ? nk : a.stages;
            const int nload = a.test_stall ? 0 : nk;
            // the ring's first weights before the preceding kernel has
            // finished, at least into L2
            for (int s = 0; s < ahead && nload; ++s) {
                if (early) {
                    int8_expect(full0 + 8 * s, stage_bytes);
                    int8_tma(ring + s * stage_bytes, &map_w, (kb0 + s) * kI8K, m0, full0 + 8 * s);
                } else {
                    int8_prefetch(&map_w, (kb0 + s) * kI8K, m0);
                }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int i = 0, s = 0;
            uint32_t round = 0;                  // times the ring has been filled before
            for (; i < nload; ++i) {
                if (round > 0 && !(ok = tc_mbar_wait(empty0 + 8 * s, (round - 1) & 1u, a.spin_limit))) break;
                const uint32_t dst = ring + s * stage_bytes, bar = full0 + 8 * s;
                if (!early || i >= ahead) {
                    int8_expect(bar, stage_bytes);
                    int8_tma(dst, &map_w, (kb0 + i) * kI8K, m0, bar);
                }
                int8_tma(dst + kI8Rows * kI8K, &map_x, (kb0 + i) * kI8K, tile_t * a.bn, bar);
                if (++s == a.stages) {
                    s = 0;
                    ++round;
                }
            }
            if (!ok) {
                atomicOr(a.err, 1u);
                smem_at<uint32_t>(kFailed) = 1u;
            }
            // copies in flight land before the CTA ends: the last fill of every stage
            for (int k = i > a.stages ? i - a.stages : 0; k < i; ++k)
                (void)tc_mbar_wait(full0 + 8 * (k % a.stages), (uint32_t)(k / a.stages) & 1u, kI8SpinLimit);
        }
    } else if (warp == 1 && aligned) {
        // ---- matrix instructions ----
        if (elect_one()) {
            const uint32_t idesc = int8_idesc(kI8Rows, a.bn);
            // the stages' tokens come after the preceding kernel, and the limit
            // of a wait is not for that kernel's time
            asm volatile("griddepcontrol.wait;" ::: "memory");
            bool ok = true;
            int s = 0;
            uint32_t round = 0;
            for (int i = 0; i < nk; ++i) {
                if (!(ok = tc_mbar_wait(full0 + 8 * s, round & 1u, a.spin_limit))) break;
                const uint64_t da = tc_smem_desc_sw128(ring + s * stage_bytes);
                const uint64_t db = tc_smem_desc_sw128(ring + s * stage_bytes + kI8Rows * kI8K);
#pragma unroll
                for (int k = 0; k < 4; ++k) int8_mma(tmem, da + 2 * k, db + 2 * k, idesc, i > 0 || k > 0);
                tc_commit(empty0 + 8 * s);
                if (++s == a.stages) {
                    s = 0;
                    ++round;
                }
            }
            tc_commit(done);   // every instruction issued above has finished (at once when there is none)
            if (!ok) {
                atomicOr(a.err, 1u);
                smem_at<uint32_t>(kFailed) = 1u;
            }
        }
    }
    __syncwarp();
    // scales are read and outputs written after the preceding kernel; they
    // are on their way while the products run.  (By plain loads: the preceding
    // kernel writes them while this one is already running, so they are not
    // what an invariant load may read.)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t0 = (int64_t)tile_t * a.bn;
    const int nt = (int)(p.T - t0 < a.bn ? p.T - t0 : a.bn);
    if (tid < a.bn) smem_at<float>(kI8SxOff + 4 * tid) = tid < nt ? p.sx[t0 + tid] : 0.f;
    if (ACC && a.splits == 1 && tid < nt) int8_prefetch_row<Y>(p, t0 + tid, m0);
    const int quarter = warp & 3;                // the lanes of tensor memory that this warp reaches
    const int row = quarter * 32 + lane, m = m0 + row;
    const int mq = 4 * lane;                     // the four channels of the split's sums
    float sw4[4];
    if (a.splits == 1) {
        sw4[0] = m < p.M ? p.sw[m] : 0.f;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) sw4[j] = m0 + mq + j < p.M ? p.sw[m0 + mq + j] : 0.f;
    }
    // every thread waits for the accumulators; the full limit even under the
    // test hook, since nothing may release them under running instructions.
    // What one thread could not confirm, none takes for confirmed.
    const bool drained = __syncthreads_and(!aligned || tc_mbar_wait(done, 0u, kI8SpinLimit)) != 0;
    tc_fence_after();
    const bool ok = drained && aligned && smem_at<const volatile uint32_t>(kFailed) == 0u;
    if (tid == 0 && (!drained || !aligned)) {
        atomicOr(a.err, drained ? 1u : 2u);
        smem_at<uint32_t>(kFailed) = 1u;         // (read by the cluster's other CTAs)
    }

    const uint32_t acc0 = tmem + ((uint32_t)(quarter * 32) << 16);
    const bool bulk = a.splits == 1 && a.bulk > (p.M - m0 >= kI8Rows ? 0 : 1);
    if (ACC && a.splits == 1) {
        int8_rows_in<Y, kI8Threads, 4>(p, kI8RingOff, t0, nt, m0, tid);
        __syncthreads();
    }
    // Every stage has been consumed: the ring holds the partial sums
    // ([bn][128] integers), or the tile of y on its way out ([bn][128] of Y).
    // Groups of 16 tokens, alternately to the two warps that reach a quarter.
    for (int g = warp >> 2; g < a.bn / 16; g += 2) {
        const int c = 16 * g;
        int v[16];
        int8_ld16(acc0 + (uint32_t)c, v);
        tc_wait_ld();
        if (a.splits > 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j) smem_at<int>((uint32_t)(kI8RingOff + ((c + j) * kI8Rows + row) * 4)) = v[j];
            continue;
        }
        float f[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 s4 = smem_at<const float4>((uint32_t)(kI8SxOff + 4 * (c + j)));
            f[j] = int8_value(v[j], s4.x, sw4[0]);
            f[j + 1] = int8_value(v[j + 1], s4.y, sw4[0]);
            f[j + 2] = int8_value(v[j + 2], s4.z, sw4[0]);
            f[j + 3] = int8_value(v[j + 3], s4.w, sw4[0]);
        }
        if (!ok) {
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = __int_as_float(0x7fc00000);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            Y& o = smem_at<Y>((uint32_t)(kI8RingOff + ((c + j) * kI8Rows + row) * (int)sizeof(Y)));
            o = from_f32<Y>(ACC ? to_f32(o) + f[j] : f[j]);
        }
    }
    if (bulk) fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 1 && drained) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
    }
    if (bulk) {
        if (tid == 0) {
            for (int c = 0; c < nt; c += kI8OutBox)
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                             ::"l"(&map_y), "r"(m0), "r"((int)(t0 + c)), "r"(ring + (uint32_t)(c * kI8Rows * (int)sizeof(Y)))
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    if (a.splits == 1 && !bulk) int8_rows_out<Y, kI8Threads, 4>(p, kI8RingOff, t0, nt, m0, tid);
    if (a.splits > 1) {
        int8_cluster_sync();
        // one lane asks each CTA whether it failed, while the sums are on their way
        const int failed = lane < a.splits ? ld_dsmem(dsmem_addr(sb + kFailed, lane)) : 0;
        // this CTA's share of the tile's tokens, added over the cluster: a
        // warp has the 128 channels of a token, four a lane, and the loads of
        // several tokens overlap
        const int c0 = nt * rank / a.splits, c1 = nt * (rank + 1) / a.splits;
        if (c0 + warp >= c1) {
            // a warp without tokens has to wait for the word that it has read
            // too: the barrier below orders no loads
            if (failed) atomicOr(a.err, 1u);
        } else if (a.splits <= 4) {
            int8_sum_split<Y, ACC, 4, 2>(p, ring, a.splits, rank, t0, c0 + warp, c1, m0, mq, sw4, failed);
        } else {
            int8_sum_split<Y, ACC, kI8MaxSplits, 2>(p, ring, a.splits, rank, t0, c0 + warp, c1, m0, mq, sw4, failed);
        }
        __syncwarp();
        // the others have read this CTA's sums (nothing to publish: a release
        // would wait for the stores of y)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    }
}

}  // namespace fluxbin
