// The 8-bit integer product for many tokens (sm_100a): pairs of CTAs.
//
// A pair owns a tile of 256 channels by `bn` tokens (a multiple of 32 up to
// 256): one tcgen05.mma (cta_group::2) reads 128 channels from each CTA's
// shared memory and half of the tokens from each, so that a CTA loads
// 128 + bn/2 rows per stage where a lone CTA would load 128 + bn for the same
// work.  That is what a product of this size needs: at the integer rate of
// the tensor cores a lone 128 x 256 tile asks for 96 bytes per clock and SM
// from L2, more than one SM takes in; the pair's asks for 64.
//
// The grid is persistent (one pair per two SMs) and each CTA holds two
// accumulators in tensor memory: eight warps empty one into y while the matrix
// instructions of the next tile run into the other.
//
// Roles per CTA: warp 0 copies (TMA, both CTAs signal the leader's full
// barriers), warp 1 of the leader issues the matrix instructions and commits
// them to both CTAs' empty barriers, warps 2-5 and 6-9 write the outputs, chunk
// by chunk in turn: scaled and rounded into a staging buffer of [tokens][128
// channels] and from there to y by TMA.  (An SM gets a store away every 13 to
// 20 clocks, however narrow it is: 32 channels of a token at a time, straight
// from the registers, left the last tile's outputs exposed for 17 us.)  Rows of
// y that TMA cannot write go out of the buffer in the widest stores they allow.
// Tiles run token tile by token tile within groups of 8 token tiles, so that
// the pairs at work share their weights and a group's tokens through L2.
//
// A pair's CTAs wait for each other while they hold tensor memory, so no two
// kernels that do may share an SM halfway: a CTA takes all of an SM's shared
// memory.
//
// Bound: the tensor cores, 96% busy while an SM has a tile (2048x28672x8192:
// 285 to 332 us with the GPU's power cap, 2.9 to 3.4 POP/s; the last of 13
// rounds has 8 tiles for 74 pairs).
#pragma once

#include "fluxbin_int8_tc.cuh"

namespace fluxbin {

constexpr int kI8PairThreads = 320;
constexpr int kI8PairStages = 6;
constexpr int kI8PairGroup = 8;          // token tiles that share a pass over the weights

struct Int8PairArgs {
    Int8Args p;
    int32_t bn, kblocks, tiles_t, tiles_m;
    int64_t tiles;
    uint32_t spin_limit;
    int32_t test_stall;
    int32_t bulk;         // y's rows can be written (and read) by TMA: 1 whole tiles, 2 a ragged last tile too
    unsigned int* err;
};

__host__ __device__ constexpr int int8_pair_stage_bytes(int bn) { return kI8Rows * kI8K + (bn / 2) * kI8K; }
// Always sized for the widest tile: all of an SM's shared memory.
constexpr int kI8PairRingOff = 1024;
constexpr int kI8PairOutOff = kI8PairRingOff + kI8PairStages * int8_pair_stage_bytes(kI8MaxBn);
constexpr int kI8PairOutBytes = 8192;    // a staging buffer: 32 tokens of a 16-bit y, 16 of a 32-bit one
constexpr int kI8PairSxOff = kI8PairOutOff + 4 * kI8PairOutBytes;  // [2][256] token scales
constexpr int kI8PairSmem = kI8PairSxOff + 2 * kI8MaxBn * 4;
__host__ __device__ constexpr int int8_pair_chunk(int size) { return kI8PairOutBytes / (kI8Rows * size); }

__device__ __forceinline__ void int8_pair_mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}
// A copy into this CTA's shared memory that signals a barrier of the pair.
__device__ __forceinline__ void int8_pair_tma(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// Arrives on the same barrier of both CTAs once this thread's matrix instructions have finished.
__device__ __forceinline__ void int8_pair_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b16 m;\n\t"
        "mov.b16 m, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}"
        ::"r"(bar) : "memory");
}
__device__ __forceinline__ void int8_remote_arrive(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void int8_ld32(uint32_t taddr, int (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

// The four output warps of a group, or both groups.
__device__ __forceinline__ void int8_out_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ void int8_out_sync_all() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

// C columns of the accumulators.
template <int C>
__device__ __forceinline__ void int8_ld(uint32_t taddr, int (&v)[C]) {
    if constexpr (C == 32) int8_ld32(taddr, v);
    else int8_ld16(taddr, v);
}

// Accumulation into a tile of y whose rows TMA cannot move, by one group: its
// chunks of 16 tokens (every other one) through an fp32 staging buffer, 128
// channels a token with a gap after every 8, so that lanes which read 8 channels
// each meet different banks.  A lane adds and writes the 16 bytes of a row that
// start on a 16-byte boundary, requested two chunks ahead (a chunk takes less
// time than a load); the ends of a row go element by element.  Against reading
// and writing a whole chunk at a time: 495x22306x1152 fp32 65 -> 39.5 us,
// 2000x11009x1000 bf16 73 -> 51; with one chunk ahead 49 and 60; without
// accumulation the same way costs 5% more than int8_rows_out.  `ready` waits for
// the tile's accumulators and scales and says whether they are right.
constexpr int kI8RowsPitch = kI8Rows + kI8Rows / 8;
__device__ __forceinline__ uint32_t int8_rows_at(uint32_t buf, int j, int ch) {
    return buf + (uint32_t)(4 * (j * kI8RowsPitch + ch + (ch >> 3)));
}

template <typename Y, typename READY>
__device__ __forceinline__ void int8_pair_rows_add(const Int8Args& p, uint32_t acc, uint32_t buf, uint32_t sx, float sw,
                                                   int64_t t0, int m0, int chunks, int group, int e, int row, READY ready) {
    constexpr int kPer = 16 / (int)sizeof(Y), kLanes = kI8Rows / kPer, kStep = 128 / kLanes, S = 16 / kStep;
    static_assert(16 * kI8RowsPitch * 4 <= 2 * kI8PairOutBytes, "a group's two staging buffers");
    const int l = e % kLanes, j0 = e / kLanes, nv = p.M - m0 < kI8Rows ? p.M - m0 : kI8Rows;
    // this lane's 16 bytes of token j start at element c, and it also has
    // element `end` (-1: none)
    struct Place { Y* y; int c, end; };
    const auto place = [&](int64_t t) {
        Place r;
        r.y = static_cast<Y*>(p.y) + t * p.ldy + m0;
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(r.y) & 15u;
        const int head = off ? (int)((16u - off) / sizeof(Y)) : 0;
        const int whole = nv > head ? (nv - head) / kPer : 0;
        r.c = t < p.T && l < whole ? head + l * kPer : -1;
        r.end = l < head ? l : whole * kPer + l;
        if (t >= p.T || l >= 2 * kPer || r.end >= nv) r.end = -1;
        return r;
    };
    struct Held { uint4 v[S]; Y end[S]; };
    const auto request = [&](int q, Held& h) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const Place r = place(t0 + 16 * q + j0 + s * kStep);
            if (r.c >= 0) h.v[s] = *reinterpret_cast<const uint4*>(r.y + r.c);
            if (r.end >= 0) h.end[s] = r.y[r.end];
        }
    };
    bool ok = true;
    const auto add = [&](int q, Held& h) {
        int v[16];
        int8_ld16(acc + (uint32_t)(16 * q), v);
        float f[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 s4 = smem_at<const float4>(sx + (uint32_t)(4 * (16 * q + j)));
            f[j] = s4.x;
            f[j + 1] = s4.y;
            f[j + 2] = s4.z;
            f[j + 3] = s4.w;
        }
        tc_wait_ld();
        int8_out_sync(group);                      // the chunk before has been read
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float x = int8_value(v[j], f[j], sw);
            smem_at<float>(int8_rows_at(buf, j, row)) = ok ? x : __int_as_float(0x7fc00000);
        }
        int8_out_sync(group);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = j0 + s * kStep;
            const Place r = place(t0 + 16 * q + j);
            if (r.c >= 0) {
                alignas(16) Y o[kPer];
                *reinterpret_cast<uint4*>(o) = h.v[s];
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    o[k] = from_f32<Y>(to_f32(o[k]) + smem_at<const float>(int8_rows_at(buf, j, r.c + k)));
                *reinterpret_cast<uint4*>(r.y + r.c) = *reinterpret_cast<const uint4*>(o);
            }
            if (r.end >= 0)
                r.y[r.end] = from_f32<Y>(to_f32(h.end[s]) + smem_at<const float>(int8_rows_at(buf, j, r.end)));
        }
        if (q + 4 < chunks) request(q + 4, h);
    };
    Held h0, h1;
    if (group < chunks) request(group, h0);
    if (group + 2 < chunks) request(group + 2, h1);
    ok = ready();
    for (int q = group; q < chunks; q += 4) {
        add(q, h0);
        if (q + 2 < chunks) add(q + 2, h1);
    }
}

struct Int8PairTile {
    int tm, tt;
};
__device__ __forceinline__ Int8PairTile int8_pair_tile(const Int8PairArgs& a, int64_t i) {
    const int64_t per_group = (int64_t)kI8PairGroup * a.tiles_m;
    const int g = (int)(i / per_group);
    const int64_t r = i % per_group;
    const int first = g * kI8PairGroup;
    const int n = a.tiles_t - first < kI8PairGroup ? a.tiles_t - first : kI8PairGroup;
    return Int8PairTile{(int)(r / n), first + (int)(r % n)};
}

template <typename Y, bool ACC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8PairThreads, 1)
    fluxbin_int8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                             const __grid_constant__ CUtensorMap map_y, const __grid_constant__ Int8PairArgs a) {
    const Int8Args& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sb = smem_base();
    // barriers: full and empty per stage, accumulator full and empty (2), done
    const uint32_t full0 = sb, empty0 = sb + 64, acc_full0 = sb + 128, acc_empty0 = sb + 144, done = sb + 160,
                   y_full0 = sb + 168;             // (four, one per staging buffer)
    constexpr uint32_t kSlot = 200, kDrained = 204;
    const uint32_t ring = sb + kI8PairRingOff;
    const uint32_t stage_bytes = (uint32_t)int8_pair_stage_bytes(a.bn);
    const int rank = (int)(blockIdx.x & 1);
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + kSlot), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < kI8PairStages; ++s) {
            tc_mbar_init(full0 + 8 * s, 1);
            tc_mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc_mbar_init(acc_full0 + 8 * b, 1);
            tc_mbar_init(acc_empty0 + 8 * b, 16);  // eight warps of each CTA
        }
        for (int b = 0; b < 4; ++b) tc_mbar_init(y_full0 + 8 * b, 1);
        tc_mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    int8_cluster_sync();                           // the other CTA's barriers exist
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = smem_at<const uint32_t>(kSlot);
    const bool aligned = (sb & 1023u) == 0;        // both CTAs have the same base
    bool ok = aligned;

    if (warp == 0) {
        if (aligned && elect_one()) {
            // ---- copies: this CTA's half of the channels and of the tokens ----
            const bool early = (p.flags & kInt8Early) != 0;
            const int half = a.bn / 2;
            const uint32_t bar0 = dsmem_addr(full0, 0);   // the leader's full barriers
            int pre = 0;                           // stages whose weights were requested early
            if (!a.test_stall && first < a.tiles) {
                // the ring's first weights before the preceding kernel has
                // finished, at least into L2
                const Int8PairTile t = int8_pair_tile(a, first);
                const int ahead = a.kblocks < kI8PairStages ? a.kblocks : kI8PairStages;
                const int wy = (t.tm * 2 + rank) * kI8Rows;
                for (int s = 0; s < ahead; ++s) {
                    if (early) {
                        if (rank == 0) int8_expect(full0 + 8 * s, 2 * stage_bytes);
                        int8_pair_tma(ring + s * stage_bytes, &map_w, s * kI8K, wy, bar0 + 8 * s);
                    } else {
                        int8_prefetch(&map_w, s * kI8K, wy);
                    }
                }
                if (early) pre = ahead;
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int s = 0;
            uint32_t round = 0;                    // times the ring has been filled before
            for (int64_t i = first; i < a.tiles && ok && !a.test_stall; i += step) {
                const Int8PairTile t = int8_pair_tile(a, i);
                const int wy = (t.tm * 2 + rank) * kI8Rows, xy = t.tt * a.bn + rank * half;
                for (int k = 0; k < a.kblocks; ++k) {
                    if (round > 0 && !(ok = tc_mbar_wait(empty0 + 8 * s, (round - 1) & 1u, a.spin_limit))) break;
                    const uint32_t dst = ring + s * stage_bytes, bar = bar0 + 8 * s;
                    if (pre > 0) {
                        --pre;
                    } else {
                        if (rank == 0) int8_expect(full0 + 8 * s, 2 * stage_bytes);
                        int8_pair_tma(dst, &map_w, k * kI8K, wy, bar);
                    }
                    int8_pair_tma(dst + kI8Rows * kI8K, &map_x, k * kI8K, xy, bar);
                    if (++s == kI8PairStages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            if (!ok) {
                atomicOr(a.err, 1u);
                // the copies in flight land within microseconds; the leader's
                // barriers cannot be waited for from the other CTA, so a copier
                // that gave up stays for a millisecond
                for (int w = 0; w < 1000; ++w) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && aligned && elect_one()) {
            // ---- matrix instructions, for both CTAs ----
            const uint32_t idesc = int8_idesc(2 * kI8Rows, a.bn);
            // the stages' tokens come after the preceding kernel, and the limit
            // of a wait is not for that kernel's time
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int s = 0;
            uint32_t round = 0;
            int64_t n = 0;                         // tiles so far
            for (int64_t i = first; i < a.tiles && ok; i += step, ++n) {
                const int b = (int)(n & 1);
                if (n >= 2 && !(ok = tc_mbar_wait(acc_empty0 + 8 * b, (uint32_t)((n >> 1) - 1) & 1u, a.spin_limit))) break;
                tc_fence_after();
                for (int k = 0; k < a.kblocks; ++k) {
                    if (!(ok = tc_mbar_wait(full0 + 8 * s, round & 1u, a.spin_limit))) break;
                    const uint64_t da = tc_smem_desc_sw128(ring + s * stage_bytes);
                    const uint64_t db = tc_smem_desc_sw128(ring + s * stage_bytes + kI8Rows * kI8K);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        int8_pair_mma(tmem + (uint32_t)(b * kI8MaxBn), da + 2 * q, db + 2 * q, idesc, k > 0 || q > 0);
                    int8_pair_commit(empty0 + 8 * s);
                    if (++s == kI8PairStages) {
                        s = 0;
                        ++round;
                    }
                }
                if (ok) int8_pair_commit(acc_full0 + 8 * b);
            }
            int8_pair_commit(done);                // every instruction issued above has finished
            if (!ok) atomicOr(a.err, 1u);
        }
    } else {
        // ---- outputs ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int C = int8_pair_chunk((int)sizeof(Y));   // tokens of a chunk
        const int group = (warp - 2) >> 2;         // takes every other chunk
        const int quarter = warp & 3;              // the lanes of tensor memory that this warp reaches
        const int e = (tid - 64) & 127, row = quarter * 32 + lane;
        const int chunks = a.bn / C;
        // the group's two staging buffers
        const uint32_t buf0 = (uint32_t)(kI8PairOutOff + 2 * group * kI8PairOutBytes), y_full = y_full0 + 16 * group;
        uint32_t y_parity = 0u;                    // of the loads of y into each of them (one bit each)
        // the group's chunks take its buffers in turn, across tiles too: the wait
        // below leaves the chunk before unread, and a tile may have an odd number
        const int odd = ((chunks - group + 1) >> 1) & 1;
        int64_t n = 0;
        for (int64_t i = first; i < a.tiles; i += step, ++n) {
            const Int8PairTile t = int8_pair_tile(a, i);
            const int b = (int)(n & 1);
            const int m0 = (t.tm * 2 + rank) * kI8Rows, m = m0 + row;
            const int64_t t0 = (int64_t)t.tt * a.bn;
            // TMA writes whole 16-byte pieces: a ragged last tile only where
            // M ends on one
            const bool bulk = a.bulk > (p.M - m0 >= kI8Rows ? 0 : 1);
            const int turn = b & odd;              // the buffer of the tile's first chunk
            // requests a chunk's y (accumulation) into its staging buffer
            const auto load_y = [&](int q) {
                const int k = ((q >> 1) & 1) ^ turn;
                int8_expect(y_full + 8 * k, (uint32_t)kI8PairOutBytes);
                int8_tma(sb + buf0 + k * kI8PairOutBytes, &map_y, m0, (int)t0 + q * C, y_full + 8 * k);
            };
            // the tile's scales, requested before the accumulators are ready
            // (plain loads: the preceding kernel may have written them after
            // this one started)
            const float sw = m < p.M ? p.sw[m] : 0.f;
            {
                const int c = tid - 64;
                smem_at<float>(kI8PairSxOff + (b * kI8MaxBn + c) * 4) = c < a.bn && t0 + c < p.T ? p.sx[t0 + c] : 0.f;
            }
            if (ACC) {                             // (the tile before may have gone out by plain stores)
                fence_async_smem();
                int8_out_sync(group);
            }
            if (ACC && bulk && e == 0 && group < chunks) {
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                load_y(group);
            }
            const uint32_t acc = tmem + (uint32_t)(b * kI8MaxBn) + ((uint32_t)(quarter * 32) << 16);
            const auto ready = [&]() {
                if (ok) ok = tc_mbar_wait(acc_full0 + 8 * b, (uint32_t)(n >> 1) & 1u, a.spin_limit);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                int8_out_sync_all();               // the token scales are in place
                return ok;
            };
            if (ACC && !bulk) {
                if (e == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                int8_pair_rows_add<Y>(p, acc, buf0, (uint32_t)(kI8PairSxOff + b * kI8MaxBn * 4), sw, t0, m0, a.bn / 16,
                                      group, e, row, ready);
            } else {
                ready();
            }
            for (int q = group; q < chunks && (!ACC || bulk); q += 2) {
                const int k = ((q >> 1) & 1) ^ turn, c = q * C;
                const uint32_t out = buf0 + (uint32_t)(k * kI8PairOutBytes);
                int v[C];
                int8_ld<C>(acc + (uint32_t)c, v);
                // the staging buffer is free once what went out of it two
                // chunks ago (in this tile or the one before) has been read;
                // with accumulation the next chunk's y is requested a chunk ahead
                if (e == 0) {
                    if (ACC) {
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        if (q + 2 < chunks) load_y(q + 2);
                    } else if (bulk) {
                        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    } else {
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                }
                if (!ACC) int8_out_sync(group);
                float f[C];
#pragma unroll
                for (int j = 0; j < C; j += 4) {
                    const float4 s4 = smem_at<const float4>(kI8PairSxOff + (b * kI8MaxBn + c + j) * 4);
                    f[j] = s4.x;
                    f[j + 1] = s4.y;
                    f[j + 2] = s4.z;
                    f[j + 3] = s4.w;
                }
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    f[j] = int8_value(v[j], f[j], sw);
                    if (!ok) f[j] = __int_as_float(0x7fc00000);
                }
                if (ACC) {
                    ok = tc_mbar_wait(y_full + 8 * k, (y_parity >> k) & 1u, kI8SpinLimit) && ok;
                    y_parity ^= 1u << k;
                }
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    Y& o = smem_at<Y>(out + (uint32_t)((j * kI8Rows + row) * (int)sizeof(Y)));
                    o = from_f32<Y>(ACC ? to_f32(o) + f[j] : f[j]);
                }
                if (ACC || bulk) fence_async_smem();
                int8_out_sync(group);
                if (ACC || bulk) {
                    if (e == 0) {
                        if (t0 + c < p.T && m0 < p.M)
                            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                                         ::"l"(&map_y), "r"(m0), "r"((int)(t0 + c)), "r"(sb + out) : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                } else {
                    int8_rows_out<Y, 128, 2>(p, out, t0 + c, C, m0, e);
                }
            }
            // this warp has read its part of the accumulators
            tc_fence_before();
            __syncwarp();
            if (lane == 0) int8_remote_arrive(dsmem_addr(acc_empty0 + 8 * b, 0));
        }
        if (a.bulk && e == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok) atomicOr(a.err, 1u);
    }
    // every role has come to its end before anyone waits for the last matrix
    // instructions: the limit of that wait is not for all of the tiles' time
    __syncwarp();
    __syncthreads();
    const bool drained = !aligned || tc_mbar_wait(done, 0u, kI8SpinLimit);
    tc_fence_before();
    // the release takes both CTAs: each knows whether the other's waits went well
    const int all_drained = __syncthreads_and(drained);
    if (tid == 0) {
        smem_at<int>(kDrained) = all_drained;
        if (!all_drained || !aligned) atomicOr(a.err, all_drained ? 1u : 2u);
    }
    int8_cluster_sync();
    const bool release = all_drained && ld_dsmem(dsmem_addr(sb + kDrained, rank ^ 1)) != 0;
    int8_cluster_sync();
    if (warp == 1 && release) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

}  // namespace fluxbin
