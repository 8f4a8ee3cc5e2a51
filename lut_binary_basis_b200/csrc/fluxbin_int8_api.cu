// C-ABI entry points of the 8-bit operators: argument validation, the choice
// of a kernel and the launch.  Declarations and the full contract are in
// include/fluxbin.h.
#include <cmath>
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/fluxbin.h"
#include "fluxbin_device.h"
#include "fluxbin_int8.cuh"
#include "fluxbin_int8_mv.cuh"
#include "fluxbin_int8_tc.cuh"
#include "fluxbin_int8_tc2.cuh"
#include "fluxbin_quant.cuh"

namespace fluxbin {
namespace {

constexpr int32_t kInt8MaxN = 131071;   // 128 * 128 * N < 2^31
constexpr int32_t kInt8MaxRows = INT32_MAX - 1023;   // a tile's last row still has a 32-bit number

// Beyond any address space: offsets and sums of them stay far from 2^63.
constexpr int64_t kMaxPitch = (int64_t)1 << 39;   // elements from a row to the next
constexpr int64_t kMaxSpan = (int64_t)1 << 57;    // bytes from the first row to the last

// A row pitch (in elements of `size` bytes) that T rows of n elements can have.
bool bad_pitch(int64_t ld, int64_t n, int64_t T, int64_t size) {
    return ld < n || ld > kMaxPitch || (T > 1 && ld * size > kMaxSpan / (T - 1));
}

bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A row-major array of T rows of N elements, `ld` elements apart.
struct Rows {
    const void* p;
    int64_t T, N, ld;
    int size;   // bytes of an element
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t end() const { return begin() + (uintptr_t)(((T - 1) * ld + N) * size); }
    bool rows_aligned16() const { return ptr_aligned(p, 16) && (ld * size) % 16 == 0; }
};
bool overlap(const Rows& a, const Rows& b) {
    return a.p && b.p && a.N > 0 && b.N > 0 && a.begin() < b.end() && b.begin() < a.end();
}

template <typename K, typename... Args>
int launch(K kernel, dim3 grid, dim3 block, size_t smem, int cluster, void* stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? FLUXBIN_OK : report_cuda_failure(e);
}

constexpr int kMaxDevices = 64;
std::mutex g_int8_mu;

struct Int8Device {
    bool ready = false;
    int index = 0;
    int sm_count = 0;
    unsigned int* err = nullptr;
} g_int8_dev[kMaxDevices];

int int8_device(Int8Device* out);

using QuantFn = void (*)(QuantArgs);

constexpr int64_t kQuantFewBlocks = 148;                 // CTAs that have an SM each
constexpr int64_t kQuantManyVecs = (int64_t)1 << 20;     // of 8 elements: 8 million elements

template <int KIND, typename E, typename H, bool VEC>
QuantFn pick_quant(int vpt) {
    switch (vpt) {
        case 1: return &fluxbin_quant_kernel<KIND, E, H, 1, VEC>;
        case 2: return &fluxbin_quant_kernel<KIND, E, H, 2, VEC>;
        default: return &fluxbin_quant_kernel<KIND, E, H, 4, VEC>;
    }
}
template <int KIND, typename E, typename H>
QuantFn pick_quant(int vpt, bool vec) { return vec ? pick_quant<KIND, E, H, true>(vpt) : pick_quant<KIND, E, H, false>(vpt); }

template <typename E>
QuantFn pick_gate(int vpt) {
    return vpt == 2   ? &fluxbin_gate_rows_kernel<E, 2>
           : vpt == 3 ? &fluxbin_gate_rows_kernel<E, 3>
                      : &fluxbin_gate_rows_kernel<E, kGateMaxVpt>;
}

// The gate for many aligned rows: vectors a thread, threads and CTAs per SM, or
// 0 vectors where the other kernel has it.  Rows of up to 1536 vectors: as many
// CTAs of up to 512 threads as an SM's registers hold, for they hide each
// other's reductions (2048x11008: two CTAs with 3 vectors 22.1 us, with 4 22.7,
// one with 2 23.6; 2048x8192 16.3); longer ones a CTA with the fewest vectors
// (2048x14336: 2 vectors 27.3, 3 28.4, two CTAs with 4 28.6).  The other kernel
// takes 24.7, 18.0, 31.0 and, at 2048x28672, 64.4 for 51.7.  A CTA should have
// four rows, two where the other kernel needs a cluster for one (296x14336 6.1
// against 6.6 here, 592 rows 10.8 and 10.1; 296x20480 11.7 and 8.5).
struct GatePlan { int vpt, threads, per_sm; };
GatePlan plan_gate(int64_t T, int64_t N) {
    GatePlan g = {0, 0, 1};
    const int64_t vecs = N / 8;
    if (vecs < 512 || vecs * 64 > kGateMaxSmem) return g;
    const int64_t most = vecs <= 3 * 512 ? 512 : kGateMaxThreads;
    const int vpt = std::max(2, (int)((vecs + most - 1) / most));
    g.threads = (int)(((vecs + vpt - 1) / vpt + 31) / 32 * 32);
    g.per_sm = kGateMaxThreads / g.threads;
    if (T >= (vecs > 2048 ? 2 : 4) * kQuantFewBlocks * g.per_sm) g.vpt = vpt;
    return g;
}

// Checks what the three operators share and launches.  `in0`, `in1` (delta or
// up, may be null), `gamma` and `h_out` as the operator has them.
template <int KIND>
int run_quant(const Rows& in0, const Rows& in1, const void* gamma, float eps, const Rows& h_out, int8_t* d_q,
              int64_t ldq, float* d_scale, uint32_t flags, void* stream) {
    const int64_t T = in0.T, N = in0.N;
    const bool h32 = KIND == kQuantNorm && (flags & FLUXBIN_FLAG_H_FP32);
    if (N > kInt8MaxN) return FLUXBIN_ERR_UNSUPPORTED;
    if (!d_scale || (N > 0 && (!in0.p || !d_q))) return FLUXBIN_ERR_INVALID_ARG;
    if (KIND == kQuantSilu && N > 0 && !in1.p) return FLUXBIN_ERR_INVALID_ARG;
    if (KIND == kQuantNorm && !gamma) return FLUXBIN_ERR_INVALID_ARG;
    if (!ptr_aligned(in0.p, in0.size) || !ptr_aligned(in1.p, in1.size) || !ptr_aligned(gamma, 2) ||
        !ptr_aligned(h_out.p, h_out.size) || !ptr_aligned(d_scale, 4) || !ptr_aligned(d_q, 16) || ldq % 16)
        return FLUXBIN_ERR_MISALIGNED;
    const Rows q{d_q, T, N, ldq, 1}, sc{d_scale, 1, T, T, 4}, g{gamma, 1, N, N, 2};
    const Rows* ins[3] = {&in0, &in1, &g};
    const Rows* outs[3] = {&q, &sc, &h_out};
    for (const Rows* o : outs)
        for (const Rows* i : ins) {
            // the stream may be updated in place
            if (o == &h_out && i == &in0 && h_out.p == in0.p && h_out.ld == in0.ld) continue;
            if (overlap(*o, *i)) return FLUXBIN_ERR_INVALID_ARG;
        }
    if (overlap(q, sc) || overlap(q, h_out) || overlap(sc, h_out)) return FLUXBIN_ERR_INVALID_ARG;

    QuantArgs a = {};
    a.a = in0.p;
    a.b = in1.p;
    a.gamma = gamma;
    a.h_out = const_cast<void*>(h_out.p);
    a.q = d_q;
    a.scale = d_scale;
    a.lda = in0.ld;
    a.ldb = in1.ld;
    a.ldo = h_out.ld;
    a.ldq = ldq;
    a.T = (int32_t)T;
    a.N = (int32_t)N;
    a.eps = eps;
    const bool vec = N % 8 == 0 && in0.rows_aligned16() && (!in1.p || in1.rows_aligned16()) &&
                     (!gamma || ptr_aligned(gamma, 16)) && (!h_out.p || h_out.rows_aligned16());
    if (KIND == kQuantSilu && vec) {
        const GatePlan g = plan_gate(T, N);
        if (g.vpt) {
            Int8Device d;
            const int st = int8_device(&d);
            if (st != FLUXBIN_OK) return st;
            const QuantFn fn = (flags & FLUXBIN_FLAG_BF16) ? pick_gate<__nv_bfloat16>(g.vpt) : pick_gate<__half>(g.vpt);
            return launch(fn, dim3((unsigned)std::min<int64_t>(T, (int64_t)d.sm_count * g.per_sm)), dim3((unsigned)g.threads),
                          (size_t)N * 8, 1, stream, a);
        }
    }
    // Vectors of 8 elements a thread, and CTAs a row (B200, us a call, a graph
    // of calls).  Few rows: one vector, and a cluster once it leaves a CTA 256
    // threads or more (gate 1x11008: four CTAs 2.2, one with two vectors 2.6;
    // norm 1x4096: one CTA 2.1, two 2.5).  Many rows: four vectors, so that
    // several CTAs of an SM are in different phases (quant 4096x8192 1 / 2 / 4
    // vectors 31 / 22 / 18.9, norm 2048x8192 27.4 / 22.4 / 21.0), but two for
    // the gate, a 32-bit stream and unaligned rows, which need more registers
    // (gate 2048x11008 24.3 / 26.8, norm of a 32-bit 2048x8192 32.3 / 32.8).
    const int64_t vecs = (N + 7) / 8;
    int vpt = 1, parts = 1;
    if (vecs >= 1024 && T * (vecs > 2048 ? 8 : 4) <= kQuantFewBlocks) {
        parts = vecs > 2048 ? 8 : 4;
    } else if (T * vecs >= kQuantManyVecs) {
        vpt = vecs < 512 ? 1 : (KIND == kQuantSilu || h32 || !vec) ? 2 : 4;
    } else if (T > kQuantFewBlocks / 4 && vecs >= 512) {
        vpt = 2;
    }
    while (vpt < 4 && vecs > (int64_t)parts * vpt * quant_max_threads(vpt)) vpt *= 2;
    while (vecs > (int64_t)parts * vpt * quant_max_threads(vpt)) parts *= 2;
    const int64_t per_thread = (int64_t)parts * vpt;
    const int tpr = std::max(32, (int)(((vecs + per_thread - 1) / per_thread + 31) / 32 * 32));
    a.parts = parts;
    const int rpc = tpr >= 128 ? 1 : 128 / tpr;
    // Rows from a CTA's own to the one that it asks L2 for, so that memory is
    // busy while the CTAs at work compute and store: about half of those that
    // fit the GPU at a time, for CTAs do not start all at once (quant 4096x8192
    // 0 / 1/4 / 1/2 / 1 of them ahead 18.9 / 18.1 / 17.0 / 16.8 us, 32-bit norm
    // 2048x8192 32.5 / 30.4 / 30.4 / 32.1).  The gate gains where a cluster has
    // the row or rows are unaligned (2048x29000 71 -> 67, 2048x28671
    // 122 -> 98) and loses a little elsewhere (2048x4096 9.8 -> 10.4).
    const int64_t resident = (vpt == 1 ? 2048 : vpt == 2 ? 1536 : 1024) / (tpr * rpc) * kQuantFewBlocks / parts;
    if (KIND != kQuantSilu || parts > 1 || !vec) a.ahead = (int)((resident + 1) / 2) * rpc;
    const bool bf = (flags & FLUXBIN_FLAG_BF16) != 0;
    QuantFn fn;
    if constexpr (KIND == kQuantNorm) {
        if (h32)
            fn = bf ? pick_quant<KIND, __nv_bfloat16, float>(vpt, vec) : pick_quant<KIND, __half, float>(vpt, vec);
        else
            fn = bf ? pick_quant<KIND, __nv_bfloat16, __nv_bfloat16>(vpt, vec)
                    : pick_quant<KIND, __half, __half>(vpt, vec);
    } else {
        fn = bf ? pick_quant<KIND, __nv_bfloat16, __nv_bfloat16>(vpt, vec) : pick_quant<KIND, __half, __half>(vpt, vec);
    }
    const int64_t blocks = (T + rpc - 1) / rpc * parts;
    if (blocks > INT32_MAX) return FLUXBIN_ERR_UNSUPPORTED;
    return launch(fn, dim3((unsigned)blocks), dim3((unsigned)tpr, (unsigned)rpc), 0, parts, stream, a);
}

// ---------------------------------------------------------------------------
// The integer product
// ---------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn g_encode = nullptr;

using Int8TcFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Int8TcArgs);
using Int8EmptyFn = void (*)(Int8Args);

template <typename Y>
Int8TcFn pick_tc(bool acc) { return acc ? &fluxbin_int8_tc_kernel<Y, true> : &fluxbin_int8_tc_kernel<Y, false>; }
Int8TcFn pick_int8_tc(uint32_t flags) {
    const bool acc = (flags & kInt8Accumulate) != 0;
    return (flags & kInt8YFp32) ? pick_tc<float>(acc) : (flags & kInt8Bf16) ? pick_tc<__nv_bfloat16>(acc) : pick_tc<__half>(acc);
}
using Int8PairFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Int8PairArgs);
template <typename Y>
Int8PairFn pick_pair(bool acc) { return acc ? &fluxbin_int8_pair_kernel<Y, true> : &fluxbin_int8_pair_kernel<Y, false>; }
Int8PairFn pick_int8_pair(uint32_t flags) {
    const bool acc = (flags & kInt8Accumulate) != 0;
    return (flags & kInt8YFp32) ? pick_pair<float>(acc) : (flags & kInt8Bf16) ? pick_pair<__nv_bfloat16>(acc) : pick_pair<__half>(acc);
}
template <typename Y>
Int8EmptyFn pick_mv(bool acc, bool two) {
    return two ? (acc ? &fluxbin_int8_mv_kernel<Y, true, 2> : &fluxbin_int8_mv_kernel<Y, false, 2>)
               : (acc ? &fluxbin_int8_mv_kernel<Y, true, 1> : &fluxbin_int8_mv_kernel<Y, false, 1>);
}
template <typename Y>
Int8EmptyFn pick_empty(bool acc) { return acc ? &fluxbin_int8_empty_kernel<Y, true> : &fluxbin_int8_empty_kernel<Y, false>; }

constexpr int kI8MaxSmem = 227 * 1024;

// Per-device set-up: the product's error word, the number of SMs, the kernels'
// opt-in to their shared memory; once the tensor-map encoder.
int int8_device(Int8Device* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda_failure(e);
    if (dev < 0 || dev >= kMaxDevices) return FLUXBIN_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_int8_mu);
    Int8Device& d = g_int8_dev[dev];
    if (!d.ready) {
        if (!g_encode) {
            void* fn = nullptr;
            cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
            e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
            if (e != cudaSuccess) return report_cuda_failure(e);
            if (q != cudaDriverEntryPointSuccess || !fn) return report_cuda_failure(cudaErrorSymbolNotFound);
            g_encode = reinterpret_cast<EncodeFn>(fn);
        }
        if ((e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return report_cuda_failure(e);
        for (const uint32_t f : {0u, kInt8YFp32, kInt8Bf16})
            for (const uint32_t acc : {0u, kInt8Accumulate})
                if ((e = cudaFuncSetAttribute(pick_int8_tc(f | acc), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              kI8MaxSmem)) != cudaSuccess ||
                    (e = cudaFuncSetAttribute(pick_int8_pair(f | acc), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              kI8PairSmem)) != cudaSuccess)
                    return report_cuda_failure(e);
        for (int vpt = 2; vpt <= kGateMaxVpt; ++vpt)
            for (const QuantFn fn : {pick_gate<__half>(vpt), pick_gate<__nv_bfloat16>(vpt)})
                if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGateMaxSmem)) != cudaSuccess)
                    return report_cuda_failure(e);
        const int st = device_error_word(dev, &d.err);
        if (st != FLUXBIN_OK) return st;
        d.index = dev;
        d.ready = true;
    }
    *out = d;
    return FLUXBIN_OK;
}

// Rows of codes as a tensor map: boxes of one swizzle row of K by `box` rows.
int encode_rows(CUtensorMap* map, const int8_t* base, int64_t rows, int64_t N, int64_t ld, int box) {
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t boxes[2] = {(cuuint32_t)kI8K, (cuuint32_t)box};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, boxes,
                                steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FLUXBIN_OK : report_cuda_failure(cudaErrorInvalidValue);
}

// Whether y's rows can be moved by TMA: 16-byte aligned, a pitch it can hold.
bool rows_allow_bulk(const Int8Args& p) {
    const int size = (p.flags & kInt8YFp32) ? 4 : 2;
    return ptr_aligned(p.y, 16) && (p.ldy * size) % 16 == 0 && p.ldy * size < ((int64_t)1 << 40);
}

// 0 where they cannot; else y as a tensor map with boxes of 128 channels by
// `box` tokens, and 1 for whole tiles only, 2 for a ragged last tile too (TMA
// writes whole 16-byte pieces).
int encode_y(CUtensorMap* map, const Int8Args& p, int box, int32_t* bulk) {
    const int size = (p.flags & kInt8YFp32) ? 4 : 2;
    *bulk = 0;
    if (!rows_allow_bulk(p)) return FLUXBIN_OK;
    *bulk = ((int64_t)p.M * size) % 16 == 0 ? 2 : 1;
    const cuuint64_t dims[2] = {(cuuint64_t)p.M, (cuuint64_t)p.T};
    const cuuint64_t strides[1] = {(cuuint64_t)p.ldy * (cuuint64_t)size};
    const cuuint32_t boxes[2] = {(cuuint32_t)kI8Rows, (cuuint32_t)box};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = g_encode(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.y,
                                dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FLUXBIN_OK : report_cuda_failure(cudaErrorInvalidValue);
}

// How many clusters of `splits` CTAs, one CTA per SM, the device holds at
// once.  (A cluster sits inside one of the GPU's processing clusters, whose
// sizes differ.  B200: 74 of 2, 45 of 3, 33 of 4, 26 of 5, 22 of 6, 15 of 7 and 8.)
int resident_clusters(const Int8Device& d, int splits) {
    static int known[kMaxDevices][kI8MaxSplits + 1];
    std::lock_guard<std::mutex> lock(g_int8_mu);
    int& n = known[d.index][splits];
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)splits);
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = (size_t)kI8MaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, pick_int8_tc(0), &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    return n;
}

// Tiles, split and ring of a call; returns the number of tiles.
//
// A tile's K is split until the CTAs fill one wave of the GPU, never more
// (B200, us a call, a graph of calls on rotated weights; splits 1 / 3 / 4:
// 16x11008x4096, 86 tiles on 296 slots 11.0 / 9.6 / 13.6 with the fourth in a
// second wave).  Two CTAs per SM (112 KB each) as long as that leaves a ring of
// three stages or more; from 113 tokens on a CTA takes the whole SM if half of
// them find work (128x4096x4096 9.1 against 9.9; 128x11008x4096, 86 tiles:
// unsplit 12.7, 3 splits on two CTAs per SM 13.4).  One CTA per SM is enough
// where a CTA's share is down to 8 stages (32x4096x4096 with 4 splits 6.5, with
// 8 6.7; 32x4096x11008 11.4 and 11.0).
int64_t plan_int8(const Int8Args& p, const Int8Device& d, Int8TcArgs* out, double* us) {
    Int8TcArgs& a = *out;
    a.kblocks = (p.N + kI8K - 1) / kI8K;
    // token tiles of equal size, a multiple of 16
    a.tiles_t = (int)(((int64_t)p.T + kI8MaxBn - 1) / kI8MaxBn);
    a.bn = (int)((((int64_t)p.T + a.tiles_t - 1) / a.tiles_t) + 15) / 16 * 16;
    const int64_t tiles = (int64_t)a.tiles_t * (((int64_t)p.M + kI8Rows - 1) / kI8Rows);
    const int one = (int)std::min<int64_t>(kI8MaxSplits, d.sm_count / tiles);
    const int two = (int)std::min<int64_t>(kI8MaxSplits, 2 * d.sm_count / tiles);
    const bool whole = a.bn > 160 || (a.bn > 112 && one * tiles * 2 >= d.sm_count);
    int splits = whole || (one >= 1 && a.kblocks <= 8 * one) ? one : two;
    splits = std::max(1, std::min(splits, a.kblocks / 2));
    const int stage = int8_stage_bytes(a.bn);
    for (;; --splits) {
        a.splits = splits;
        const int per_cta = a.kblocks / splits + 1;
        const int room = ((whole ? kI8MaxSmem : 112 * 1024) - kI8RingOff) / stage;
        a.stages = std::max(2, std::min(std::min(kI8MaxStages, per_cta), room));
        // the ring holds the tile's partial sums, or its y, at the end
        a.stages = std::max(a.stages, (a.bn * kI8Rows * 4 + stage - 1) / stage);
        // (32x6144x4096, 48 tiles: 4 and 5 splits 7.3 and 7.9 us, 6, which do not
        // all fit, 12.6)
        if (splits == 1 || resident_clusters(d, splits) * (whole ? 1 : 2) >= tiles) break;
    }
    // The call's time, to be set against the pair kernel's: a fixed part (the
    // outputs, the clusters' meeting) and the stages of a CTA in each wave.
    const int64_t slots = (whole ? 1 : 2) * (int64_t)d.sm_count;
    const int64_t waves = (tiles * splits + slots - 1) / slots;
    const double fixed = splits == 1 ? 4.0 + 0.01 * a.bn : 3.8 + 0.03 * std::min(a.bn, 128) + 0.012 * std::max(a.bn - 128, 0);
    const double stage_us = whole ? std::max(0.25, 0.00125 * a.bn) : tiles * splits > d.sm_count ? 0.42 : 0.25;
    // rows of y that no bulk copy can move (below)
    const bool acc = (p.flags & kInt8Accumulate) != 0;
    const double rows_us = rows_allow_bulk(p) ? 0. : splits == 1 ? (acc ? 4. : 1.) : (acc ? 1. : 0.3);
    *us = fixed + (double)waves * (((a.kblocks + splits - 1) / splits) * stage_us + rows_us);
    return tiles;
}

// Token tile of the pair kernel, a multiple of 32: the one whose rounds of
// the persistent grid cost least.  Below 256 tokens a round gets only a little
// shorter, since issuing and the weights' copies bound it (512x4096x4096, one
// round with 128 / 192 / 256 tokens a tile: 12.0 / 12.9 / 15.0 us).
// 512x11008x4096: 128 tokens, three rounds, 25.4; 192 and 256, two, 21.7 and
// 24.3.  2048x28672x8192: 160 / 192 / 256 tokens 365 / 359 / 323.
int pair_tile(const Int8Args& p, const Int8Device& d, double* us) {
    const int64_t tiles_m = ((int64_t)p.M + 2 * kI8Rows - 1) / (2 * kI8Rows), pairs = d.sm_count / 2;
    int best = kI8MaxBn;
    int64_t cost = INT64_MAX, rounds = 1;
    for (int bn = kI8MaxBn; bn >= 96; bn -= 32) {
        const int64_t r = (tiles_m * (((int64_t)p.T + bn - 1) / bn) + pairs - 1) / pairs;
        if (r * (384 + bn / 2) < cost) {
            cost = r * (384 + bn / 2);
            best = bn;
            rounds = r;
        }
    }
    // (the chunks of a tile wait for their rows of y in turn:
    // 315x149x2209, accumulated in bf16, 14.6 us against 8.9 for the single CTAs)
    const double rows_us = rows_allow_bulk(p) ? 0. : (p.flags & kInt8Accumulate) ? 4. : 1.2;
    *us = 4.0 + (double)rounds * (((p.N + kI8K - 1) / kI8K) * 0.24 + rows_us);
    return best;
}

int run_pairs(const Int8Args& p, const Int8Device& d, int bn, void* stream) {
    Int8PairArgs a = {};
    a.p = p;
    a.kblocks = (p.N + kI8K - 1) / kI8K;
    a.bn = bn;
    a.tiles_t = (int)(((int64_t)p.T + a.bn - 1) / a.bn);
    a.tiles_m = (int)(((int64_t)p.M + 2 * kI8Rows - 1) / (2 * kI8Rows));
    a.tiles = (int64_t)a.tiles_t * a.tiles_m;
    a.test_stall = (p.flags & FLUXBIN_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    a.spin_limit = a.test_stall ? kI8TestSpinLimit : kI8SpinLimit;
    a.err = d.err;
    CUtensorMap mw, mx;
    int st;
    if ((st = encode_rows(&mw, p.w, p.M, p.N, p.ldw, kI8Rows)) != FLUXBIN_OK) return st;
    if ((st = encode_rows(&mx, p.x, p.T, p.N, p.ldx, a.bn / 2)) != FLUXBIN_OK) return st;
    CUtensorMap my = mx;
    if ((st = encode_y(&my, p, int8_pair_chunk((p.flags & kInt8YFp32) ? 4 : 2), &a.bulk)) != FLUXBIN_OK) return st;
    const int64_t pairs = std::min<int64_t>(a.tiles, d.sm_count / 2);
    return launch(pick_int8_pair(p.flags), dim3((unsigned)(2 * pairs)), dim3(kI8PairThreads), (size_t)kI8PairSmem, 1,
                  stream, mw, mx, my, a);
}

// The register kernel: layers of which one wave of its CTAs (two per SM) holds
// all channels and whose K its warps take in one go, or for 8 tokens in two
// (B200, us a call, register / ring kernel; 1 token: 512x4096 2.1 / 3.9,
// 4096x4096 3.9 / 6.0, 4736x8192 8.7 / 8.7, 6976x512 5.0 / 3.7, 2048x16384
// 10.2 / 9.5; 16 tokens: 512x4096 3.1 / 4.2, 4096x4096 5.6 / 6.2, 2048x8192
// 8.5 / 6.6, 6976x4096 10.2 / 7.5).
constexpr int32_t kMvMaxRows = 296 * kMvRows;
constexpr int32_t kMvPass = kMvWarps * kMvBatch * kMvSegment;
bool use_mv(const Int8Args& p) {
    if (p.flags & FLUXBIN_FLAG_TEST_WAIT_TIMEOUT) return false;   // it has no waits
    return p.T <= 2 * kMvTokens && p.M <= kMvMaxRows && p.N <= (p.T <= kMvTokens ? 2 : 1) * kMvPass;
}

int run_int8(const Int8Args& p, void* stream) {
    const bool acc = (p.flags & kInt8Accumulate) != 0;
    if (p.N == 0) {
        const int64_t blocks = ((int64_t)p.T * p.M + 255) / 256;
        if (blocks > INT32_MAX) return FLUXBIN_ERR_UNSUPPORTED;
        Int8EmptyFn fn = (p.flags & kInt8YFp32) ? pick_empty<float>(acc)
                         : (p.flags & kInt8Bf16) ? pick_empty<__nv_bfloat16>(acc) : pick_empty<__half>(acc);
        return launch(fn, dim3((unsigned)blocks), dim3(256), 0, 1, stream, p);
    }
    if (use_mv(p)) {
        const bool two = p.T > kMvTokens;
        Int8EmptyFn fn = (p.flags & kInt8YFp32) ? pick_mv<float>(acc, two)
                         : (p.flags & kInt8Bf16) ? pick_mv<__nv_bfloat16>(acc, two) : pick_mv<__half>(acc, two);
        return launch(fn, dim3((unsigned)((p.M + (int64_t)kMvRows - 1) / kMvRows)), dim3(32 * kMvWarps), 0, 1, stream, p);
    }
    Int8Device d;
    int st = int8_device(&d);
    if (st != FLUXBIN_OK) return st;
    // The kernel whose estimated time is shorter.  Both sides measured (B200,
    // us a call, single / pairs): 128x4096x4096 12.4 / 14.3, 512 tokens 14.3 /
    // 12.9; 256x8192x8192 21.6 / 20.9, 512 tokens 29.2 / 27.4; 512x4096x11008
    // 22.8 / 24.1, 640 tokens 29.1 / 24.6; 160x28672x8192 46.7 / 50.9, 176 tokens
    // 57.1 / 52.7; 128x2048x2048 9.3 / 8.6.
    double us_single = 0., us_pairs = 0.;
    Int8TcArgs a = {};
    a.p = p;
    const int64_t tiles = plan_int8(p, d, &a, &us_single);
    const int pair_bn = pair_tile(p, d, &us_pairs);
    if (us_pairs < us_single) return run_pairs(p, d, pair_bn, stream);
    const int stage = int8_stage_bytes(a.bn), splits = a.splits;
    a.tmem_cols = 32;
    while ((int)a.tmem_cols < a.bn) a.tmem_cols *= 2;
    a.test_stall = (p.flags & FLUXBIN_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    a.spin_limit = a.test_stall ? kI8TestSpinLimit : kI8SpinLimit;
    a.err = d.err;
    if (tiles * splits > INT32_MAX) return FLUXBIN_ERR_UNSUPPORTED;
    CUtensorMap mw, mx;
    if ((st = encode_rows(&mw, p.w, p.M, p.N, p.ldw, kI8Rows)) != FLUXBIN_OK) return st;
    if ((st = encode_rows(&mx, p.x, p.T, p.N, p.ldx, a.bn)) != FLUXBIN_OK) return st;
    CUtensorMap my = mx;
    if (splits == 1 && (st = encode_y(&my, p, kI8OutBox, &a.bulk)) != FLUXBIN_OK) return st;
    return launch(pick_int8_tc(p.flags), dim3((unsigned)(tiles * splits)), dim3(kI8Threads),
                  (size_t)(kI8RingOff + a.stages * stage), splits, stream, mw, mx, my, a);
}

}  // namespace
}  // namespace fluxbin

using namespace fluxbin;

extern "C" {

int fluxbin_quant_rows(int32_t T, int32_t N, const uint16_t* d_x, int64_t ldx, int8_t* d_q, int64_t ldq,
                       float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~FLUXBIN_FLAG_BF16) return FLUXBIN_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || bad_pitch(ldx, N, T, 2) || bad_pitch(ldq, N, T, 1)) return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    return run_quant<kQuantQuant>(Rows{d_x, T, N, ldx, 2}, Rows{nullptr, T, N, 0, 2}, nullptr, 0.f,
                                  Rows{nullptr, T, N, 0, 2}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_silu_mul_quant(int32_t T, int32_t N, const uint16_t* d_gate, int64_t ldg, const uint16_t* d_up,
                           int64_t ldu, int8_t* d_q, int64_t ldq, float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~FLUXBIN_FLAG_BF16) return FLUXBIN_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || bad_pitch(ldg, N, T, 2) || bad_pitch(ldu, N, T, 2) || bad_pitch(ldq, N, T, 1))
        return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    return run_quant<kQuantSilu>(Rows{d_gate, T, N, ldg, 2}, Rows{d_up, T, N, ldu, 2}, nullptr, 0.f,
                                 Rows{nullptr, T, N, 0, 2}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_rmsnorm_quant(int32_t T, int32_t N, const void* d_h, int64_t ldh, const uint16_t* d_delta, int64_t ldd,
                          const uint16_t* d_gamma, float eps, void* d_h_out, int64_t ldo, int8_t* d_q, int64_t ldq,
                          float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~(FLUXBIN_FLAG_BF16 | FLUXBIN_FLAG_H_FP32)) return FLUXBIN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return FLUXBIN_ERR_INVALID_ARG;
    const int hs = (flags & FLUXBIN_FLAG_H_FP32) ? 4 : 2;
    if (T < 0 || N < 0 || bad_pitch(ldh, N, T, hs) || bad_pitch(ldq, N, T, 1) ||
        (d_delta && bad_pitch(ldd, N, T, 2)) || (d_h_out && bad_pitch(ldo, N, T, hs)))
        return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    if (N == 0) return FLUXBIN_ERR_BAD_SHAPE;   // no mean of h^2 to take
    return run_quant<kQuantNorm>(Rows{d_h, T, N, ldh, hs}, Rows{d_delta, T, N, ldd, 2}, d_gamma, eps,
                                 Rows{d_h_out, T, N, ldo, hs}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_int8_linear(int32_t M, int32_t N, const int8_t* d_w, int64_t ldw, const float* d_wscale,
                        const int8_t* d_x, int64_t ldx, const float* d_xscale, int32_t T, void* d_y, int64_t ldy,
                        uint32_t flags, void* stream) {
    if (flags & ~(FLUXBIN_FLAG_ACCUMULATE | FLUXBIN_FLAG_Y_FP32 | FLUXBIN_FLAG_EARLY_WEIGHTS | FLUXBIN_FLAG_BF16 |
                  FLUXBIN_FLAG_TEST_WAIT_TIMEOUT))
        return FLUXBIN_ERR_INVALID_ARG;
    if ((flags & FLUXBIN_FLAG_Y_FP32) && (flags & FLUXBIN_FLAG_BF16)) return FLUXBIN_ERR_INVALID_ARG;
    const int ys = (flags & FLUXBIN_FLAG_Y_FP32) ? 4 : 2;
    if (M < 0 || N < 0 || T < 0 || bad_pitch(ldw, N, M, 1) || bad_pitch(ldx, N, T, 1) || bad_pitch(ldy, M, T, ys))
        return FLUXBIN_ERR_BAD_SHAPE;
    if (N > kInt8MaxN || M > kInt8MaxRows || T > kInt8MaxRows) return FLUXBIN_ERR_UNSUPPORTED;
    if (M == 0 || T == 0) return FLUXBIN_OK;
    if (!d_y || !d_wscale || !d_xscale || (N > 0 && (!d_w || !d_x))) return FLUXBIN_ERR_INVALID_ARG;
    if (!ptr_aligned(d_y, ys) || !ptr_aligned(d_wscale, 4) || !ptr_aligned(d_xscale, 4) || !ptr_aligned(d_w, 16) ||
        !ptr_aligned(d_x, 16) || ldw % 16 || ldx % 16)
        return FLUXBIN_ERR_MISALIGNED;
    const Rows y{d_y, T, M, ldy, ys};
    const Rows ins[4] = {{d_w, M, N, ldw, 1}, {d_x, T, N, ldx, 1}, {d_wscale, 1, M, M, 4}, {d_xscale, 1, T, T, 4}};
    for (const Rows& i : ins)
        if (overlap(y, i)) return FLUXBIN_ERR_INVALID_ARG;
    Int8Args a = {};
    a.w = d_w;
    a.sw = d_wscale;
    a.x = d_x;
    a.sx = d_xscale;
    a.y = d_y;
    a.ldw = ldw;
    a.ldx = ldx;
    a.ldy = ldy;
    a.M = M;
    a.N = N;
    a.T = T;
    a.flags = flags;
    a.vec4 = ptr_aligned(d_y, 4 * ys) && ldy % 4 == 0;
    return run_int8(a, stream);
}

}  // extern "C"
