// C-ABI entry points of the 8-bit operators: argument validation, the choice
// of a kernel and the launch.  Declarations and the full contract are in
// include/fluxbin.h.
#include <cmath>
#include <cuda_runtime.h>

#include "../../include/fluxbin.h"
#include "fluxbin_device.h"
#include "fluxbin_int8.cuh"
#include "fluxbin_quant.cuh"

namespace fluxbin {
namespace {

constexpr int32_t kInt8MaxN = 131071;   // 128 * 128 * N < 2^31

constexpr int64_t kMaxPitch = (int64_t)1 << 40;   // beyond any device memory: offsets stay far from 2^63

// A row pitch (in elements) that rows of n elements can have.
bool bad_pitch(int64_t ld, int64_t n) { return ld < n || ld > kMaxPitch; }

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
int launch(K kernel, dim3 grid, dim3 block, size_t smem, void* stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? FLUXBIN_OK : report_cuda_failure(e);
}

using QuantFn = void (*)(QuantArgs);

template <int KIND, typename E, typename H>
QuantFn pick_quant(int vpt, bool vec) {
    if (vec) {
        switch (vpt) {
            case 1: return &fluxbin_quant_kernel<KIND, E, H, 1, true>;
            case 2: return &fluxbin_quant_kernel<KIND, E, H, 2, true>;
            case 4: return &fluxbin_quant_kernel<KIND, E, H, 4, true>;
            default: return &fluxbin_quant_kernel<KIND, E, H, 0, true>;
        }
    }
    switch (vpt) {
        case 1: return &fluxbin_quant_kernel<KIND, E, H, 1, false>;
        case 2: return &fluxbin_quant_kernel<KIND, E, H, 2, false>;
        case 4: return &fluxbin_quant_kernel<KIND, E, H, 4, false>;
        default: return &fluxbin_quant_kernel<KIND, E, H, 0, false>;
    }
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
    // threads of a row: enough for one vector of 8 elements each, up to 1024
    const int64_t vecs = (N + 7) / 8;
    int tpr = 32;
    while (tpr < 1024 && tpr < vecs) tpr *= 2;
    const int64_t per = (vecs + tpr - 1) / tpr;
    const int vpt = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 0;
    const int rpc = tpr >= 128 ? 1 : 128 / tpr;
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
    return launch(fn, dim3((unsigned)((T + rpc - 1) / rpc)), dim3((unsigned)tpr, (unsigned)rpc), 0, stream, a);
}

}  // namespace
}  // namespace fluxbin

using namespace fluxbin;

extern "C" {

int fluxbin_quant_rows(int32_t T, int32_t N, const uint16_t* d_x, int64_t ldx, int8_t* d_q, int64_t ldq,
                       float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~FLUXBIN_FLAG_BF16) return FLUXBIN_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || bad_pitch(ldx, N) || bad_pitch(ldq, N)) return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    return run_quant<kQuantQuant>(Rows{d_x, T, N, ldx, 2}, Rows{nullptr, T, N, 0, 2}, nullptr, 0.f,
                                  Rows{nullptr, T, N, 0, 2}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_silu_mul_quant(int32_t T, int32_t N, const uint16_t* d_gate, int64_t ldg, const uint16_t* d_up,
                           int64_t ldu, int8_t* d_q, int64_t ldq, float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~FLUXBIN_FLAG_BF16) return FLUXBIN_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || bad_pitch(ldg, N) || bad_pitch(ldu, N) || bad_pitch(ldq, N)) return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    return run_quant<kQuantSilu>(Rows{d_gate, T, N, ldg, 2}, Rows{d_up, T, N, ldu, 2}, nullptr, 0.f,
                                 Rows{nullptr, T, N, 0, 2}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_rmsnorm_quant(int32_t T, int32_t N, const void* d_h, int64_t ldh, const uint16_t* d_delta, int64_t ldd,
                          const uint16_t* d_gamma, float eps, void* d_h_out, int64_t ldo, int8_t* d_q, int64_t ldq,
                          float* d_scale, uint32_t flags, void* stream) {
    if (flags & ~(FLUXBIN_FLAG_BF16 | FLUXBIN_FLAG_H_FP32)) return FLUXBIN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return FLUXBIN_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || bad_pitch(ldh, N) || bad_pitch(ldq, N) || (d_delta && bad_pitch(ldd, N)) ||
        (d_h_out && bad_pitch(ldo, N)))
        return FLUXBIN_ERR_BAD_SHAPE;
    if (T == 0) return FLUXBIN_OK;
    if (N == 0) return FLUXBIN_ERR_BAD_SHAPE;   // no mean of h^2 to take
    const int hs = (flags & FLUXBIN_FLAG_H_FP32) ? 4 : 2;
    return run_quant<kQuantNorm>(Rows{d_h, T, N, ldh, hs}, Rows{d_delta, T, N, ldd, 2}, d_gamma, eps,
                                 Rows{d_h_out, T, N, ldo, hs}, d_q, ldq, d_scale, flags, stream);
}

int fluxbin_int8_linear(int32_t M, int32_t N, const int8_t* d_w, int64_t ldw, const float* d_wscale,
                        const int8_t* d_x, int64_t ldx, const float* d_xscale, int32_t T, void* d_y, int64_t ldy,
                        uint32_t flags, void* stream) {
    if (flags & ~(FLUXBIN_FLAG_ACCUMULATE | FLUXBIN_FLAG_Y_FP32 | FLUXBIN_FLAG_EARLY_WEIGHTS | FLUXBIN_FLAG_BF16))
        return FLUXBIN_ERR_INVALID_ARG;
    if ((flags & FLUXBIN_FLAG_Y_FP32) && (flags & FLUXBIN_FLAG_BF16)) return FLUXBIN_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || T < 0 || bad_pitch(ldw, N) || bad_pitch(ldx, N) || bad_pitch(ldy, M))
        return FLUXBIN_ERR_BAD_SHAPE;
    if (N > kInt8MaxN) return FLUXBIN_ERR_UNSUPPORTED;
    if (M == 0 || T == 0) return FLUXBIN_OK;
    if (!d_y || !d_wscale || !d_xscale || (N > 0 && (!d_w || !d_x))) return FLUXBIN_ERR_INVALID_ARG;
    const int ys = (flags & FLUXBIN_FLAG_Y_FP32) ? 4 : 2;
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
    const int64_t tm = ((int64_t)M + kInt8Tile - 1) / kInt8Tile, tt = ((int64_t)T + kInt8Tile - 1) / kInt8Tile;
    if (tt > 65535) return FLUXBIN_ERR_UNSUPPORTED;
    return launch(&fluxbin_int8_kernel, dim3((unsigned)tm, (unsigned)tt), dim3(256), 0, stream, a);
}

}  // extern "C"
