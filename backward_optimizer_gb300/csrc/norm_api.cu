// norm_api.cu -- the C ABI of the norms (include/forge.h): argument checks, launch shapes, dispatch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "forge.h"
#include "host.h"
#include "norm_kernel.cuh"

namespace {

namespace host = forge::host;
using forge::kNormThreads;
using forge::NormArgs;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

forge_status check_norm(const forge_norm_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->T < 0 || s->T > (1ll << 40) || s->D < 1 || s->D > (1ll << 24)) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->kind != FORGE_NORM_LAYER && s->kind != FORGE_NORM_RMS) return FORGE_ERR_INVALID_ARGUMENT;
    for (int32_t t : {s->x_type, s->w_type})
        if (t != FORGE_TYPE_BF16 && t != FORGE_TYPE_FP32) return FORGE_ERR_INVALID_ARGUMENT;
    return FORGE_OK;
}

// How a row is shared out: `threads` a row, `groups` rows at a time in a block, nv runs of vec elements
// a thread (0: the row does not fit in registers).
struct NormShape {
    int vec, nv, threads, groups;
};

NormShape norm_shape(const forge_norm_shape& s, bool vectors, int most) {
    NormShape n;
    n.vec = vectors ? (s.x_type == FORGE_TYPE_BF16 ? 8 : 4) : 1;
    // scalars take few registers: eight runs of one element cost less than one of eight
    const int nv_most = vectors ? most : 8;
    const int64_t runs = ceil_div(s.D, n.vec);
    n.threads = 32;
    while (n.threads < kNormThreads && runs > 2 * n.threads) n.threads *= 2;
    const int64_t nv = ceil_div(runs, n.threads);
    n.nv = nv > nv_most ? 0 : nv > 4 ? 8 : nv > 2 ? 4 : static_cast<int>(nv);
    n.groups = n.nv == 0 ? 1 : kNormThreads / n.threads;
    return n;
}

template <class TX, int VEC, bool CENTER, bool BWD>
forge_status run_norm_as(const NormArgs& a, const NormShape& n, int blocks, size_t smem, cudaStream_t stream) {
    auto go = [&](auto kernel) {
        kernel<<<blocks, dim3(n.threads, n.groups), smem, stream>>>(a);
        host::count_launch();
        return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
    };
#define FORGE_NORM_CASE(NV)                                                                   \
    case NV:                                                                                  \
        if constexpr (BWD) return go(forge::forge_norm_bwd_kernel<TX, VEC, NV, CENTER>);      \
        else return go(forge::forge_norm_kernel<TX, VEC, NV, CENTER>);
    switch (n.nv) {
        FORGE_NORM_CASE(1)
        FORGE_NORM_CASE(2)
        FORGE_NORM_CASE(4)
        FORGE_NORM_CASE(0)
        case 8:
            if constexpr (VEC == 1) {
                if constexpr (BWD) return go(forge::forge_norm_bwd_kernel<TX, 1, 8, CENTER>);
                else return go(forge::forge_norm_kernel<TX, 1, 8, CENTER>);
            }
    }
#undef FORGE_NORM_CASE
    return FORGE_ERR_UNSUPPORTED;
}

template <bool BWD>
forge_status run_norm(const NormArgs& a, const forge_norm_shape& s, const NormShape& n, int blocks, size_t smem,
                      cudaStream_t stream) {
    const bool center = s.kind == FORGE_NORM_LAYER;
    if (s.x_type == FORGE_TYPE_BF16) {
        if (n.vec == 8)
            return center ? run_norm_as<__nv_bfloat16, 8, true, BWD>(a, n, blocks, smem, stream)
                          : run_norm_as<__nv_bfloat16, 8, false, BWD>(a, n, blocks, smem, stream);
        return center ? run_norm_as<__nv_bfloat16, 1, true, BWD>(a, n, blocks, smem, stream)
                      : run_norm_as<__nv_bfloat16, 1, false, BWD>(a, n, blocks, smem, stream);
    }
    if (n.vec == 4)
        return center ? run_norm_as<float, 4, true, BWD>(a, n, blocks, smem, stream)
                      : run_norm_as<float, 4, false, BWD>(a, n, blocks, smem, stream);
    return center ? run_norm_as<float, 1, true, BWD>(a, n, blocks, smem, stream)
                  : run_norm_as<float, 1, false, BWD>(a, n, blocks, smem, stream);
}

// 16-byte runs need the row length and every pointer to allow them
bool vectors_fit(const forge_norm_shape& s, std::initializer_list<const void*> ps) {
    if (s.D % (s.x_type == FORGE_TYPE_BF16 ? 8 : 4) != 0) return false;
    for (const void* p : ps)
        if (!aligned(p, 16)) return false;
    return true;
}

// every pointer at least on its element's own boundary
bool elements_fit(const forge_norm_shape& s, std::initializer_list<const void*> xs, std::initializer_list<const void*> ws,
                  std::initializer_list<const void*> fs) {
    for (const void* p : xs)
        if (!aligned(p, s.x_type == FORGE_TYPE_BF16 ? 2 : 4)) return false;
    for (const void* p : ws)
        if (!aligned(p, s.w_type == FORGE_TYPE_BF16 ? 2 : 4)) return false;
    for (const void* p : fs)
        if (!aligned(p, 4)) return false;
    return true;
}

int backward_blocks(const forge_norm_shape& s, const NormShape& n, int num_sms) {
    return static_cast<int>(std::min<int64_t>(ceil_div(s.T, n.groups), num_sms));
}

}  // namespace

extern "C" {

forge_status forge_layer_norm(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                              float eps, const forge_norm_shape* shape, struct CUstream_st* stream) {
    forge_status st = check_norm(shape);
    if (st != FORGE_OK) return st;
    const forge_norm_shape& s = *shape;
    if (!(eps >= 0.0f)) return FORGE_ERR_INVALID_ARGUMENT;
    if (s.kind == FORGE_NORM_RMS && (bias != nullptr || mean != nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    if (s.T == 0) return FORGE_OK;
    if (x == nullptr || weight == nullptr || y == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    if (!elements_fit(s, {x, y}, {weight, bias}, {mean, rstd})) return FORGE_ERR_MISALIGNED;
    host::Device dev;
    st = host::device(&dev);
    if (st != FORGE_OK) return st;
    NormArgs a{};
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.w_bf16 = s.w_type == FORGE_TYPE_BF16;
    a.mean = mean;
    a.rstd = rstd;
    a.T = s.T;
    a.D = static_cast<int>(s.D);
    a.eps = eps;
    a.y = y;
    NormShape n = norm_shape(s, vectors_fit(s, {x, weight, bias, y}), 4);
    if (n.nv > 0) n.groups = std::max(1, 128 / n.threads);
    const int blocks = static_cast<int>(std::min<int64_t>(ceil_div(s.T, n.groups), 1 << 20));
    return run_norm<false>(a, s, n, blocks, 0, stream);
}

int64_t forge_layer_norm_backward_workspace(const forge_norm_shape* shape) {
    if (check_norm(shape) != FORGE_OK) return -1;
    if (shape->T == 0) return 0;
    host::Device dev;
    if (host::device(&dev) != FORGE_OK) return -1;
    int64_t most = 0;
    for (bool vectors : {false, true}) {
        const NormShape n = norm_shape(*shape, vectors, 4);
        const int64_t blocks = backward_blocks(*shape, n, dev.num_sms);
        most = std::max(most, blocks > 1 ? blocks * 2 * shape->D * 4 : 0);
    }
    return most;
}

forge_status forge_layer_norm_backward(const void* dy, const void* x, const void* weight, const float* mean,
                                       const float* rstd, const void* add, void* dx, float* dweight, float* dbias,
                                       void* workspace, int64_t workspace_bytes, const forge_norm_shape* shape,
                                       struct CUstream_st* stream) {
    forge_status st = check_norm(shape);
    if (st != FORGE_OK) return st;
    const forge_norm_shape& s = *shape;
    const bool layer = s.kind == FORGE_NORM_LAYER;
    if (dweight == nullptr || layer != (dbias != nullptr) || (!layer && mean != nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    if (!elements_fit(s, {dy, x, add, dx}, {weight}, {mean, rstd, dweight, dbias})) return FORGE_ERR_MISALIGNED;
    if (s.T > 0 && (dy == nullptr || x == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr ||
                    (layer && mean == nullptr)))
        return FORGE_ERR_INVALID_ARGUMENT;
    host::Device dev;
    st = host::device(&dev);
    if (st != FORGE_OK) return st;
    if (s.T == 0) {  // no tokens: the gradients are zero
        if (cudaMemsetAsync(dweight, 0, static_cast<size_t>(s.D) * 4, stream) != cudaSuccess ||
            (layer && cudaMemsetAsync(dbias, 0, static_cast<size_t>(s.D) * 4, stream) != cudaSuccess))
            return FORGE_ERR_CUDA;
        return FORGE_OK;
    }
    NormShape n = norm_shape(s, vectors_fit(s, {dy, x, add, weight, dx}), 4);
    const int blocks = backward_blocks(s, n, dev.num_sms);
    const int64_t width = (layer ? 2 : 1) * s.D;
    if (blocks > 1 && (workspace == nullptr || workspace_bytes < blocks * width * 4)) return FORGE_ERR_INVALID_ARGUMENT;
    if (blocks > 1 && !aligned(workspace, 16)) return FORGE_ERR_MISALIGNED;
    NormArgs a{};
    a.x = x;
    a.w = weight;
    a.w_bf16 = s.w_type == FORGE_TYPE_BF16;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.T = s.T;
    a.D = static_cast<int>(s.D);
    a.dy = dy;
    a.add = add;
    a.dx = dx;
    a.part = blocks > 1 ? static_cast<float*>(workspace) : dweight;
    a.part_b = blocks > 1 ? a.part + s.D : dbias;
    a.part_step = width;
    const size_t smem = n.groups > 1 ? static_cast<size_t>(width) * 4 : 0;
    st = run_norm<true>(a, s, n, blocks, smem, stream);
    if (st != FORGE_OK || blocks == 1) return st;
    forge::forge_norm_columns_kernel<<<static_cast<unsigned>(ceil_div(width, 32)), 256, 0, stream>>>(
        a.part, width, blocks, static_cast<int>(width), dweight, dbias, a.D);
    host::count_launch();
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

}  // extern "C"
