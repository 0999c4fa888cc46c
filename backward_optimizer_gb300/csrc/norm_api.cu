// norm_api.cu -- the C ABI of the norms (include/forge.h): argument checks, launch shapes, dispatch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

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

NormShape norm_shape(const forge_norm_shape& s, bool vectors, bool backward) {
    NormShape n;
    n.vec = vectors ? (s.x_type == FORGE_TYPE_BF16 ? 8 : 4) : 1;
    const int64_t runs = ceil_div(s.D, n.vec);
    // Four 16-byte runs a thread, eight scalars: longer runs mean fewer threads in a row's sums.  The
    // layer norm's backward pass holds a weight and two column sums per element, and four runs of them
    // spill at 512 threads: it takes two or three, whichever keeps more of the block's threads at work
    // (bf16, 4096 tokens: width 4096 28.7 us with two, 35.3 with four; width 5120 37.5 us with three, 40.6
    // with two; the RMS norm 24.9 us with four, 30.1 with two).
    auto shape = [&](int most) {
        n.threads = static_cast<int>(std::min<int64_t>(ceil_div(runs, 32 * most) * 32, kNormThreads));
        const int64_t nv = ceil_div(runs, n.threads);
        n.nv = nv > (vectors ? 4 : 8) ? 0 : nv > 4 ? 8 : static_cast<int>(nv);
        n.groups = n.nv == 0 ? 1 : kNormThreads / n.threads;
    };
    shape(vectors ? 4 : 8);
    if (vectors && backward && s.kind == FORGE_NORM_LAYER && n.nv > 2) {
        const NormShape four = n;
        shape(3);
        const NormShape three = n;
        shape(2);
        // runs at work at once, per run of a thread; rows too long for three runs a thread keep four
        auto busy = [&](const NormShape& m) { return m.groups * runs * (m.nv == 2 ? 3 : 2); };
        if (three.nv != 3 && n.nv != 2) n = four;
        else if (n.nv != 2 || (three.nv == 3 && busy(three) > busy(n))) n = three;
    }
    return n;
}

// Shared memory of the rings; the rest is the block's own few KB of static memory.
constexpr int64_t kRingBytes = 200 * 1024;

// Slots of each group's ring: what the groups' shares hold (0: the row is not made of 16-byte runs, or
// too long for registers; those that fit there always leave two slots).
int ring_slots(const forge_norm_shape& s, const NormShape& n, int tensors) {
    if (n.vec == 1 || n.nv == 0) return 0;
    const int64_t slot = s.D * (s.x_type == FORGE_TYPE_BF16 ? 2 : 4) * tensors;
    return static_cast<int>(std::min<int64_t>(kRingBytes / n.groups / slot, forge::kNormMaxSlots));
}

// slots: of the rings, or 0 for the kernels without them
template <class TX, int VEC, bool CENTER, bool BWD>
forge_status run_norm_as(const NormArgs& a, const NormShape& n, int blocks, size_t smem, int slots,
                         cudaStream_t stream) {
    auto go = [&](auto kernel) {
        return host::launch_early(kernel, dim3(blocks), dim3(n.threads, n.groups), smem, stream, a) == cudaSuccess
                   ? FORGE_OK
                   : FORGE_ERR_CUDA;
    };
    if constexpr (VEC > 1) {
        auto ring = [&](auto kernel) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
                return FORGE_ERR_CUDA;
            return host::launch_early(kernel, dim3(blocks), dim3(n.threads, n.groups), smem, stream, a, slots) ==
                           cudaSuccess
                       ? FORGE_OK
                       : FORGE_ERR_CUDA;
        };
        auto pick = [&](auto nv) {
            if constexpr (BWD) return ring(forge::forge_norm_bwd_ring_kernel<TX, nv.value, CENTER>);
            else return ring(forge::forge_norm_ring_kernel<TX, nv.value, CENTER>);
        };
        switch (slots > 0 ? n.nv : 0) {
            case 1: return pick(std::integral_constant<int, 1>{});
            case 2: return pick(std::integral_constant<int, 2>{});
            case 3: return pick(std::integral_constant<int, 3>{});
            case 4: return pick(std::integral_constant<int, 4>{});
        }
    }
#define FORGE_NORM_CASE(NV, REACHED)                                                          \
    case NV:                                                                                  \
        if constexpr (REACHED) {                                                              \
            if constexpr (BWD) return go(forge::forge_norm_bwd_kernel<TX, VEC, NV, CENTER>);  \
            else return go(forge::forge_norm_kernel<TX, VEC, NV, CENTER>);                    \
        }                                                                                     \
        break;
    switch (n.nv) {
        FORGE_NORM_CASE(1, VEC == 1)
        FORGE_NORM_CASE(2, VEC == 1)
        FORGE_NORM_CASE(3, VEC == 1)
        FORGE_NORM_CASE(4, VEC == 1)
        FORGE_NORM_CASE(8, VEC == 1)
        FORGE_NORM_CASE(0, true)
    }
#undef FORGE_NORM_CASE
    return FORGE_ERR_UNSUPPORTED;
}

template <bool BWD>
forge_status run_norm(const NormArgs& a, const forge_norm_shape& s, const NormShape& n, int blocks, size_t smem,
                      int slots, cudaStream_t stream) {
    const bool center = s.kind == FORGE_NORM_LAYER;
    if (s.x_type == FORGE_TYPE_BF16) {
        if (n.vec == 8)
            return center ? run_norm_as<__nv_bfloat16, 8, true, BWD>(a, n, blocks, smem, slots, stream)
                          : run_norm_as<__nv_bfloat16, 8, false, BWD>(a, n, blocks, smem, slots, stream);
        return center ? run_norm_as<__nv_bfloat16, 1, true, BWD>(a, n, blocks, smem, slots, stream)
                      : run_norm_as<__nv_bfloat16, 1, false, BWD>(a, n, blocks, smem, slots, stream);
    }
    if (n.vec == 4)
        return center ? run_norm_as<float, 4, true, BWD>(a, n, blocks, smem, slots, stream)
                      : run_norm_as<float, 4, false, BWD>(a, n, blocks, smem, slots, stream);
    return center ? run_norm_as<float, 1, true, BWD>(a, n, blocks, smem, slots, stream)
                  : run_norm_as<float, 1, false, BWD>(a, n, blocks, smem, slots, stream);
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

// Blocks that walk rows: one per SM, and no more groups than there are rows for.
int norm_blocks(const forge_norm_shape& s, NormShape& n, int num_sms) {
    const int blocks = static_cast<int>(std::min<int64_t>(s.T, num_sms));
    n.groups = static_cast<int>(std::min<int64_t>(n.groups, ceil_div(s.T, blocks)));
    return blocks;
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
    a.status = dev.status;
    a.wait_limit_ns = host::wait_limit_ns();
    NormShape n = norm_shape(s, vectors_fit(s, {x, weight, bias, y}), false);
    const int slots = ring_slots(s, n, 1);
    if (slots > 0) {
        a.withhold = host::take_withhold();
        const int blocks = norm_blocks(s, n, dev.num_sms);
        const int64_t smem = n.groups * slots * s.D * (s.x_type == FORGE_TYPE_BF16 ? 2 : 4);
        return run_norm<false>(a, s, n, blocks, static_cast<size_t>(smem), slots, stream);
    }
    if (n.nv > 0) n.groups = std::max(1, 128 / n.threads);
    const int blocks = static_cast<int>(std::min<int64_t>(ceil_div(s.T, n.groups), 1 << 20));
    return run_norm<false>(a, s, n, blocks, 0, 0, stream);
}

int64_t forge_layer_norm_backward_workspace(const forge_norm_shape* shape) {
    if (check_norm(shape) != FORGE_OK) return -1;
    if (shape->T == 0) return 0;
    host::Device dev;
    if (host::device(&dev) != FORGE_OK) return -1;
    const int64_t blocks = std::min<int64_t>(shape->T, dev.num_sms);
    return blocks > 1 ? blocks * 2 * shape->D * 4 : 0;
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
    NormShape n = norm_shape(s, vectors_fit(s, {dy, x, add, weight, dx}), true);
    const int blocks = norm_blocks(s, n, dev.num_sms);
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
    a.status = dev.status;
    a.wait_limit_ns = host::wait_limit_ns();
    const int slots = ring_slots(s, n, add != nullptr ? 3 : 2);
    if (slots > 0) a.withhold = host::take_withhold();
    // the rings, and after them the groups' columns
    const int64_t slot_bytes = s.D * (s.x_type == FORGE_TYPE_BF16 ? 2 : 4) * (add != nullptr ? 3 : 2);
    const int64_t smem = n.nv == 0 ? 0 : std::max(n.groups * slots * slot_bytes, n.groups * width * 4);
    st = run_norm<true>(a, s, n, blocks, static_cast<size_t>(smem), slots, stream);
    if (st != FORGE_OK || blocks == 1) return st;
    return host::launch_early(forge::forge_norm_columns_kernel, dim3(static_cast<unsigned>(ceil_div(width, 32))),
                              dim3(32 * forge::kColumnWarps), 0, stream, a.part, width, blocks,
                              static_cast<int>(width), dweight, dbias, a.D) == cudaSuccess
               ? FORGE_OK
               : FORGE_ERR_CUDA;
}

}  // extern "C"
