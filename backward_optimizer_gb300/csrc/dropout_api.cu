// dropout_api.cu -- the C ABI of dropout from a counter (include/forge.h), and its kernel.
//
// y[e] = (residual[e] +) x[e] s where element e is kept, (residual[e]) + 0 where it is dropped.  Whether it is comes
// from the framework's generator (Philox4x32-10, opt_math.cuh) at a counter that e and the step make up, so the
// backward pass makes the same mask again and none is ever stored.  One call of the generator serves eight
// elements, 16 bits each: element e is dropped where its number is below p 2^16 (rounded), and s is
// 2^16 / (2^16 - that number), so that the expectation is x[e] exactly, whatever p was rounded to.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "forge.h"
#include "host.h"
#include "opt_math.cuh"
#include "ptx.cuh"

namespace {

namespace host = forge::host;

constexpr int kThreads = 256;
constexpr int kGroups = 4;  // groups of eight elements that a thread has in flight

struct DropArgs {
    const void* x;
    const void* residual;
    void* y;
    int64_t n;
    uint64_t seed, step;
    const int64_t* step_at;
    uint32_t below;  // elements with a number below it are dropped
    float scale;
};

// Bit i of the result: element i of the group is kept.
__device__ __forceinline__ uint32_t kept_of(int64_t group, uint64_t seed, uint64_t step, uint32_t below) {
    const forge::Philox4 r = forge::sr_words(static_cast<uint64_t>(group), seed, step, forge::kStreamDropout);
    const uint32_t w[4] = {r.x0, r.x1, r.x2, r.x3};
    uint32_t kept = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        kept |= ((w[i] & 0xFFFFu) >= below ? 1u : 0u) << (2 * i);
        kept |= ((w[i] >> 16) >= below ? 2u : 0u) << (2 * i);
    }
    return kept;
}

// A dropped element adds nothing, not 0 times its value: an infinite x that is dropped leaves no NaN.
__device__ __forceinline__ float one(float x, bool kept, float scale, float r) { return kept ? __fmaf_rn(x, scale, r) : r; }

__device__ __forceinline__ float load(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load(const uint16_t* p, int64_t i) { return __uint_as_float(static_cast<uint32_t>(p[i]) << 16); }
__device__ __forceinline__ void store(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store(uint16_t* p, int64_t i, float v) {
    p[i] = static_cast<uint16_t>(forge::pack_bf16x2_rn(__float_as_uint(v), 0u));
}

// kWords: 32-bit words of a group of eight: 4 (bfloat16) or 8 (binary32).  kVector: every pointer is a multiple of 16;
// otherwise element by element (8192 x 5120 with residual, us, vectors / elements: bfloat16 38 / 110, binary32 72 / 178).
template <class T, bool kVector, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    constexpr int kWords = 8 * sizeof(T) / 4;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    T* y = static_cast<T*>(a.y);
    const int64_t whole = a.n / 8;  // whole groups
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kGroups) + threadIdx.x;
    forge::stream_wait();
    const uint64_t step = a.step_at != nullptr ? static_cast<uint64_t>(__ldcg(a.step_at)) : a.step;
    if constexpr (kVector) {
        uint32_t v[kGroups][kWords], r[kGroups][kWords];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t g = first + i * kThreads;
            if (g < whole) {
#pragma unroll
                for (int h = 0; h < kWords / 4; ++h) {
                    forge::ld_v4(x + 8 * g + h * (16 / sizeof(T)), *reinterpret_cast<uint32_t(*)[4]>(&v[i][4 * h]));
                    if (kResidual)
                        forge::ld_v4(res + 8 * g + h * (16 / sizeof(T)), *reinterpret_cast<uint32_t(*)[4]>(&r[i][4 * h]));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t g = first + i * kThreads;
            if (g >= whole) break;
            const uint32_t kept = kept_of(g, a.seed, step, a.below);
            uint32_t o[kWords];
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                if constexpr (sizeof(T) == 2) {
                    const float lo = one(forge::bf16_lo(v[i][j]), kept >> (2 * j) & 1, a.scale, kResidual ? forge::bf16_lo(r[i][j]) : 0.0f);
                    const float hi = one(forge::bf16_hi(v[i][j]), kept >> (2 * j + 1) & 1, a.scale, kResidual ? forge::bf16_hi(r[i][j]) : 0.0f);
                    o[j] = forge::pack_bf16x2_rn(__float_as_uint(lo), __float_as_uint(hi));
                } else {
                    o[j] = __float_as_uint(one(__uint_as_float(v[i][j]), kept >> j & 1, a.scale, kResidual ? __uint_as_float(r[i][j]) : 0.0f));
                }
            }
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h)
                forge::st_v4(y + 8 * g + h * (16 / sizeof(T)), *reinterpret_cast<uint32_t(*)[4]>(&o[4 * h]));
        }
    }
    // what no vector takes: the last group, or every one
    for (int i = 0; i < kGroups; ++i) {
        const int64_t g = first + i * kThreads;
        if (8 * g >= a.n) break;
        if (kVector && g < whole) continue;
        const uint32_t kept = kept_of(g, a.seed, step, a.below);
        const int left = static_cast<int>(a.n - 8 * g < 8 ? a.n - 8 * g : 8);
        for (int j = 0; j < left; ++j)
            store(y, 8 * g + j, one(load(x, 8 * g + j), kept >> j & 1, a.scale, kResidual ? load(res, 8 * g + j) : 0.0f));
    }
}

template <class T>
cudaError_t launch(const DropArgs& a, bool vector, cudaStream_t stream) {
    const int64_t per = 8ll * kThreads * kGroups;
    const dim3 grid(static_cast<unsigned>((a.n + per - 1) / per)), block(kThreads);
    auto kernel = vector ? (a.residual ? dropout_kernel<T, true, true> : dropout_kernel<T, true, false>)
                         : (a.residual ? dropout_kernel<T, false, true> : dropout_kernel<T, false, false>);
    return host::launch_early(kernel, grid, block, 0, stream, a);
}

}  // namespace

extern "C" forge_status forge_dropout(const void* x, const void* residual, void* y, int64_t n, int32_t type, double p,
                                      uint64_t seed, uint64_t step, const int64_t* step_at, struct CUstream_st* stream) {
    if (n < 0 || n > (1ll << 42) || (type != FORGE_TYPE_BF16 && type != FORGE_TYPE_FP32)) return FORGE_ERR_INVALID_ARGUMENT;
    if (!(p >= 0.0 && p <= 1.0)) return FORGE_ERR_INVALID_ARGUMENT;
    if (n == 0) return FORGE_OK;
    if (x == nullptr || y == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(y);
    if (all % (type == FORGE_TYPE_BF16 ? 2 : 4) != 0 || reinterpret_cast<uintptr_t>(step_at) % 8 != 0) return FORGE_ERR_MISALIGNED;
    host::Device dev;
    const forge_status st = host::device(&dev);
    if (st != FORGE_OK) return st;
    DropArgs a{x, residual, y, n, seed, step, step_at, 0, 0.0f};
    a.below = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    a.scale = a.below < 65536u ? static_cast<float>(65536.0 / (65536.0 - a.below)) : 0.0f;
    const cudaError_t err = type == FORGE_TYPE_BF16 ? launch<uint16_t>(a, all % 16 == 0, stream) : launch<float>(a, all % 16 == 0, stream);
    return err == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
