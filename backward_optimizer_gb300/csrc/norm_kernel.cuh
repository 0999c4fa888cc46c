// norm_kernel.cuh -- layer norm and RMS norm, forward and backward.
//
//   mu = mean(x) (RMS norm: 0), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r, y = xh w (+ b)
//   dx = r (w dy - mean(w dy) - xh mean(w dy xh)) (RMS norm: without mean(w dy)) (+ add)
//   dw = sum_t dy xh, db = sum_t dy
//
// Both passes are bound by device memory: x is read once (dy and x in the backward), y (dx) written
// once.  A row belongs to a group of threads that keeps it in registers between the row's sums and
// its result, NV runs of VEC consecutive elements each, so the variance is taken about the mean in a
// second pass over registers, not as a difference of large sums.  VEC fills 16 bytes where the row
// length and the pointers allow it, else it is 1.  Rows too long for registers are read again from
// L1/L2 (NV = 0).
//
// dw and db are sums over all tokens of a column.  A thread owns the same columns in every row of its
// group, so they gather in its registers; the groups of a block add up in shared memory, a block
// leaves one row of partial sums, and a second kernel adds the blocks' rows up in their order: no
// atomics, the same bits every time.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"

namespace forge {

constexpr int kNormThreads = 512;  // of a block: groups x threads per row

struct NormArgs {
    const void* x;
    const void* w;   // [D], binary32 or bfloat16
    const void* b;   // [D] or null, same type
    int w_bf16;
    float* mean;     // [T]; null for RMS norm
    float* rstd;     // [T]
    int64_t T;
    int D;
    float eps;
    void* y;         // forward
    const void* dy;  // backward
    const void* add;
    void* dx;
    float* part;     // [blocks][2][D], or dw and db themselves when there is one block
    float* part_b;
    int64_t part_step;
};

// VEC elements of type TX as they lie in memory
template <class TX, int VEC>
struct NormVec {
    static constexpr int kWords = VEC * static_cast<int>(sizeof(TX)) / 4 > 0 ? VEC * static_cast<int>(sizeof(TX)) / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const TX* p) {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(TX) == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
            else w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            static_assert(kWords == 4, "16 bytes");
            ld_v4(p, w);
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(TX) == 4) return __uint_as_float(w[j]);
        else if constexpr (VEC == 1) return __uint_as_float(w[0] << 16);
        else return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    }
};

template <class TX, int VEC>
__device__ __forceinline__ void norm_store(TX* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(TX) == 2) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f[0]);
        else *reinterpret_cast<float*>(p) = f[0];
    } else {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TX) == 2) r[i] = pack_bf16x2_rn(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
            else r[i] = __float_as_uint(f[i]);
        }
        st_v4(p, r);
    }
}

// VEC weights from column c
template <int VEC>
__device__ __forceinline__ void norm_weights(const void* w, int bf16, int c, float (&f)[VEC]) {
    if (bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(w) + c;
        if constexpr (VEC == 8) {
            uint32_t r[4];
            ld_v4(p, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float((j & 1) ? r[j >> 1] & 0xFFFF0000u : r[j >> 1] << 16);
        } else if constexpr (VEC == 4) {
            uint32_t r[2];
            ld_v2(p, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = __uint_as_float((j & 1) ? r[j >> 1] & 0xFFFF0000u : r[j >> 1] << 16);
        } else {
            f[0] = __uint_as_float(static_cast<uint32_t>(*p) << 16);
        }
    } else {
        const float* p = static_cast<const float*>(w) + c;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                uint32_t r[4];
                ld_v4(p + 4 * q, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * q + j] = __uint_as_float(r[j]);
            }
        } else {
            f[0] = *p;
        }
    }
}

// Sums over a group (threadIdx.x = 0 .. blockDim.x - 1 of one threadIdx.y; blockDim.x a multiple of
// 32).  `slot` alternates between calls, so that one barrier per sum is enough: a slot is written
// again only after the barrier of the call between.
struct GroupSum {
    float2 (*buf)[kNormThreads / 32];  // [2][warps of the block]
    int slot;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (blockDim.x == 32) return make_float2(a, b);
        const int warps = blockDim.x >> 5, first = threadIdx.y * warps;
        float2* s = buf[slot];
        slot ^= 1;
        if ((threadIdx.x & 31) == 0) s[first + (threadIdx.x >> 5)] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(static_cast<int>(blockDim.x)) : "memory");
        a = b = 0.0f;
        for (int i = 0; i < warps; ++i) {
            a += s[first + i].x;
            b += s[first + i].y;
        }
        return make_float2(a, b);
    }
};

// ---------------------------------------------------------------- forward

template <class TX, int VEC, int NV, bool CENTER>
__global__ void __launch_bounds__(kNormThreads) forge_norm_kernel(const NormArgs a) {
    __shared__ float2 buf[2][kNormThreads / 32];
    GroupSum sum{buf, 0};
    const float inv = 1.0f / static_cast<float>(a.D);
    const int step = blockDim.x * VEC;
    const int first = threadIdx.x * VEC;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.T;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y) {
        const TX* x = static_cast<const TX*>(a.x) + row * a.D;
        TX* y = static_cast<TX*>(a.y) + row * a.D;
        float mean = 0.0f, rstd;
        if constexpr (NV > 0) {
            NormVec<TX, VEC> v[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) v[i].load(x + first + i * step);
            if constexpr (CENTER) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (first + i * step < a.D) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) s += v[i].get(j);
                    }
                mean = sum(s, 0.0f).x * inv;
            }
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = v[i].get(j) - mean;
                        q = fmaf(d, d, q);
                    }
                }
            rstd = 1.0f / sqrtf(fmaf(sum(q, 0.0f).x, inv, a.eps));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = first + i * step;
                if (c < a.D) {
                    float w[VEC], b[VEC], o[VEC];
                    norm_weights<VEC>(a.w, a.w_bf16, c, w);
                    if (a.b != nullptr) norm_weights<VEC>(a.b, a.w_bf16, c, b);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        o[j] = (v[i].get(j) - mean) * rstd * w[j];
                        if (a.b != nullptr) o[j] += b[j];
                    }
                    norm_store<TX, VEC>(y + c, o);
                }
            }
        } else {
            if constexpr (CENTER) {
                float s = 0.0f;
                for (int c = first; c < a.D; c += step) {
                    NormVec<TX, VEC> v;
                    v.load(x + c);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s += v.get(j);
                }
                mean = sum(s, 0.0f).x * inv;
            }
            float q = 0.0f;
            for (int c = first; c < a.D; c += step) {
                NormVec<TX, VEC> v;
                v.load(x + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) q = fmaf(v.get(j) - mean, v.get(j) - mean, q);
            }
            rstd = 1.0f / sqrtf(fmaf(sum(q, 0.0f).x, inv, a.eps));
            for (int c = first; c < a.D; c += step) {
                NormVec<TX, VEC> v;
                v.load(x + c);
                float w[VEC], b[VEC], o[VEC];
                norm_weights<VEC>(a.w, a.w_bf16, c, w);
                if (a.b != nullptr) norm_weights<VEC>(a.b, a.w_bf16, c, b);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    o[j] = (v.get(j) - mean) * rstd * w[j];
                    if (a.b != nullptr) o[j] += b[j];
                }
                norm_store<TX, VEC>(y + c, o);
            }
        }
        if (threadIdx.x == 0) {
            if (CENTER && a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
    }
}

// ---------------------------------------------------------------- backward

template <class TX, int VEC, int NV, bool CENTER>
__global__ void __launch_bounds__(kNormThreads) forge_norm_bwd_kernel(const NormArgs a) {
    __shared__ float2 buf[2][kNormThreads / 32];
    extern __shared__ float cols[];  // [2][D], where a block has several groups
    GroupSum sum{buf, 0};
    const float inv = 1.0f / static_cast<float>(a.D);
    const int step = blockDim.x * VEC;
    const int first = threadIdx.x * VEC;
    float* part_w = a.part + blockIdx.x * a.part_step;
    float* part_b = CENTER ? a.part_b + blockIdx.x * a.part_step : nullptr;
    constexpr int kN = NV > 0 ? NV : 1;
    float dw[kN][VEC], db[kN][VEC];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
    bool fresh = true;  // NV = 0: the block's row of partial sums is not written yet
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.T; row += stride) {
        const TX* x = static_cast<const TX*>(a.x) + row * a.D;
        const TX* dy = static_cast<const TX*>(a.dy) + row * a.D;
        const TX* add = a.add == nullptr ? nullptr : static_cast<const TX*>(a.add) + row * a.D;
        TX* dx = static_cast<TX*>(a.dx) + row * a.D;
        const float mean = CENTER ? a.mean[row] : 0.0f, rstd = a.rstd[row];
        auto result = [&](const NormVec<TX, VEC>& vx, const NormVec<TX, VEC>& vd, int c, float2 s) {
            float w[VEC], o[VEC];
            norm_weights<VEC>(a.w, a.w_bf16, c, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (vx.get(j) - mean) * rstd;
                o[j] = rstd * (w[j] * vd.get(j) - (CENTER ? s.x : 0.0f) - xh * s.y);
            }
            if (add != nullptr) {
                NormVec<TX, VEC> r;
                r.load(add + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[j] += r.get(j);
            }
            norm_store<TX, VEC>(dx + c, o);
        };
        auto gather = [&](const NormVec<TX, VEC>& vx, const NormVec<TX, VEC>& vd, int c, float& sa, float& sb,
                          float (&cw)[VEC], float (&cb)[VEC]) {
            float w[VEC];
            norm_weights<VEC>(a.w, a.w_bf16, c, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = vd.get(j), xh = (vx.get(j) - mean) * rstd, g = w[j] * d;
                if (CENTER) sa += g;
                sb = fmaf(g, xh, sb);
                cw[j] = fmaf(d, xh, cw[j]);
                if (CENTER) cb[j] += d;
            }
        };
        float sa = 0.0f, sb = 0.0f;
        if constexpr (NV > 0) {
            NormVec<TX, VEC> vx[kN], vd[kN];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) {
                    vd[i].load(dy + first + i * step);
                    vx[i].load(x + first + i * step);
                }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) gather(vx[i], vd[i], first + i * step, sa, sb, dw[i], db[i]);
            float2 s = sum(sa, sb);
            s.x *= inv;
            s.y *= inv;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) result(vx[i], vd[i], first + i * step, s);
        } else {
            // one group per block: its partial sums are carried in its own row of memory
            for (int c = first; c < a.D; c += step) {
                NormVec<TX, VEC> vx, vd;
                vx.load(x + c);
                vd.load(dy + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    dw[0][j] = fresh ? 0.0f : part_w[c + j];
                    if (CENTER) db[0][j] = fresh ? 0.0f : part_b[c + j];
                }
                gather(vx, vd, c, sa, sb, dw[0], db[0]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    part_w[c + j] = dw[0][j];
                    if (CENTER) part_b[c + j] = db[0][j];
                }
            }
            fresh = false;
            float2 s = sum(sa, sb);
            s.x *= inv;
            s.y *= inv;
            for (int c = first; c < a.D; c += step) {
                NormVec<TX, VEC> vx, vd;
                vx.load(x + c);
                vd.load(dy + c);
                result(vx, vd, c, s);
            }
        }
    }
    if constexpr (NV > 0) {
        // the groups of the block add their columns up one after another
        for (int g = 1; g < static_cast<int>(blockDim.y); ++g) {
            __syncthreads();
            if (static_cast<int>(threadIdx.y) == g) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (first + i * step < a.D) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            cols[first + i * step + j] = dw[i][j];
                            if (CENTER) cols[a.D + first + i * step + j] = db[i][j];
                        }
                    }
            }
            __syncthreads();
            if (threadIdx.y == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (first + i * step < a.D) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            dw[i][j] += cols[first + i * step + j];
                            if (CENTER) db[i][j] += cols[a.D + first + i * step + j];
                        }
                    }
            }
        }
        if (threadIdx.y == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        part_w[first + i * step + j] = dw[i][j];
                        if (CENTER) part_b[first + i * step + j] = db[i][j];
                    }
                }
        }
    }
}

// dw and db from the blocks' rows: a block takes 32 columns, its 8 warps share the rows.
__global__ void __launch_bounds__(256)
    forge_norm_columns_kernel(const float* part, int64_t step, int blocks, int n, float* dw, float* db, int D) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // column of the n = D (dw) or 2 D (dw, db) values of a row
    float v = 0.0f;
    if (c < n) {
#pragma unroll 4
        for (int r = warp; r < blocks; r += 8) v += part[r * step + c];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < n) {
        for (int w = 1; w < 8; ++w) v += s[w][lane];
        if (c < D) dw[c] = v;
        else db[c - D] = v;
    }
}

}  // namespace forge
