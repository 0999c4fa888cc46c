// norm_kernel.cuh -- layer norm and RMS norm, forward and backward.
//
//   mu = mean(x) (RMS norm: 0), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r, y = xh w (+ b)
//   dx = r (w dy - mean(w dy) - xh mean(w dy xh)) (RMS norm: without mean(w dy)) (+ add)
//   dw = sum_t dy xh, db = sum_t dy
//
// Both passes are bound by device memory: x is read once (dy and x in the backward), y (dx) written
// once.  A row belongs to a group of threads, NV runs of VEC consecutive elements each.
//
// Rows of 16-byte runs (the row length and the pointers allow it) take the ring kernels: one block per
// SM walks its rows, each group behind a ring of row slots in shared memory that bulk copies fill
// ahead of it, so the bytes in flight depend neither on registers nor on how far a group is in a row's
// arithmetic; weights and the column sums stay in registers; arithmetic is on pairs of binary32
// (the f32x2 instructions), which halves the instructions that issue between two rows.  Other rows
// take scalars (VEC = 1) in registers, and rows too long for those are read again from L1/L2 (NV = 0).
// Either way the variance is taken about the mean in a second pass over data on the SM, not as a
// difference of large sums.
//
// Measured on one GB300 (copy rate 6.78 TB/s), bf16: RMS norm forward 8192 x 5120 29.5 us (5.7 TB/s),
// 32768 x 5120 103 us (6.5 TB/s); layer norm forward 32768 x 4096 96 us (5.6); layer norm backward
// 4096 x 4096 26.6 us (3.8), 32768 x 4096 140 us (5.7), RMS norm backward 32768 x 5120 153 us (6.6).  A
// backward call has some 10 us of its own: two launches, the rings' first and last rows, the columns' join.
// Binary32, 8192 x 4096: RMS norm 43 us forward and 65 backward (6.2 TB/s), layer norm 47 and 75 (5.7, 5.4).
// Rows too long for scalars in registers, 2048 x 5003 bf16: layer norm 39 us forward (1.1), 111 backward (0.6).
// The layer norm's backward arithmetic issues at 0.53 of the schedulers' rate with the 16 warps that its
// registers leave; 32 warps of one run each took longer (32.5 us: more of a row's time in its sums).
//
// dw and db are sums over all tokens of a column.  A thread owns the same columns in every row of its
// group, so they gather in its registers; the groups of a block add up in shared memory, a block
// leaves one row of partial sums, and a second kernel adds the blocks' rows up in their order: no
// atomics, the same bits every time.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "pairs.cuh"
#include "ptx.cuh"
#include "tile_kernel.cuh"

namespace forge {

constexpr int kNormThreads = 512;  // of a block: groups x threads per row, at most
// Slots of a group's ring, at most: two leave the copies too little time, and more than three only put
// more rows in flight than device memory serves well (bf16 RMS norm, width 5120, 32768 tokens: 102 us
// with three slots, 115 with six; width 4096, 4096 tokens: 14.2 us with three, 15.8 with six, 16.3 with two).
constexpr int kNormMaxSlots = 3;

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
    int* status;     // device status word
    uint64_t wait_limit_ns;
    int withhold;    // test switch: no group's first slots are armed or filled, so that waits run out
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

// A 16-byte run of a row in shared memory as pairs, and a run of results to device memory.
template <class TX>
struct Run2 {
    static constexpr int kPairs = 8 / static_cast<int>(sizeof(TX));
    uint32_t w[4];
    __device__ __forceinline__ void load(uint32_t addr) { ld_shared_v4(addr, w); }
    __device__ __forceinline__ F2 get(int i) const {
        if constexpr (sizeof(TX) == 4) return F2::of(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return F2::of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(int i, F2 f) {
        if constexpr (sizeof(TX) == 4) {
            w[2 * i] = __float_as_uint(f.lo());
            w[2 * i + 1] = __float_as_uint(f.hi());
        } else {
            w[i] = pack_bf16x2_rn(__float_as_uint(f.lo()), __float_as_uint(f.hi()));
        }
    }
    __device__ __forceinline__ void store(TX* p) const { st_v4(p, w); }
};

// Weights of a run, as pairs.
template <int PAIRS>
__device__ __forceinline__ void norm_weights2(const void* w, int bf16, int c, F2 (&f)[PAIRS]) {
    float s[2 * PAIRS];
    norm_weights<2 * PAIRS>(w, bf16, c, s);
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) f[i] = F2::of(s[2 * i], s[2 * i + 1]);
}

// Sums over a group (threadIdx.x = 0 .. blockDim.x - 1 of one threadIdx.y; blockDim.x a multiple of
// 32, up to 15 groups of more than one warp).  `slot` alternates between calls, so that one barrier per sum is enough: a slot is written
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
        if (blockDim.x == 32) {
            __syncwarp();
            return make_float2(a, b);
        }
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
    stream_wait();
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
    extern __shared__ float cols[];  // [groups][dw, db]
    stream_wait();
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
        // the groups' columns side by side in shared memory, then one sum over the groups a column
        const int width = CENTER ? 2 * a.D : a.D;
        float* mine = cols + static_cast<size_t>(threadIdx.y) * width;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    mine[first + i * step + j] = dw[i][j];
                    if (CENTER) mine[a.D + first + i * step + j] = db[i][j];
                }
            }
        __syncthreads();
        const int threads = blockDim.x * blockDim.y;
        for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < width; c += threads) {
            float v = cols[c];
            for (int g = 1; g < static_cast<int>(blockDim.y); ++g) v += cols[static_cast<size_t>(g) * width + c];
            if (c < a.D) part_w[c] = v;
            else part_b[c - a.D] = v;
        }
    }
}

// ---------------------------------------------------------------- rings of rows

// One group's ring: `slots` slots of `tensors` rows each, filled by bulk copies that its thread 0
// issues.  Row k of the group is row base + k * stride of the tensors and goes through slot
// k mod slots.
//
// Every wait is bounded.  One that runs out records FORGE_ERR_TIMEOUT and sets the block's abort flag;
// the block's later waits then return at once and its results are void, but every thread still reaches
// every barrier.  A slot whose copies have not landed must not be armed again, so a group whose thread 0 had
// a wait run out issues nothing more, and it waits for what it has issued before its memory is given up.
template <class TX, int TENSORS>
struct NormRing {
    const TX* src[TENSORS];
    uint8_t* mem;
    uint64_t* full;
    int64_t base, stride, rows;
    int slots, D, tensors;
    uint32_t row_bytes;
    int slot;
    uint32_t phase;
    bool ok;  // this thread's waits so far ended with their copies landed

    __device__ __forceinline__ void issue(int64_t k, int at) const {
        mbar_arrive_expect_tx(&full[at], row_bytes * tensors);
        const int64_t el = (base + k * stride) * D;
        uint8_t* dst = mem + static_cast<size_t>(at) * row_bytes * tensors;
#pragma unroll
        for (int i = 0; i < TENSORS; ++i)
            if (i < tensors) bulk_load(dst + i * row_bytes, src[i] + el, row_bytes, &full[at]);
    }
    __device__ __forceinline__ void start() const {
        for (int k = 0; k < slots && k < rows; ++k) issue(k, k);
    }
    // shared-memory address of row k's slot, once its copies have landed
    __device__ __forceinline__ uint32_t wait(const AbortCtx& ab) {
        ok = wait_bounded(&full[slot], phase, ab) && ok;
        return smem_addr(mem) + static_cast<uint32_t>(slot) * row_bytes * tensors;
    }
    // thread 0, where every thread of the group is known to be done with row k - 1
    __device__ __forceinline__ void refill(int64_t k) const {
        if (ok && k > 0 && k - 1 + slots < rows) issue(k - 1 + slots, slot == 0 ? slots - 1 : slot - 1);
    }
    __device__ __forceinline__ void next() {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    // Thread 0 of an aborted block: no copy may be in flight when the block's memory is given up.  Where all rows
    // were issued, each slot's last one is waited for.  Where the ring stopped before, the limit is waited out: a
    // count of the rows issued made calls that abort nothing slower (layer norm, one token 3.33 us against 3.01;
    // backward, 4096 x 4096, 31.2 against 26.4), and without the loop the compiler orders the row loop otherwise
    // (RMS norm backward: 32768 x 5120 169 us against 153, 4096 x 4096 24.4 against 26.1).
    __device__ __forceinline__ void drain(uint64_t limit_ns) const {
        for (int i = 0; i < slots && i < rows; ++i)
            drain_bounded(&full[i], static_cast<uint32_t>(((rows - 1 - i) / slots) & 1), limit_ns);
        if (!ok) wait_out(limit_ns);
    }
};

// Barriers and abort flag of a block, then the group's ring ready to start.
template <class TX, int TENSORS>
__device__ __forceinline__ NormRing<TX, TENSORS> norm_ring(const NormArgs& a, const void* const (&src)[TENSORS], int tensors,
                                                           int slots, uint8_t* mem, uint64_t* bars, int* abort_flag) {
    NormRing<TX, TENSORS> r;
#pragma unroll
    for (int i = 0; i < TENSORS; ++i) r.src[i] = static_cast<const TX*>(src[i]);
    r.row_bytes = static_cast<uint32_t>(a.D) * sizeof(TX);
    r.D = a.D;
    r.tensors = tensors;
    r.slots = slots;
    r.mem = mem + static_cast<size_t>(threadIdx.y) * slots * r.row_bytes * tensors;
    r.full = bars + threadIdx.y * kNormMaxSlots;
    r.base = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    r.stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    r.rows = r.base < a.T ? (a.T - 1 - r.base) / r.stride + 1 : 0;
    r.ok = true;
    r.slot = 0;
    r.phase = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(&r.full[i], 1);
        if (threadIdx.y == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    stream_wait();
    if (threadIdx.x == 0 && a.withhold == 0) r.start();  // its own barriers; the others wait on them past the block's barrier
    __syncthreads();
    return r;
}

template <class TX, int NV, bool CENTER>
__global__ void __launch_bounds__(kNormThreads, 1) forge_norm_ring_kernel(const NormArgs a, const int slots) {
    using Run = Run2<TX>;
    constexpr int kP = Run::kPairs;
    extern __shared__ __align__(128) uint8_t ring_mem[];
    __shared__ float2 buf[2][kNormThreads / 32];
    __shared__ uint64_t bars[kNormThreads / 32 * kNormMaxSlots];
    __shared__ int abort_flag;
    GroupSum sum{buf, 0};
    const void* const src[1] = {a.x};
    NormRing<TX, 1> ring = norm_ring<TX, 1>(a, src, 1, slots, ring_mem, bars, &abort_flag);
    const AbortCtx ab{&abort_flag, a.status, a.wait_limit_ns};
    const float inv = 1.0f / static_cast<float>(a.D);
    const int step = blockDim.x * 2 * kP, first = threadIdx.x * 2 * kP;
    F2 w[NV][kP], b[CENTER ? NV : 1][kP];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.D) {
            norm_weights2<kP>(a.w, a.w_bf16, first + i * step, w[i]);
            if constexpr (CENTER) {
                if (a.b != nullptr) norm_weights2<kP>(a.b, a.w_bf16, first + i * step, b[i]);
                else
#pragma unroll
                    for (int j = 0; j < kP; ++j) b[i][j] = F2::all(0.0f);
            }
        }
    for (int64_t k = 0; k < ring.rows; ++k) {
        const int64_t row = ring.base + k * ring.stride;
        const uint32_t at = ring.wait(ab) + static_cast<uint32_t>(first) * sizeof(TX);
        const uint32_t pitch = static_cast<uint32_t>(step) * sizeof(TX);
        Run v[NV];
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) v[i].load(at + i * pitch);
        if constexpr (CENTER) {
            F2 s = F2::all(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < a.D) {
#pragma unroll
                    for (int j = 0; j < kP; ++j) s = add2(s, v[i].get(j));
                }
            mean = sum(s.lo() + s.hi(), 0.0f).x * inv;
        }
        const F2 less = F2::all(-mean);
        F2 q = F2::all(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 d = CENTER ? add2(v[i].get(j), less) : v[i].get(j);
                    q = fma2(d, d, q);
                }
            }
        const float rstd = 1.0f / sqrtf(fmaf(sum(q.lo() + q.hi(), 0.0f).x, inv, a.eps));
        // past the sum's barrier the whole group has the row in registers
        if (threadIdx.x == 0) ring.refill(k);
        const F2 r2 = F2::all(rstd);
        TX* y = static_cast<TX*>(a.y) + row * a.D + first;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 xh = mul2(CENTER ? add2(v[i].get(j), less) : v[i].get(j), r2);
                    v[i].set(j, CENTER ? fma2(xh, w[i][j], b[i][j]) : mul2(xh, w[i][j]));
                }
                v[i].store(y + i * step);
            }
        if (threadIdx.x == 0) {
            if (CENTER && a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        ring.next();
    }
    if (abort_flag && threadIdx.x == 0) ring.drain(a.wait_limit_ns);
}

template <class TX, int NV, bool CENTER>
__global__ void __launch_bounds__(kNormThreads, 1) forge_norm_bwd_ring_kernel(const NormArgs a, const int slots) {
    using Run = Run2<TX>;
    constexpr int kP = Run::kPairs;
    extern __shared__ __align__(128) uint8_t ring_mem[];
    __shared__ float2 buf[2][kNormThreads / 32];
    __shared__ uint64_t bars[kNormThreads / 32 * kNormMaxSlots];
    __shared__ int abort_flag;
    GroupSum sum{buf, 0};
    const void* const src[3] = {a.dy, a.x, a.add};
    NormRing<TX, 3> ring = norm_ring<TX, 3>(a, src, a.add != nullptr ? 3 : 2, slots, ring_mem, bars, &abort_flag);
    const AbortCtx ab{&abort_flag, a.status, a.wait_limit_ns};
    const float inv = 1.0f / static_cast<float>(a.D);
    const int step = blockDim.x * 2 * kP, first = threadIdx.x * 2 * kP;
    F2 w[NV][kP], dw[NV][kP], db[CENTER ? NV : 1][kP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            dw[i][j] = F2::all(0.0f);
            if constexpr (CENTER) db[i][j] = F2::all(0.0f);
        }
        if (first + i * step < a.D) norm_weights2<kP>(a.w, a.w_bf16, first + i * step, w[i]);
    }
    // a row's mean and rstd are loaded one row ahead
    float mean = 0.0f, rstd = 0.0f;
    if (ring.rows > 0) {
        if (CENTER) mean = a.mean[ring.base];
        rstd = a.rstd[ring.base];
    }
    for (int64_t k = 0; k < ring.rows; ++k) {
        const int64_t row = ring.base + k * ring.stride;
        float mean_next = 0.0f, rstd_next = 0.0f;
        if (k + 1 < ring.rows) {
            if (CENTER) mean_next = a.mean[row + ring.stride];
            rstd_next = a.rstd[row + ring.stride];
        }
        const uint32_t at = ring.wait(ab) + static_cast<uint32_t>(first) * sizeof(TX);
        const uint32_t pitch = static_cast<uint32_t>(step) * sizeof(TX);
        const F2 less = F2::all(-mean), r2 = F2::all(rstd);
        F2 sa = F2::all(0.0f), sb = F2::all(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) {
                Run vd, vx;
                vd.load(at + i * pitch);
                vx.load(at + i * pitch + ring.row_bytes);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 d = vd.get(j), xh = mul2(CENTER ? add2(vx.get(j), less) : vx.get(j), r2);
                    const F2 g = mul2(w[i][j], d);
                    if constexpr (CENTER) sa = add2(sa, g);
                    sb = fma2(g, xh, sb);
                    dw[i][j] = fma2(d, xh, dw[i][j]);
                    if constexpr (CENTER) db[i][j] = add2(db[i][j], d);
                }
            }
        float2 s = sum(sa.lo() + sa.hi(), sb.lo() + sb.hi());
        if (threadIdx.x == 0) ring.refill(k);
        // dx = r (w dy - c1 - xh c2) = (w dy) r + ((x - mu) (-r r c2) - r c1)
        const F2 along = F2::all(-rstd * (rstd * (s.y * inv))), flat = F2::all(-rstd * (s.x * inv));
        TX* dx = static_cast<TX*>(a.dx) + row * a.D + first;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.D) {
                Run vd, vx, va;
                vd.load(at + i * pitch);
                vx.load(at + i * pitch + ring.row_bytes);
                if (a.add != nullptr) va.load(at + i * pitch + 2 * ring.row_bytes);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 t = CENTER ? fma2(add2(vx.get(j), less), along, flat) : mul2(vx.get(j), along);
                    F2 o = fma2(mul2(w[i][j], vd.get(j)), r2, t);
                    if (a.add != nullptr) o = add2(o, va.get(j));
                    vd.set(j, o);
                }
                vd.store(dx + i * step);
            }
        mean = mean_next;
        rstd = rstd_next;
        ring.next();
    }
    if (abort_flag && threadIdx.x == 0) ring.drain(a.wait_limit_ns);
    // the groups' columns side by side in shared memory, then one sum over the groups a column
    __syncthreads();
    float* cols = reinterpret_cast<float*>(ring_mem);
    const int width = CENTER ? 2 * a.D : a.D;
    const uint32_t mine = smem_addr(cols + static_cast<size_t>(threadIdx.y) * width);
    auto put = [&](int c, const F2& p, const F2& q) {
        st_shared_v4(mine + 4u * static_cast<uint32_t>(c), __float_as_uint(p.lo()), __float_as_uint(p.hi()),
                     __float_as_uint(q.lo()), __float_as_uint(q.hi()));
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.D) {
#pragma unroll
            for (int j = 0; j < kP; j += 2) {
                put(first + i * step + 2 * j, dw[i][j], dw[i][j + 1]);
                if constexpr (CENTER) put(a.D + first + i * step + 2 * j, db[i][j], db[i][j + 1]);
            }
        }
    __syncthreads();
    const int threads = blockDim.x * blockDim.y;
    for (int c = 4 * (threadIdx.y * blockDim.x + threadIdx.x); c < width; c += 4 * threads) {
        float4 v = *reinterpret_cast<const float4*>(cols + c);
        for (int g = 1; g < static_cast<int>(blockDim.y); ++g) {
            const float4 u = *reinterpret_cast<const float4*>(cols + static_cast<size_t>(g) * width + c);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        float* out = c < a.D ? a.part + blockIdx.x * a.part_step + c : a.part_b + blockIdx.x * a.part_step + c - a.D;
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = f[j];  // dw and db themselves may start anywhere
    }
}

// dw and db from the blocks' rows: a block takes 32 columns, its 16 warps share the rows, whose loads
// are all in flight at once (a GPU has at most 160 SMs: ten rows a warp).
constexpr int kColumnWarps = 16;
constexpr int kColumnRows = 10;
__global__ void __launch_bounds__(32 * kColumnWarps)
    forge_norm_columns_kernel(const float* part, int64_t step, int blocks, int n, float* dw, float* db, int D) {
    __shared__ float s[kColumnWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // column of the n = D (dw) or 2 D (dw, db) values of a row
    stream_wait();
    float v = 0.0f;
    if (c < n) {
        for (int first = warp; first < blocks; first += kColumnWarps * kColumnRows) {
            float f[kColumnRows];
#pragma unroll
            for (int i = 0; i < kColumnRows; ++i) {
                const int r = first + i * kColumnWarps;
                f[i] = r < blocks ? __ldcg(part + r * step + c) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kColumnRows; ++i) v += f[i];
        }
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < n) {
#pragma unroll
        for (int w = 1; w < kColumnWarps; ++w) v += s[w][lane];
        if (c < D) dw[c] = v;
        else db[c - D] = v;
    }
}

}  // namespace forge
