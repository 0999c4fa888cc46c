// rows_kernel.cuh -- the product of one token with a weight matrix: y[n] = sum_k x[k] W[n, k].
//
// Every weight is read once and used once, so the time is the weights' way from memory.  The tensor core's
// 128-row tiles would be almost empty, and the splitting and joining along k that few tiles need costs
// more than the products.  Here a block stays on its SM and walks groups of weight rows through a ring of
// bulk copies (whole rows, contiguous in memory, up to 200 KB in flight per SM).  16 warps share each row
// along k and keep their parts of x in registers; a warp leaves its sum of a group in shared memory and
// goes on to the next group.  The groups' sums are joined eight groups at a time, one output a warp: a
// join behind every group, with all warps waiting for it, took as long as the copies of the next one.
//
// GATED: a group holds the same rows of the gate and of the up projection, and its result is
// act(g) u (with g and u themselves where they are wanted); else y (+ add).
#pragma once

#include <cstdint>

#include "block_kernel.cuh"

namespace forge {

constexpr int kRowsWarps = 16;                     // that share a row
constexpr int kRowsThreads = 32 * kRowsWarps + 32;  // and one that issues copies
constexpr int kRowsLanes = 32 * kRowsWarps;
constexpr int kRowsMaxSlots = 12;
constexpr int kRowsRing = 200 * 1024;
constexpr int kRowsMaxVecs = 5;  // 16-byte pieces of x a thread holds: k up to 20480
constexpr int kRowsBatch = 8;    // groups between joins

struct RowsArgs {
    const uint16_t* x;      // [K]
    const uint16_t* w;      // [N, K]: gate, or W
    const uint16_t* w2;     // GATED: up [N, K]
    const uint16_t* add;    // not GATED: residual [N] or null
    uint16_t* y;            // [N]
    uint16_t* g_out;        // GATED: [N], or null
    uint16_t* u_out;
    int N, K, act;
    int slots;
    // The launch before this one on the stream does not write W, and was itself launched so that all work
    // before it is done once this one starts: the ring may fill before stream_wait().
    int weights_ready;
    int* status;
    uint64_t wait_limit_ns;
};

// ROWS: weight rows per group (GATED: half of them the gate's); VECS: ceil(K / 8 / 512)
template <int ROWS, int VECS, bool GATED>
__global__ void __launch_bounds__(kRowsThreads, 1) forge_rows_kernel(const RowsArgs a) {
    extern __shared__ __align__(128) uint8_t rows_ring[];
    __shared__ float part[2][kRowsBatch][ROWS][kRowsWarps];
    __shared__ uint64_t full[kRowsMaxSlots], empty[kRowsMaxSlots];
    __shared__ int abort_flag;
    constexpr int kN = GATED ? ROWS / 2 : ROWS;  // outputs per group
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.K) * 2u, slot_bytes = row_bytes * ROWS;
    const int groups = a.N / kN, stride = static_cast<int>(gridDim.x);
    const int mine = (groups - static_cast<int>(blockIdx.x) + stride - 1) / stride;
    const AbortCtx ab{&abort_flag, a.status, a.wait_limit_ns};
    auto issue = [&](int k, int slot) {
        const size_t at = (blockIdx.x + static_cast<size_t>(k) * stride) * kN * a.K;
        uint8_t* dst = rows_ring + static_cast<size_t>(slot) * slot_bytes;
        mbar_arrive_expect_tx(&full[slot], slot_bytes);
        bulk_load(dst, a.w + at, row_bytes * kN, &full[slot]);
        if constexpr (GATED) bulk_load(dst + row_bytes * kN, a.w2 + at, row_bytes * kN, &full[slot]);
    };
    const bool producer = tid == kRowsLanes;
    if (producer) {
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kRowsWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
        if (a.weights_ready)
            for (int k = 0; k < a.slots && k < mine; ++k) issue(k, k);
    }
    stream_wait();
    // not before: what starts after this launch may rely on the work before it being done
    stream_release();
    __syncthreads();
    if (warp == kRowsWarps) {
        if (!producer) return;
        int slot = 0, issued = a.weights_ready ? (a.slots < mine ? a.slots : mine) : 0;
        uint32_t phase = a.weights_ready ? 1u : 0u;  // of the next turn through the ring
        bool ok = true;
        for (int k = issued; ok && k < mine; ++k) {
            // the slot's first turn finds it empty: the barrier's phase before its first
            ok = wait_bounded(&empty[slot], phase ^ 1u, ab);
            if (!ok) break;
            issue(k, slot);
            ++issued;
            if (++slot == a.slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        // an aborted block's copies land before its memory is given up
        if (!ok)
            for (int i = 0; i < a.slots && i < issued; ++i)
                drain_bounded(&full[i], static_cast<uint32_t>(((issued - 1 - i) / a.slots) & 1), a.wait_limit_ns);
        return;
    }
    uint32_t x[VECS][4];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int k = 8 * (tid + i * kRowsLanes);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0u;
        if (k < a.K) ld_v4(a.x + k, x[i]);
    }
    auto pair = [](uint32_t w) { return F2::of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); };
    // the outputs of groups first .. first + n - 1 of this block
    auto join = [&](int first, int n) {
        const int buf = (first / kRowsBatch) & 1, half = lane >> 4;
        // a half warp sums one row's 16 parts: gated, the two halves take an output's gate and up rows
        for (int o = GATED ? warp : 2 * warp + half; o < n * kN + (GATED ? 0 : half); o += GATED ? kRowsWarps : 2 * kRowsWarps) {
            const bool real = o < n * kN;
            const int g = real ? o / kN : 0, c = real ? o - g * kN : 0;
            float v = part[buf][g][GATED ? c + half * kN : c][lane & 15];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
            const int at = (static_cast<int>(blockIdx.x) + (first + g) * stride) * kN + c;
            auto put = [&](uint16_t* p, float f) {
                p[at] = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(f), 0u) & 0xFFFFu);
            };
            if constexpr (GATED) {
                const float u = __shfl_sync(0xFFFFFFFFu, v, 16);
                if (lane == 0) {
                    if (a.g_out != nullptr) {
                        put(a.g_out, v);
                        put(a.u_out, u);
                    }
                    put(a.y, act_value(v, a.act) * u);
                }
            } else {
                if ((lane & 15) == 0 && real)
                    put(a.y, a.add == nullptr ? v : v + __uint_as_float(static_cast<uint32_t>(a.add[at]) << 16));
            }
        }
    };
    int slot = 0;
    uint32_t phase = 0;
    for (int k = 0; k < mine; ++k) {
        wait_bounded(&full[slot], phase, ab);
        const uint32_t src = smem_addr(rows_ring) + static_cast<uint32_t>(slot) * slot_bytes + 16u * tid;
        F2 sum[ROWS][2];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) sum[r][0] = sum[r][1] = F2::all(0.0f);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            if (8 * (tid + i * kRowsLanes) < a.K) {
                uint32_t w[ROWS][4];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) ld_shared_v4(src + r * row_bytes + i * (16u * kRowsLanes), w[r]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const F2 xp = pair(x[i][j]);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) sum[r][j & 1] = fma2(pair(w[r][j]), xp, sum[r][j & 1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);  // this warp has read the slot
        float(&out)[ROWS][kRowsWarps] = part[(k / kRowsBatch) & 1][k % kRowsBatch];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const F2 both = add2(sum[r][0], sum[r][1]);
            float v = both.lo() + both.hi();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) out[r][warp] = v;
        }
        if (k % kRowsBatch == kRowsBatch - 1 || k + 1 == mine) {
            // the other buffer is written before the next such barrier, which no warp passes before it is
            // done with this join
            asm volatile("bar.sync 1, %0;" ::"n"(kRowsLanes) : "memory");
            join(k - k % kRowsBatch, k % kRowsBatch + 1);
        }
        if (++slot == a.slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
}

}  // namespace forge
