// rows_kernel.cuh -- products of one to four tokens with a weight matrix: y[t, n] = sum_k x[t, k] W[n, k].
//
// Every weight is read once and used a few times, so the time is the weights' way from memory.  The tensor core's
// 128-row tiles would be almost empty, and the splitting and joining along k that few tiles need costs
// more than the products.  Here a block stays on its SM and walks groups of weight rows through a ring of
// bulk copies (whole rows, contiguous in memory, up to 200 KB in flight per SM).  16 warps share each row
// along k and keep their parts of x in registers; a warp leaves its sums of a group in shared memory and
// goes on to the next group.  The groups' sums are joined eight groups at a time, one output a warp: a
// join behind every group, with all warps waiting for it, took as long as the copies of the next one (one
// token, 4096/14336: 58.9 us against 54.2).
//
// GATED: a group holds the same rows of the gate and of the up projection, and its result is
// act(g) u (with g and u themselves where they are wanted); else y (+ add).
//
// Measured, both products of a gated block: 4096/14336 one token 54.9 us, 6.4 TB/s of weights (0.95 of the
// copy rate), two 56.9; 2048/5632 one token 17.6 us, of which half is the two launches.
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
    const uint16_t* x;      // [T, K]
    const uint16_t* w;      // [N, K]: gate, or W
    const uint16_t* w2;     // GATED: up [N, K]
    const uint16_t* add;    // not GATED: residual [T, N] or null
    uint16_t* y;            // [T, N]
    uint16_t* g_out;        // GATED: [T, N], or null
    uint16_t* u_out;
    int T, N, K, act;
    int slots;
    // The launch before this one on the stream does not write W, and all work before that one is done once
    // this one starts (ptx.cuh): the ring may fill before stream_wait().
    int weights_ready;
    int withhold;  // test switch: bytes that each slot is armed for but never gets, so that waits run out
    int* status;
    uint64_t wait_limit_ns;
};

// Sums each of V values (a power of two) over a warp: every exchange halves the values a lane still holds,
// V - 1 of them and then log2(32 / V) more, instead of 5 V.  Afterwards a lane holds the sum of value `at`.
template <int V>
__device__ __forceinline__ float warp_sums(float (&v)[V], int lane, int& at) {
    at = 0;
    int o = 16;
#pragma unroll
    for (int n = V / 2; n > 0; n /= 2, o /= 2) {
        const bool high = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = high ? v[i + n] : v[i], give = high ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
        if (high) at += n;
    }
#pragma unroll
    for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    return v[0];
}

// T: tokens, at most (three run as four); ROWS: weight rows per group (GATED: half of them the gate's); VECS: ceil(K / 8 / 512)
template <int T, int ROWS, int VECS, bool GATED>
__global__ void __launch_bounds__(kRowsThreads, 1) forge_rows_kernel(const RowsArgs a) {
    extern __shared__ __align__(128) uint8_t rows_ring[];
    __shared__ float part[2][kRowsBatch][ROWS * T][kRowsWarps];
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
        mbar_arrive_expect_tx(&full[slot], slot_bytes + static_cast<uint32_t>(a.withhold));
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
    __syncthreads();
    if (warp == kRowsWarps) {
        if (!producer) return;
        int slot = 0;
        uint32_t phase = a.weights_ready ? 1u : 0u;  // of the next turn through the ring
        for (int k = a.weights_ready ? a.slots : 0; k < mine; ++k) {
            // The slot's first turn finds it empty: the barrier's phase before its first.  Once the flag is up,
            // warps go on without their data and their arrivals say nothing: a slot whose copies have not landed
            // must not be armed again.
            if (!wait_bounded(&empty[slot], phase ^ 1u, ab) || *ab.flag) break;
            issue(k, slot);
            if (++slot == a.slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        return;
    }
    uint32_t x[T][VECS][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int k = 8 * (tid + i * kRowsLanes);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[t][i][j] = 0u;
            if (k < a.K && t < a.T) ld_v4(a.x + static_cast<size_t>(t) * a.K + k, x[t][i]);
        }
    auto pair = [](uint32_t w) { return F2::of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); };
    // the outputs of groups first .. first + n - 1 of this block
    auto join = [&](int first, int n) {
        const int buf = (first / kRowsBatch) & 1, half = lane >> 4;
        // output o = (group, column, token); a half warp sums one row's 16 parts: gated, the two halves take
        // an output's gate and up rows
        const int outputs = n * kN * T;
        for (int o = GATED ? warp : 2 * warp + half; o < outputs + (GATED ? 0 : half); o += GATED ? kRowsWarps : 2 * kRowsWarps) {
            const bool real = o < outputs;
            const int g = real ? o / (kN * T) : 0, c = real ? o / T - g * kN : 0, t = o % T;
            float v = part[buf][g][(GATED ? c + half * kN : c) * T + t][lane & 15];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
            const size_t at = static_cast<size_t>(t) * a.N + (static_cast<int>(blockIdx.x) + (first + g) * stride) * kN + c;
            auto put = [&](uint16_t* p, float f) {
                p[at] = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(f), 0u) & 0xFFFFu);
            };
            if constexpr (GATED) {
                const float u = __shfl_sync(0xFFFFFFFFu, v, 16);
                if (lane == 0 && t < a.T) {
                    if (a.g_out != nullptr) {
                        put(a.g_out, v);
                        put(a.u_out, u);
                    }
                    put(a.y, act_value(v, a.act) * u);
                }
            } else {
                if ((lane & 15) == 0 && real && t < a.T)
                    put(a.y, a.add == nullptr ? v : v + __uint_as_float(static_cast<uint32_t>(a.add[at]) << 16));
            }
        }
    };
    int slot = 0;
    uint32_t phase = 0;
    for (int k = 0; k < mine; ++k) {
        wait_bounded(&full[slot], phase, ab);
        const uint32_t src = smem_addr(rows_ring) + static_cast<uint32_t>(slot) * slot_bytes + 16u * tid;
        // two chains of sums per output where there are few outputs
        constexpr int kChains = T == 1 ? 2 : 1;
        F2 sum[ROWS][T][kChains];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int h = 0; h < kChains; ++h) sum[r][t][h] = F2::all(0.0f);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            if (8 * (tid + i * kRowsLanes) < a.K) {
                uint32_t w[ROWS][4];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) ld_shared_v4(src + r * row_bytes + i * (16u * kRowsLanes), w[r]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    F2 xp[T];
#pragma unroll
                    for (int t = 0; t < T; ++t) xp[t] = pair(x[t][i][j]);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const F2 wp = pair(w[r][j]);
#pragma unroll
                        for (int t = 0; t < T; ++t) {
                            F2& to = sum[r][t][j & (kChains - 1)];
                            to = fma2(wp, xp[t], to);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);  // this warp has read the slot
        float v[ROWS * T];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const F2 s = kChains == 2 ? add2(sum[r][t][0], sum[r][t][kChains - 1]) : sum[r][t][0];
                v[r * T + t] = s.lo() + s.hi();
            }
        int at;
        const float total = warp_sums(v, lane, at);
        // the lanes that hold the same value differ in the bits past its exchanges
        if ((lane & (32 / (ROWS * T) - 1)) == 0) part[(k / kRowsBatch) & 1][k % kRowsBatch][at][warp] = total;
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
    // an aborted block's warps have not waited for all copies: they land before its memory is given up
    if (tid == 0 && *ab.flag) wait_out(a.wait_limit_ns);
}

}  // namespace forge
