// block_kernel.cuh -- the persistent matrix-product kernel of the operators around the fused layers:
// the gated feed-forward block and the softmax cross entropy of a linear head, forward and backward.
//
// Every product of these operators is C = A B over a long reduction, followed by arithmetic on the
// finished tile of C.  One pipeline serves them all (the roles of tile_kernel.cuh):
//   warp 0      TMA producer: 64-deep slices of A and B into a shared-memory ring, 128-byte swizzle
//   warp 1      MMA issuer: tcgen05.mma kind::f16, bf16 x bf16 -> f32, accumulating in TMEM; two
//               accumulators, so the next tile's mainloop overlaps this tile's epilogue
//   warps 2-9   epilogue: thread = output row; tcgen05.ld gives it 32 columns at a time, or 16
// What is computed per finished tile is the EPI parameter:
//   kBlockGatedFwd   A = X, B = the gate's and the up projection's rows side by side: the tile holds
//                    G and U of the same columns, and H = act(G) U leaves the chip with them (or
//                    without them, where no backward pass follows)
//   kBlockGatedBwd   the tile is dH = dY Wd, which is never written: with G and U it becomes dG, dU, H
//   kBlockLossStats  the tile is a piece of the logits, which are never written: each row leaves its
//                    maximum and its sum of exponentials over the tile's columns
//   kBlockLossGrad   the logits again; g = dloss (exp(l - lse) - [target]) is written for one piece of
//                    the vocabulary
//   kBlockStore      the tile itself, rounded to bfloat16, with a residual added or with the FP32 sum
//                    of earlier pieces carried in memory; up to NP products in one launch
//
// Layouts.  An operand is K-major when the reduction index runs along memory (X and W of y = X W^T),
// MN-major when it does not; kBlockStore takes either for each operand of each product, the other
// epilogues have theirs fixed.  A product may have two pairs of operands whose products are summed in
// one accumulator (dX = dG Wg + dU Wu).
//
// One copy per operand and slice.  A slice of either order is one box of a 3-D tensor map: K-major
// (64 of the reduction, rows, -), MN-major (64 columns, the slice's 64 rows, blocks of 64 columns).  The
// thread that issues copies sets the pace of the mainloop: with two copies of half the rows for each
// operand, and their addresses worked out per slice, 4096 tokens against 65536 vocabulary entries of 4096
// ran at 1.42-1.6 PFLOP/s, with one each at 1.73.  An MN-major operand whose width is no multiple of 64
// takes two copies: its last block of 64 columns would reach past its rows.
//
// What bounds it, measured on one GB300.  Large products: the tensor core under the chip's power limit.  In
// bursts below the limit, 4096 tokens: block forward 4096/14336 804-817 us (1.77-1.79 PFLOP/s, 0.93 of the measured
// burst peak), block backward 1661-1676 us (1.72-1.74), loss forward over 32768 x 4096 578-586 us (1.88-1.90), loss
// backward 1813-1835 us (1.80-1.82); run on end, at the limit, 1.62, 1.57, 1.72 and 1.64.  Products with MN-major operands
// (dX, dW, dH) reach less there than K-major ones.  The tile with dH also shares the memory system with G,
// U, dG, dU and H: 165 us at 2048 tokens (1.45 PFLOP/s), the same with 16 epilogue warps, with G and U
// prefetched into L2, or loaded first to be evicted.  With one row of tiles: memory, 6.3 TB/s of weights for
// the loss of one token over 131072 x 4096, 6.4 for 16 tokens over 155648 x 4096 (one token there: 3.8 to 4.8).
//
// Why these tiles.  A pair's 256 x 256 tile moves 32 KB into each SM's shared memory per 512 cycles of its
// tensor core; single CTAs on 128 x 128 or 128 x 64 move more per product, fill the GPU with less and serve small
// calls.  The host picks one by what it costs (kTiles in block_api.cu).
//
// Units of work.  A unit is one tile over its whole reduction, or one of `parts` pieces of it.  A
// split tile has no CTA that waits for another: each epilogue warp leaves its FP32 values in memory,
// counts itself in, and the warp that arrives last adds the parts up in their order and runs the
// epilogue.  The order of the sum is fixed, so results do not depend on which one is last.
//
// Waits are bounded as in tile_kernel.cuh, and an aborted launch drains its copies the same way.
#pragma once

#include <cstdint>
#include <type_traits>

#include "block_launch.h"
#include "pairs.cuh"
#include "tile_kernel.cuh"

namespace forge {

enum BlockEpi : int { kBlockStore = 0, kBlockGatedFwd = 1, kBlockGatedBwd = 2, kBlockLossStats = 3, kBlockLossGrad = 4 };
enum BlockAct : int { kActSilu = 0, kActGeluTanh = 1, kActRelu = 2 };

constexpr float kLog2e = 1.4426950408889634f;

// Whether an epilogue's results go to memory through shared memory, on pairs (WarpOut).
constexpr bool staged(int epi) { return epi == kBlockGatedFwd || epi == kBlockLossGrad; }

template <int BN, int CG, int EPI, bool STAGED = CG == 2 && staged(EPI)>
struct BlockCfg {
    static_assert((BN == 256 && CG == 2) || ((BN == 128 || BN == 64) && CG == 1), "tile shapes");
    static constexpr int kBLoad = BN / CG;  // B rows (or columns) staged by this CTA
    static constexpr int kABytes = kBM * kBK * 2;
    static constexpr int kBBytes = kBLoad * kBK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, half the columns each
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    // two 2 KiB buffers per epilogue warp, 32 rows x 32 columns of bfloat16 each, on their way to memory
    static constexpr int kStaging = STAGED ? kEpiWarps * 4096 : 0;
    static constexpr int kStages = (7 * 32768 - kStaging) / kStageBytes;
    static constexpr int kRingBytes = kStages * kStageBytes;
    // where A has few rows (BlockGroup::a_rows) its slices are smaller and the ring holds more stages
    static constexpr int kMaxStages = BN == 64 ? 24 : CG == 1 ? 13 : kStages;
    static constexpr int kSmemBytes = kRingBytes + kStaging + 512 + 1024;  // barriers, alignment slack
    static_assert(kSmemBytes <= 232448, "shared memory");
    static constexpr int stages(int a_rows) {
        const int fit = kRingBytes / (a_rows * 128 + kBBytes);
        return fit < kMaxStages ? fit : kMaxStages;
    }
};

struct BlockProblem {
    int rows, cols;       // of the output (gated forward: cols = d_ff, a tile spans BN / 2 of them)
    TileOrder order;
    int unit_start;       // number of its first unit
    int split_from;       // tiles from here on are cut into `parts` units along the reduction
    int parts;
    int kb[2];            // 64-deep reduction slices of the two operand pairs (the second may have none)
    int a_mn, b_mn;       // operand orders (kBlockStore): 1 = MN-major
    int a_flat, b_flat;   // MN-major and no multiple of 64 wide: (column, row, -) maps, a copy for each 64 columns
    int64_t part_base;    // where its split tiles' FP32 values start (floats)
    int count_base;       // and their counters
    // kBlockStore: add: residual [rows, ld] or null; sum: FP32 [rows, cols] of earlier pieces, read if
    // sum_in, written instead of the result if sum_out
    const uint16_t* add;
    float* sum;
    int sum_in, sum_out;
    int64_t ld;
    // gated backward: G, U [rows, cols] bf16; gated forward: whether G and U are wanted
    const uint16_t* g_in;
    const uint16_t* u_in;
    int keep;
    int act;
    // loss: columns are vocabulary entries v0 .. v0 + cols - 1
    const int64_t* target;
    int64_t v0, vocab, ignore;
    float2* stats;        // [2 * tile columns][rows]: (max, sum of exponentials), base 2
    float* target_logit;  // [rows]
    const float* lse;     // [rows]
    const float* dloss;   // [rows]
    // kBlockLossGrad writes g / *unit, and kBlockStore multiplies its finished sums by *unit (there, null: 1)
    const float* unit;
    // kBlockLossGrad: where this launch leaves the unit that it finds itself, or null
    float* own_unit;
};

// Up to NP products, the one with the longest units first.  What every role reads at its start comes first.
template <int NP>
struct BlockGroup {
    int n;
    // Rows of A that a stage holds: 128, or on single CTAs with one row of tiles the rows there are, rounded
    // up to a multiple of 8 (A's tensor maps have boxes of that many rows then).  The MMA reads 128 rows
    // whatever lies in the rest of the stage: an accumulator row depends on its own row of A alone, and rows
    // past the output's last are not used.  One token's X or H would otherwise be copied as 64 rows of zero
    // fill, as many bytes as the weights beside it.
    int a_rows;
    UnitPlan units;
    int zero_n;
    int* status;
    uint64_t wait_limit_ns, acc_wait_limit_ns;
    float* parts;
    // Arrival counters of split tiles: zero before the launch, and zero again after it (the last arrival
    // resets its own).  zero_n: counters, from zero_at, that this launch clears for the stream's next ones.
    uint32_t* counts;
    uint32_t* zero_at;
    int withhold_first_stage;  // test switch, as TileArgs::withhold_first_stage
    // results: kBlockStore's out of each product; G, U, H; dG, dU, H; kBlockLossGrad's g
    uint16_t* to[NP > 3 ? NP : 3];
    BlockProblem prob[NP];
    CUtensorMap maps[4 * NP];  // per product: A, B of the first pair, A, B of the second
};

constexpr int products_of(int epi) { return epi == kBlockStore ? kMaxProducts : 1; }

// The results' maps besides, for pairs whose epilogue is staged.  Other launches go without: a small call's
// time shows every parameter (256 tokens through 256/512: 13.0 us with them, 12.75 without).
template <int EPI>
struct PairGroup : BlockGroup<products_of(EPI)> {
    CUtensorMap outs[EPI == kBlockGatedFwd ? 3 : 1];
};
template <int CG, int EPI>
using GroupOf = std::conditional_t<CG == 2 && staged(EPI), PairGroup<EPI>, BlockGroup<products_of(EPI)>>;

struct Unit {
    int prob, mb, nb, part, split;  // split: which split tile of the product, or -1
    int k_first, k_end;             // slices of the concatenated operand pairs
};

// stream_wait() with a role's first unit in hand: the compiler may not move its computation past the wait.
__device__ __forceinline__ void stream_wait_with(int& u, Unit& w) {
    asm volatile(FORGE_STREAM_WAIT
                 : "+r"(u), "+r"(w.prob), "+r"(w.mb), "+r"(w.nb), "+r"(w.part), "+r"(w.split), "+r"(w.k_first), "+r"(w.k_end)
                 :
                 : "memory");
}

template <int NP>
__device__ __forceinline__ Unit unit_of(const BlockGroup<NP>& g, int u, int l) {
    if constexpr (NP > 1) {
        while (l + 1 < g.n && u >= g.prob[l + 1].unit_start) ++l;
    } else {
        l = 0;
    }
    const BlockProblem& b = g.prob[l];
    int t = u - b.unit_start;
    Unit r{l, 0, 0, 0, -1, 0, b.kb[0] + b.kb[1]};
    if (t >= b.split_from) {
        const int s = t - b.split_from, kb = r.k_end;
        r.split = s / b.parts;
        r.part = s - r.split * b.parts;
        r.k_first = static_cast<int>(static_cast<int64_t>(kb) * r.part / b.parts);
        r.k_end = static_cast<int>(static_cast<int64_t>(kb) * (r.part + 1) / b.parts);
        t = b.split_from + r.split;
    }
    tile_coords(t, b.order, r.mb, r.nb);
    return r;
}

// ---------------------------------------------------------------- arithmetic

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// act(g), and for the backward pass its derivative.  gelu with the tanh form is
// g (1 + tanh y) / 2 = g sigmoid(2 y), y = sqrt(2 / pi) (g + 0.044715 g^3).
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)

__device__ __forceinline__ float act_value(float g, int act) {
    if (act == kActRelu) return g > 0.0f ? g : (g != g ? g : 0.0f);
    const float a = act == kActSilu ? g : kGelu2 * (g + 0.044715f * g * g * g);
    return __fdividef(g, 1.0f + __expf(-a));
}

__device__ __forceinline__ void act_both(float g, int act, float& value, float& slope) {
    if (act == kActRelu) {
        value = g > 0.0f ? g : (g != g ? g : 0.0f);
        slope = g > 0.0f ? 1.0f : 0.0f;
    } else if (act == kActSilu) {
        const float p = sigmoid_fast(g);
        value = g * p;
        slope = p * (1.0f + g * (1.0f - p));
    } else {
        const float p = sigmoid_fast(kGelu2 * (g + 0.044715f * g * g * g));
        value = g * p;
        // p (1 - p) is 0 long before g^2 is 1e30, and times infinity it would be NaN
        slope = p + g * p * (1.0f - p) * (kGelu2 * (1.0f + 3.0f * 0.044715f * fminf(g * g, 1e30f)));
    }
}

// 2^x by the hardware approximation (2 ulp)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- rows of bfloat16 in memory

// 2 W columns of one row, packed in pairs; `left`: columns from here to the end of the row (loaded in runs
// of 8); wide: the row's address is a multiple of 32 bytes at every 16th column
template <int W>
__device__ __forceinline__ void load_run(const uint16_t* p, uint32_t (&v)[W], int left, bool wide) {
#pragma unroll
    for (int h = 0; h < W / 8; ++h) {
        if (wide && left >= 16 * h + 16) {
            uint32_t r[8];
            ld_v8(p + 16 * h, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * h + i] = r[i];
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t r[4] = {0u, 0u, 0u, 0u};
                if (left >= 16 * h + 8 * q + 8) ld_v4(p + 16 * h + 8 * q, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[8 * h + 4 * q + i] = r[i];
            }
        }
    }
}

// A warp's results on their way to memory: 32 rows x 32 columns of bfloat16 at a time, each lane its row.
// Staged, they go through shared memory and a tiled store, which writes whole row pieces and leaves out what
// lies past the last row or column: stores by the lanes themselves, one row each, take 32 passes through the
// L1 for 32 rows and set the pace of tiles with short reductions and much to write (forward, 4637 tokens, 80
// wide, through d_ff = 7224: 138 us with them, 119 so; 8192 tokens through 5120/17408: 2760 and 2715; the
// loss's gradient, 4096 x 32768, 128 wide: 174 and 170).  It costs a stage of the ring, which launches
// where operands from memory set the pace (gradients of 256 and 512 tokens through 4096/14336: 202 and 292 us
// so, 195.5 and 285 by the lanes), and single CTAs, which small calls have, some 0.5 us.
template <bool kStaged>
struct WarpOut {
    const CUtensorMap* maps;
    uint16_t* const* to;
    int64_t ld;  // the results' width
    int rows;
    uint32_t buf;  // staged: two buffers, 1024-byte aligned
    int turn;
    // result i, its columns from col on
    template <int W>
    __device__ __forceinline__ void put(int i, const uint32_t (&v)[W], int col, int row0) {
        const uint32_t lane = threadIdx.x & 31u;
        if constexpr (kStaged) {
            static_assert(W == 16);
            if (lane == 0) bulk_wait_read<1>();  // the buffer's last store has read it
            __syncwarp();
            const uint32_t at = buf + (static_cast<uint32_t>(turn) << 11);
            turn ^= 1;
            // the 64-byte swizzle: 16-byte piece j of row r lies at piece j ^ ((r / 2) mod 4)
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                st_shared_v4(at + lane * 64u + ((j ^ ((lane >> 1) & 3u)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                             v[4 * j + 3]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&maps[i], at, col, row0);
                bulk_commit();
            }
        } else if (row0 + static_cast<int>(lane) < rows) {
            uint16_t* p = to[i] + (static_cast<size_t>(row0) + lane) * ld + col;
            const int left = static_cast<int>(ld) - col;
            const bool wide = (ld & 15) == 0;
#pragma unroll
            for (int h = 0; h < W / 8; ++h) {
                if (wide && left >= 16 * h + 16) {
                    const uint32_t r[8] = {v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3],
                                           v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]};
                    st_v8(p + 16 * h, r);
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t r[4] = {v[8 * h + 4 * q], v[8 * h + 4 * q + 1], v[8 * h + 4 * q + 2],
                                               v[8 * h + 4 * q + 3]};
                        if (left >= 16 * h + 8 * q + 8) st_v4(p + 16 * h + 8 * q, r);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void end() {
        // shared memory stays until the last stores have read it
        if constexpr (kStaged) {
            if ((threadIdx.x & 31u) == 0) bulk_wait_read<0>();
        }
    }
};

// ---------------------------------------------------------------- the accumulator a warp reads
// Column `c` of the tile, 32 at a time, for this thread's row: from TMEM, or the sum of a split
// tile's parts.

struct AccTmem {
    uint32_t taddr;
    __device__ __forceinline__ void load(int c, uint32_t (&g)[32]) const {
        __syncwarp();  // tcgen05.ld is a warp's: lanes that skipped a row's stores rejoin here
        tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(c), g);
        tmem_ld_wait(g);
    }
    __device__ __forceinline__ void load(int c, uint32_t (&g)[16]) const {
        __syncwarp();
        tmem_ld_16(taddr + static_cast<uint32_t>(c), g);
    }
};

struct AccParts {
    const float* p;  // this thread's row of part 0; columns are 32 floats apart
    size_t step;     // floats from part to part
    int parts;
    bool valid;      // rows past the output's last left nothing in memory
    template <int N>
    __device__ __forceinline__ void load(int c, uint32_t (&g)[N]) const {
        // two parts' loads are in flight at once: a trip to the L2 takes longer than all of a part's adds
        float s[N], n[N];
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = valid ? __ldcg(p + static_cast<size_t>(c + j) * 32) : 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) n[j] = valid ? __ldcg(p + step + static_cast<size_t>(c + j) * 32) : 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = __fadd_rn(s[j], n[j]);
        for (int k = 2; k < parts; k += 2) {
            const bool both = valid && k + 1 < parts;
            float m[N];
#pragma unroll
            for (int j = 0; j < N; ++j) n[j] = valid ? __ldcg(p + k * step + static_cast<size_t>(c + j) * 32) : 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) m[j] = both ? __ldcg(p + (k + 1) * step + static_cast<size_t>(c + j) * 32) : -0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] = __fadd_rn(__fadd_rn(s[j], n[j]), m[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = __float_as_uint(s[j]);
    }
};

// ---------------------------------------------------------------- epilogues
// `row`: this thread's output row; h: the half of the tile's columns that the warp owns; out: its way to
// memory.  A warp whose first row is past the output's last does nothing.

// Columns at a time where the arithmetic is long: on single CTAs, which serve small calls, half as many, since
// a launch's first pass through it waits for its instructions (256 tokens through 256/512: 12.75 us with 32
// columns, 11.8 with 16; its gradients 18.6 and 17.5; a loss of 130 x 4099: 9.6 and 9.2).
template <int BN>
constexpr int kEpiStep = BN == 256 ? 32 : 16;

__device__ __forceinline__ int warp_row0(int row) { return row - static_cast<int>(threadIdx.x & 31u); }

template <int BN, class Acc, class Out>
__device__ __forceinline__ void epi_store(const BlockProblem& b, const Acc& acc, int row, int nb, int h, Out& out) {
    if (warp_row0(row) >= b.rows) return;
    const bool wide = (b.ld & 15) == 0, mine = row < b.rows;
    // from the L2, not by __ldg: a launch that may still run when this one starts writes it
    const float unit = b.unit != nullptr ? __ldcg(b.unit) : 1.0f;
#pragma unroll 1
    for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
        const int col = nb * BN + c, left = b.cols - col;
        if (left <= 0) break;  // the same for the whole warp
        uint32_t add[16];
        if (b.add != nullptr && mine) load_run(b.add + static_cast<size_t>(row) * b.ld + col, add, left, wide);
        uint32_t g[32];
        acc.load(c, g);
        if (b.sum_in && mine) {
            const float* s = b.sum + static_cast<size_t>(row) * b.cols + col;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t r[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                if (left >= 8 * q + 8) ld_v8(s + 8 * q, r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    g[8 * q + i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), __uint_as_float(g[8 * q + i])));
            }
        }
        if (b.sum_out) {
            if (mine) {
                float* s = b.sum + static_cast<size_t>(row) * b.cols + col;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t r[8] = {g[8 * q], g[8 * q + 1], g[8 * q + 2], g[8 * q + 3],
                                           g[8 * q + 4], g[8 * q + 5], g[8 * q + 6], g[8 * q + 7]};
                    if (left >= 8 * q + 8) st_v8(s + 8 * q, r);
                }
            }
            continue;
        }
        if (b.unit != nullptr) {
#pragma unroll
            for (int j = 0; j < 32; ++j) g[j] = __float_as_uint(__fmul_rn(__uint_as_float(g[j]), unit));
        }
        if (b.add != nullptr && mine) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                g[2 * j] = __float_as_uint(__fadd_rn(__uint_as_float(g[2 * j]), bf16_lo(add[j])));
                g[2 * j + 1] = __float_as_uint(__fadd_rn(__uint_as_float(g[2 * j + 1]), bf16_hi(add[j])));
            }
        }
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2_rn(g[2 * j], g[2 * j + 1]);
        out.put(0, o, col, warp_row0(row));
    }
}

template <int BN, class Acc, class Out>
__device__ __forceinline__ void epi_gated_fwd(const BlockProblem& b, const Acc& acc, int row, int nb, int h, Out& out) {
    if (warp_row0(row) >= b.rows) return;
    constexpr int kCols = BN / 4, kStep = kEpiStep<BN>;
#pragma unroll 1
    for (int c = h * kCols; c < (h + 1) * kCols; c += kStep) {
        const int col = nb * (BN / 2) + c;
        if (b.cols - col <= 0) break;
        uint32_t g[kStep], u[kStep];
        acc.load(c, g);
        acc.load(BN / 2 + c, u);
        uint32_t o[kStep / 2];
        if (b.keep) {
#pragma unroll
            for (int j = 0; j < kStep / 2; ++j) o[j] = pack_bf16x2_rn(g[2 * j], g[2 * j + 1]);
            out.put(0, o, col, warp_row0(row));
#pragma unroll
            for (int j = 0; j < kStep / 2; ++j) o[j] = pack_bf16x2_rn(u[2 * j], u[2 * j + 1]);
            out.put(1, o, col, warp_row0(row));
        }
        // H is rounded to bfloat16, the type of the next product's operand
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
            const float a0 = act_value(__uint_as_float(g[2 * j]), b.act) * __uint_as_float(u[2 * j]);
            const float a1 = act_value(__uint_as_float(g[2 * j + 1]), b.act) * __uint_as_float(u[2 * j + 1]);
            o[j] = pack_bf16x2_rn(__float_as_uint(a0), __float_as_uint(a1));
        }
        out.put(2, o, col, warp_row0(row));
    }
}

template <int BN, class Acc, class Out>
__device__ __forceinline__ void epi_gated_bwd(const BlockProblem& b, const Acc& acc, int row, int nb, int h, Out& out) {
    if (warp_row0(row) >= b.rows) return;
    const bool wide = (b.cols & 15) == 0, mine = row < b.rows;
    constexpr int kStep = kEpiStep<BN>;
#pragma unroll 1
    for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += kStep) {
        const int col = nb * BN + c, left = b.cols - col;
        if (left <= 0) break;
        const size_t at = static_cast<size_t>(row) * b.cols + col;
        uint32_t g[kStep / 2], u[kStep / 2];
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) g[j] = u[j] = 0u;
        if (mine) {
            load_run(b.g_in + at, g, left, wide);
            load_run(b.u_in + at, u, left, wide);
        }
        uint32_t d[kStep];
        acc.load(c, d);
        uint32_t o[kStep / 2];
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
            float a0, s0, a1, s1;
            act_both(bf16_lo(g[j]), b.act, a0, s0);
            act_both(bf16_hi(g[j]), b.act, a1, s1);
            const float u0 = bf16_lo(u[j]), u1 = bf16_hi(u[j]);
            const float d0 = __uint_as_float(d[2 * j]), d1 = __uint_as_float(d[2 * j + 1]);
            g[j] = pack_bf16x2_rn(__float_as_uint(d0 * u0 * s0), __float_as_uint(d1 * u1 * s1));
            u[j] = pack_bf16x2_rn(__float_as_uint(d0 * a0), __float_as_uint(d1 * a1));
            o[j] = pack_bf16x2_rn(__float_as_uint(a0 * u0), __float_as_uint(a1 * u1));
        }
        out.put(0, g, col, warp_row0(row));
        out.put(1, u, col, warp_row0(row));
        out.put(2, o, col, warp_row0(row));
    }
}

// What a row's exponentials are taken relative to, given its maximum so far: an infinite one takes nothing out, so
// that a row of -inf keeps sum 0 and a row with +inf has sum +inf.
__device__ __forceinline__ float stats_base(float top) { return fabsf(top) == INFINITY ? 0.0f : top; }

// One pass over the warp's columns with the running maximum and sum, in base 2.  Maxima and sums run in
// four chains each, the sums in pairs of binary32: a single chain of dependent operations over 128 columns
// took longer than the products of a 1024-long reduction, and set the tile's pace.
template <int BN, class Acc>
__device__ __forceinline__ void epi_loss_stats(const BlockProblem& b, const Acc& acc, int row, int nb, int h) {
    const bool mine = row < b.rows;
    const int64_t t = mine ? b.target[row] : -1;
    const int64_t first = b.v0 + static_cast<int64_t>(nb) * BN;  // vocabulary entry of the tile's column 0
    float m = -INFINITY, s = 0.0f;
    constexpr int kStep = kEpiStep<BN>;
#pragma unroll 1
    for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += kStep) {
        const int left = b.cols - (nb * BN + c);
        if (left <= 0) break;
        uint32_t g[kStep];
        acc.load(c, g);
        const int64_t at = t - (first + c);
        if (at >= 0 && at < kStep && t < b.vocab) {
            float lt = 0.0f;
#pragma unroll
            for (int j = 0; j < kStep; ++j) lt = at == j ? __uint_as_float(g[j]) : lt;
            b.target_logit[row] = lt;
        }
        if (left < kStep) {
#pragma unroll
            for (int j = 0; j < kStep; ++j) g[j] = j < left ? g[j] : __float_as_uint(-INFINITY);
        }
        float top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = __uint_as_float(g[k]);
#pragma unroll
        for (int j = 4; j < kStep; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(g[j]));
        const float mn = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * kLog2e);
        const float base = stats_base(mn);
        const F2 scale = F2::all(kLog2e), less = F2::all(-base);
        F2 e[4];
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
            const F2 x = fma2(F2::of(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1])), scale, less);
            const F2 y = F2::of(exp2_fast(x.lo()), exp2_fast(x.hi()));
            e[j & 3] = j < 4 ? y : add2(e[j & 3], y);
        }
        const F2 sum = add2(add2(e[0], e[1]), add2(e[2], e[3]));
        s = __fmaf_rn(s, exp2_fast(m - base), sum.lo() + sum.hi());
        m = mn;
    }
    if (mine) b.stats[static_cast<size_t>(2 * nb + h) * b.rows + row] = make_float2(m, s);
}

// What a token adds to the largest |dloss|.  An infinite one adds nothing: relative to it every other token's g
// would be 0, and 0 times it NaN.
__device__ __forceinline__ float loss_weight(float dloss, int64_t target, int64_t ignore) {
    return target == ignore || fabsf(dloss) == INFINITY ? 0.0f : fabsf(dloss);
}

// The number that g is kept relative to: the largest finite |dloss| of the tokens that count, or 1 where there is
// none above 0.  With few tokens every warp finds it itself while the first tile's slices come in, and one of them
// leaves it for the products that follow.
__device__ __forceinline__ float loss_unit(const BlockProblem& b, bool leave) {
    if (b.own_unit == nullptr) return __ldcg(b.unit);
    const int lane = static_cast<int>(threadIdx.x & 31u);
    float m = 0.0f;
    for (int i = lane; i < b.rows; i += 32) m = fmaxf(m, loss_weight(b.dloss[i], b.target[i], b.ignore));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    m = m > 0.0f ? m : 1.0f;
    if (leave && lane == 0) *b.own_unit = m;
    return m;
}

template <int BN, class Acc, class Out>
__device__ __forceinline__ void epi_loss_grad(const BlockProblem& b, const Acc& acc, int row, int nb, int h, Out& out,
                                              float unit) {
    if (warp_row0(row) >= b.rows) return;
    const bool mine = row < b.rows;
    const int64_t t = mine ? b.target[row] : -1;
    const bool counts = t != b.ignore;
    const float shift = mine ? -b.lse[row] * kLog2e : 0.0f;
    // a target outside the vocabulary that is not the ignored one shows as NaN
    const float given = !mine || !counts ? 0.0f : (t >= 0 && t < b.vocab ? b.dloss[row] : NAN);
    // Under the usual mean over tokens every dloss is the same number, and so is, nearly, every
    // target's entry -dloss (1 - p): rounded to bfloat16 as it is, that number's one rounding error (up
    // to 2^-8) would stand in all of dX and dW.  Relative to the largest dloss the entry is -(1 - p).
    const float scale = given / unit;
    const int64_t first = b.v0 + static_cast<int64_t>(nb) * BN;
#pragma unroll 1
    for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
        const int left = static_cast<int>(b.ld) - (nb * BN + c);
        if (left <= 0) break;
        uint32_t g[32];
        acc.load(c, g);
        const int64_t off = t - (first + c);
        const int at = off >= 0 && off < 32 ? static_cast<int>(off) : -1;
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const F2 x = fma2(F2::of(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1])), F2::all(kLog2e), F2::all(shift));
            const float p0 = exp2_fast(x.lo()), p1 = exp2_fast(x.hi());
            const F2 v = mul2(F2::of(at == 2 * j ? p0 - 1.0f : p0, at == 2 * j + 1 ? p1 - 1.0f : p1), F2::all(scale));
            o[j] = counts ? pack_bf16x2_rn(__float_as_uint(v.lo()), __float_as_uint(v.hi())) : 0u;
        }
        out.put(0, o, nb * BN + c, warp_row0(row));
    }
}

template <int BN, int EPI, class Acc, class Out>
__device__ __forceinline__ void block_epilogue(const BlockProblem& b, const Acc& acc, int row, int nb, int h, Out& out,
                                               float unit) {
    if constexpr (EPI == kBlockStore) epi_store<BN>(b, acc, row, nb, h, out);
    else if constexpr (EPI == kBlockGatedFwd) epi_gated_fwd<BN>(b, acc, row, nb, h, out);
    else if constexpr (EPI == kBlockGatedBwd) epi_gated_bwd<BN>(b, acc, row, nb, h, out);
    else if constexpr (EPI == kBlockLossStats) epi_loss_stats<BN>(b, acc, row, nb, h);
    else epi_loss_grad<BN>(b, acc, row, nb, h, out, unit);
}

// ---------------------------------------------------------------- the kernel

// drain_copies (tile_kernel.cuh) for a ring of `stages` stages.
template <int CG>
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, uint64_t n_own, uint64_t n_peer, int64_t withheld,
                                           uint32_t stage_bytes, uint64_t limit_ns) {
    auto last_of = [&](uint64_t n, int s) -> int64_t {
        return n > static_cast<uint64_t>(s) ? s + stages * static_cast<int64_t>((n - 1 - s) / stages) : -1;
    };
    for (int s = 0; s < stages; ++s) {
        const int64_t lo = last_of(n_own, s), lp = CG == 1 ? lo : last_of(n_peer, s);
        const int64_t last = lo > lp ? lo : lp;
        if (last < 0) continue;
        if (CG == 2 && lo < last) mbar_arrive_expect_tx(&full[s], stage_bytes);
        if (CG == 2 && lp < last) mbar_complete_tx(&full[s], stage_bytes);
        if (last == withheld) mbar_complete_tx(&full[s], stage_bytes);
        drain_bounded(&full[s], static_cast<uint32_t>((last / stages) & 1), limit_ns);
    }
}

template <int BN, int CG, int EPI>
__global__ void __launch_bounds__(BlockCfg<BN, CG, EPI>::kThreads, 1)
    forge_block_kernel(const __grid_constant__ GroupOf<CG, EPI> grp) {
    using C = BlockCfg<BN, CG, EPI>;
    constexpr bool kGated = EPI == kBlockGatedFwd;
    constexpr int kColsPerTile = kGated ? BN / 2 : BN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const int a_rows = CG == 1 ? grp.a_rows : kBM;
    const int n_stages = CG == 1 ? C::stages(a_rows) : C::kStages;
    const uint32_t stage_bytes = static_cast<uint32_t>(a_rows) * 128u + C::kBBytes;
    uint8_t* sA = smem;
    uint8_t* sB = smem + n_stages * a_rows * 128;  // behind A: the MMA's reads past A's rows stay inside the ring
    uint8_t* staging = smem + C::kRingBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + C::kStaging);
    uint64_t* empty = full + C::kMaxStages;
    uint64_t* acc_full = empty + C::kMaxStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint64_t* peer_done = drain + 1;
    uint64_t* peer_count = peer_done + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(peer_count + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG > 1 ? cluster_ctarank() : 0u;
    const int pair = static_cast<int>(blockIdx.x) / CG;
    const int pairs = static_cast<int>(gridDim.x) / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < n_stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kEpiWarps * CG);
        }
        mbar_init(drain, 1);
        mbar_init(peer_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        for (int l = 0; l < grp.n; ++l) {
            tma_prefetch_desc(&grp.maps[4 * l]);
            tma_prefetch_desc(&grp.maps[4 * l + 1]);
        }
    }
    if (warp == 1) {
        tmem_alloc<CG>(tmem_slot, C::kTmemCols);
        tmem_relinquish<CG>();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();
    tc_fence_after();
    // None of this touches memory of the stream's other work, and neither does finding a role's first
    // unit: its divisions and the first reads of the launch's parameters take some 2000 cycles, which pass
    // while the launch before this one ends.
    const uint32_t tmem_base = *tmem_slot;
    const AbortCtx ab{abort_flag, grp.status, grp.wait_limit_ns};
    uint64_t n_issued = 0;
    int64_t withheld = -1;

    // operand orders: fixed by what the epilogue's product is, or the product's own (kBlockStore)
    auto a_mn = [&](const BlockProblem& b) { return EPI == kBlockStore ? b.a_mn != 0 : false; };
    auto b_mn = [&](const BlockProblem& b) { return EPI == kBlockStore ? b.b_mn != 0 : EPI == kBlockGatedBwd; };

    if (warp == 0) {
        UnitCursor cur;
        int u = cur.next(grp.units, pair, pairs);
        Unit w = unit_of(grp, u < 0 ? 0 : u, 0);
        stream_wait_with(u, w);
        auto advance = [&]() {
            u = cur.next(grp.units, pair, pairs);
            if (u >= 0) w = unit_of(grp, u, w.prob);
        };
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint64_t keep = policy_evict_last();
            const uint64_t once = policy_evict_first();
            const bool leader = rank == 0;
            const bool withhold = grp.withhold_first_stage && leader;
            const uint32_t bars = CG == 2 ? map_to_rank(smem_addr(full), 0) : smem_addr(full);
            const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * 128u;
            const uint32_t a_ring = smem_addr(sA), b_ring = smem_addr(sB);
            for (; ok && u >= 0; advance()) {
                const int l = w.prob;
                const BlockProblem& b = grp.prob[l];
                const bool amn = a_mn(b), bmn = b_mn(b), a_flat = b.a_flat != 0, b_flat = b.b_flat != 0;
                const int row_a = w.mb * kBM * CG + static_cast<int>(rank) * kBM;
                // with one row of tiles B passes through once
                const uint64_t pol_b = b.order.tiles_m == 1 ? once : keep;
                // gated forward: the even CTA (or the first half of the columns) holds the gate's
                // rows, the other the up projection's, of the same d_ff columns
                const int col_b = kGated ? w.nb * kColsPerTile : w.nb * BN + static_cast<int>(rank) * C::kBLoad;
#pragma unroll 1
                for (int seg = 0; seg < 2 && ok; ++seg) {
                    // the unit's slices of this operand pair
                    const int from = seg == 0 ? w.k_first : (w.k_first > b.kb[0] ? w.k_first : b.kb[0]);
                    const int to = seg == 0 && w.k_end > b.kb[0] ? b.kb[0] : w.k_end;
                    if (from >= to) continue;
                    const int k0 = (from - (seg == 0 ? 0 : b.kb[0])) * kBK;
                    const CUtensorMap* ma = &grp.maps[4 * l + 2 * seg];
                    const CUtensorMap* mb = kGated && CG == 2 && rank == 1 ? &grp.maps[4 * l + 3] : ma + 1;
                    const CUtensorMap* mu = &grp.maps[4 * l + 3];  // gated forward, one CTA: the up projection's
                    // coordinates of the first slice and their steps: one of them moves along the reduction
                    int a0 = amn ? (a_flat ? row_a : 0) : k0, a1 = amn ? k0 : row_a, a2 = amn && !a_flat ? row_a / 64 : 0;
                    int b0 = bmn ? (b_flat ? col_b : 0) : k0, b1 = bmn ? k0 : col_b, b2 = bmn && !b_flat ? col_b / 64 : 0;
                    const int da0 = amn ? 0 : kBK, da1 = amn ? kBK : 0, db0 = bmn ? 0 : kBK, db1 = bmn ? kBK : 0;
#pragma unroll 1
                    for (int n = to - from; n > 0; --n) {
                        if (!wait_bounded(&empty[stage], phase ^ 1u, ab)) { ok = false; break; }
                        const uint32_t bar = bars + 8u * static_cast<uint32_t>(stage);
                        if (leader) mbar_arrive_expect_tx(&full[stage], CG * stage_bytes);
                        if (withhold && n_issued == 0) {
                            // test switch: arm this stage but never copy into it
                            withheld = 0;
                        } else {
                            const uint32_t a_dst = a_ring + static_cast<uint32_t>(stage) * a_bytes;
                            const uint32_t b_dst = b_ring + static_cast<uint32_t>(stage) * C::kBBytes;
                            tma_load_3d_cg<CG>(a_dst, ma, bar, a0, a1, a2, keep);
                            tma_load_3d_cg<CG>(b_dst, mb, bar, b0, b1, b2, pol_b);
                            if (EPI == kBlockStore && a_flat) tma_load_3d_cg<CG>(a_dst + kBK * 128, ma, bar, a0 + 64, a1, 0, keep);
                            if (kGated && CG == 1) tma_load_3d_cg<CG>(b_dst + BN / 2 * 128, mu, bar, b0, b1, 0, pol_b);
                            if (C::kBLoad == 128 && (EPI == kBlockStore || EPI == kBlockGatedBwd) && b_flat)
                                tma_load_3d_cg<CG>(b_dst + kBK * 128, mb, bar, b0 + 64, b1, 0, pol_b);
                        }
                        a0 += da0;
                        a1 += da1;
                        b0 += db0;
                        b1 += db1;
                        ++n_issued;
                        if (++stage == n_stages) { stage = 0; phase ^= 1u; }
                    }
                    if (kGated) break;  // its fourth map is the up projection's, not a second pair's
                }
            }
            if constexpr (CG == 2) {
                if (rank == 1) {
                    st_shared_cluster_u64(map_to_rank(smem_addr(peer_count), 0), n_issued);
                    mbar_arrive_remote(map_to_rank(smem_addr(peer_done), 0));
                }
            }
        }
    } else if (warp == 1) {
        UnitCursor cur;
        int u = cur.next(grp.units, pair, pairs);
        Unit w = unit_of(grp, u < 0 ? 0 : u, 0);
        stream_wait_with(u, w);
        auto advance = [&]() {
            u = cur.next(grp.units, pair, pairs);
            if (u >= 0) w = unit_of(grp, u, w.prob);
        };
        if (lane == 0 && rank == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued_any = false;
            for (; ok && u >= 0; advance()) {
                const BlockProblem& b = grp.prob[w.prob];
                const bool amn = a_mn(b), bmn = b_mn(b);
                const uint32_t idesc = idesc_bf16_f32(kBM * CG, BN, amn, bmn);
                // MN-major: 16 reduction steps are 16 rows of 128 bytes, 64-element blocks 8 KiB apart;
                // K-major: 32 bytes within each 128-byte row, 8-row groups 1024 bytes apart.  A
                // descriptor's address field counts 16 bytes, and no sum below leaves it
                const uint32_t a_step = (amn ? 2048u : 32u) >> 4, b_step = (bmn ? 2048u : 32u) >> 4;
                const uint64_t a_desc = smem_desc_sw128(smem_addr(sA), amn ? kBK * 128u : 16u, 1024);
                const uint64_t b_desc = smem_desc_sw128(smem_addr(sB), bmn ? kBK * 128u : 16u, 1024);
                if (!wait_bounded(&acc_empty[acc], acc_phase ^ 1u, ab)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
                for (int kb = w.k_first; kb < w.k_end; ++kb) {
                    if (!wait_bounded(&full[stage], phase, ab)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = a_desc + static_cast<uint32_t>(stage) * (static_cast<uint32_t>(a_rows) * 128u >> 4);
                    const uint64_t bd = b_desc + static_cast<uint32_t>(stage) * (C::kBBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk)
                        tc_mma_bf16<CG>(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc,
                                        (kb != w.k_first || kk != 0) ? 1u : 0u);
                    issued_any = true;
                    tc_commit_mask<CG>(&empty[stage], 0x3u);
                    if (++stage == n_stages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit_mask<CG>(&acc_full[acc], 0x3u);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok && issued_any) {
                tc_commit_local<CG>(drain);
                drain_bounded(drain, 0, grp.wait_limit_ns);
            }
        }
    } else {
        const int e = warp - 2;
        const int quarter = warp & 3;  // a warp may only touch TMEM lanes 32 (warp mod 4) .. +31
        const int half = e >> 2;
        const AbortCtx ab_acc{abort_flag, grp.status, grp.acc_wait_limit_ns};
        int acc = 0;
        uint32_t acc_phase = 0;
        WarpOut<(C::kStaging > 0)> out{nullptr, grp.to, 0, 0, smem_addr(staging) + static_cast<uint32_t>(e) * 4096u, 0};
        if constexpr (C::kStaging > 0) out.maps = grp.outs;
        UnitCursor cur;
        int l = 0;
        stream_wait();
        float unit = 1.0f;
        if constexpr (EPI == kBlockLossGrad) unit = loss_unit(grp.prob[0], blockIdx.x == 0 && e == 0);
        if (blockIdx.x == 0)
            for (int i = threadIdx.x - 64; i < grp.zero_n; i += C::kThreads - 64) grp.zero_at[i] = 0u;
        for (int u = cur.next(grp.units, pair, pairs); u >= 0; u = cur.next(grp.units, pair, pairs)) {
            const Unit w = unit_of(grp, u, l);
            l = w.prob;
            const BlockProblem& b = grp.prob[l];
            const int row = w.mb * kBM * CG + static_cast<int>(rank) * kBM + quarter * 32 + lane;
            int ok = 1;
            if (lane == 0) ok = wait_bounded(&acc_full[acc], acc_phase, ab_acc) ? 1 : 0;
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const AccTmem tm{tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN)};
            if constexpr (EPI == kBlockStore) {
                out.to = &grp.to[l];
            }
            out.ld = b.ld;
            out.rows = b.rows;
            if (w.split < 0) block_epilogue<BN, EPI>(b, tm, row, w.nb, half, out, unit);
            // [split tile][part][CTA][lane quarter][column][lane]
            const size_t step = static_cast<size_t>(CG) * 4 * BN * 32;
            const size_t own = (static_cast<size_t>(rank) * 4 + quarter) * BN * 32 + lane;
            if (w.split >= 0) {
                float* p = grp.parts + b.part_base +
                           (static_cast<size_t>(w.split) * b.parts + w.part) * step + own;
                // the columns whose epilogue this warp runs: gate and up columns come from both halves
                constexpr int kRuns = kGated ? 2 : 1, kRun = BN / 2 / kRuns, kStep = kRun < 32 ? kRun : 32;
#pragma unroll 1
                for (int r = 0; r < kRuns; ++r) {
#pragma unroll 1
                    for (int c = 0; c < kRun; c += kStep) {
                        const int at = r * (BN / 2) + half * kRun + c;
                        uint32_t g[kStep];
                        tm.load(at, g);
                        if (row < b.rows) {
#pragma unroll
                            for (int j = 0; j < kStep; ++j)
                                __stcg(p + static_cast<size_t>(at + j) * 32, __uint_as_float(g[j]));
                        }
                    }
                }
            }
            // the accumulator's reads are done: it may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(map_to_rank(smem_addr(&acc_empty[acc]), 0));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            if (w.split >= 0) {
                // every lane's values are visible device-wide before the warp counts itself in; the
                // last one to arrive sees the other parts' values
                __threadfence();
                __syncwarp();
                uint32_t before = 0;
                uint32_t* count = grp.counts + b.count_base + (w.split * CG + static_cast<int>(rank)) * C::kEpiWarps + e;
                if (lane == 0) before = atomicAdd(count, 1u);
                before = __shfl_sync(0xFFFFFFFFu, before, 0);
                if (before + 1 == static_cast<uint32_t>(b.parts)) {
                    __threadfence();
                    if (lane == 0) *count = 0u;
                    const AccParts sum{grp.parts + b.part_base + static_cast<size_t>(w.split) * b.parts * step + own,
                                       step, b.parts, row < b.rows};
                    block_epilogue<BN, EPI>(b, sum, row, w.nb, half, out, unit);
                }
            }
        }
        out.end();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0 && lane == 0 && rank == 0 && *abort_flag) {
        uint64_t n_peer = n_issued;
        bool counted = true;
        if constexpr (CG == 2) {
            counted = false;
            const uint64_t t0 = global_timer_ns();
            while (!counted && global_timer_ns() - t0 <= 4 * grp.wait_limit_ns) counted = mbar_try_wait_cluster(peer_done, 0);
            if (counted) n_peer = ld_shared_volatile_u64(peer_count);
        }
        if (counted) drain_ring<CG>(full, n_stages, n_issued, n_peer, withheld, stage_bytes, grp.wait_limit_ns);
        else drain_ring<1>(full, n_stages, n_issued, n_issued, withheld, stage_bytes, grp.wait_limit_ns);
    }
    if constexpr (CG > 1) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, C::kTmemCols);
    }
}

}  // namespace forge
