// expert_kernel.cuh -- the persistent matrix-product kernel of products grouped by expert.
//
// Rows of X lie sorted by expert: expert e owns rows off_e .. off_{e+1}-1 of it and a matrix W_e of its own.  The
// offsets are on the device (a router leaves them there), so the host knows the number of rows and of experts
// but no expert's share.  Three kinds of product:
//   rows by expert      Y[r] = X[r] W_e^T, dX[r] = dY[r] W_e for r of expert e: tiles of rows, each of one expert
//   gated block         the same with the epilogues of block_kernel.cuh: G, U, H of the forward pass in one tile,
//                       dG, dU, H of the backward pass behind dH
//   weights' gradients  dW_e = sum over r of dY[r]^T X[r]: tiles of each dW_e, the reduction as long as e's run
// The pipeline, tiles, roles, bounded waits and drains are those of forge_block_kernel.
//
// Ragged runs.  A launch in front (expert_plan_kernel) turns the offsets into a list of row tiles and, for the
// weights' gradients, into a tensor map per expert and operand (a linear layer's two, a gated block's five) whose token
// dimension ends with the run: the copy itself fills what a slice reaches past the run with zeros, for both operands, so
// neither values of the next expert nor its infinities or NaN enter a sum.  An expert without rows takes one slice of zero
// fill and stores a zero gradient.  Row products need no such maps: a row of the result depends on its own row of X alone,
// and rows past the run are not stored.
//
// Few tiles.  The plan knows how many row tiles there are; where the last wave of tiles leaves SMs idle it cuts them
// along the reduction (expert_parts), and the parts are joined as in forge_block_kernel: no CTA waits for another, the
// last to arrive adds the parts in their order.  Gradients of few tiles are cut along their runs by the host's rule, the
// same number of parts for each: a run of fewer slices leaves some parts a slice of zeros.
#pragma once

#include "block_kernel.cuh"

namespace forge {

constexpr int kExpertGrad = 5, kExpertBoth = 6;
// Beside BlockEpi's kBlockStore, kBlockGatedFwd and kBlockGatedBwd, whose A are rows by expert: kExpertGrad, up to three
// weights' gradients, and kExpertBoth, the same behind a row product (dX) in one launch.  (One kernel for both cost the
// gradients alone 3 %: 512 rows of 64 experts, gated backward 2048/1408: 383 us against 370.)
__host__ __device__ constexpr bool expert_grads(int epi) { return epi == kExpertGrad || epi == kExpertBoth; }
// The first gradient's place among the products, and the products.
__host__ __device__ constexpr int expert_first_grad(int epi) { return epi == kExpertBoth ? 1 : 0; }
__host__ __device__ constexpr int expert_products(int epi) { return expert_grads(epi) ? expert_first_grad(epi) + 3 : 1; }

// On pairs every epilogue works in shared memory: 4 KiB a warp.
template <int BN, int CG, int EPI>
using ExpertCfg = BlockCfg<BN, CG, EPI, CG == 2>;

struct ExpertProblem {
    int cols;             // of the result (gated forward: d_ff, a tile spans BN / 2 of them)
    int tiles_n;          // column tiles
    int rows, tiles_m;    // gradients: rows of each expert's result, and their tiles
    int unit_start;       // gradients: number of its first unit among theirs
    int kb[2];            // rows by expert: 64-deep reduction slices of the two operand pairs
    int a_flat, b_flat;   // MN-major and no multiple of 64 wide: a copy for each 64 columns
    int b_mn;             // row products: W is read MN-major
    int map_a, map_b;     // gradients: numbers of the operands' run maps
    int64_t ld;           // the result's width
};

template <int EPI>
struct ExpertGroup {
    int n;                // products
    int n_units;          // of gradients
    int chunk;            // neighbouring units of gradients that a pair or CTA takes
    int ways;             // parts into which each of the gradients' tiles is cut along its run (single CTAs); n_units counts them
    int experts;
    int a_rows;           // rows of A that a stage holds, and of a tile on single CTAs (128, 64 or 32)
    int stream_b;         // each weight is read by one row tile or few: leave it out of the L2
    int act, keep;
    int withhold_first_stage;
    const int4* cut;      // row products: tiles before .x are whole, the others cut into .y parts; .z units
    const int* n_tiles;   // row tiles
    const int4* tiles;    // each: expert, first row, one past its last row
    const int* offsets;   // [experts + 1], as the plan left them: in order and within the rows
    const CUtensorMap* runs;  // [map][expert]
    const uint16_t* g_in;
    const uint16_t* u_in;
    float* parts;         // of cut tiles
    uint32_t* counts;     // their arrivals: zero before the launch and after it
    int* status;
    uint64_t wait_limit_ns, acc_wait_limit_ns;
    uint16_t* to[expert_products(EPI) > 3 ? 4 : 3];  // results: kBlockStore's; of each product; G, U, H; dG, dU, H
    ExpertProblem prob[expert_products(EPI)];
    // rows by expert: the weights of each operand pair, or the gate's and the up projection's; then the rows of each pair
    CUtensorMap maps[EPI == kExpertGrad ? 1 : 4];
    CUtensorMap outs[expert_products(EPI)];  // gradients on pairs
};

struct ExpertUnit {
    int prob, expert, nb, row0, end;  // row0: the tile's first row of the result; end: one past its last
    int k_first, k_end;               // slices (rows by expert: of both operand pairs, one after the other)
    int split, part;                  // which cut tile, or -1
};

// How the last wave of a row product is cut: `tiles` tiles of kb slices on `width` pairs or CTAs.  A part costs its
// slices and its share of the join, in slices (the host's figures for the tile: TileCost).  Parts fit one wave.
struct ExpertCut {
    int tiles_n, kb, width, join, per_part;
};
constexpr int kExpertMinSlices = 8, kExpertMaxParts = 16;

FORGE_HD int expert_parts(const ExpertCut& c, int rest) {
    int best = 1, time = c.kb;
    for (int p = 2; p <= kExpertMaxParts && c.kb >= kExpertMinSlices * p && rest * p <= c.width; ++p) {
        const int t = (c.kb + p - 1) / p + c.join + c.per_part * p;
        if (t < time) {
            best = p;
            time = t;
        }
    }
    return best;
}

// The units of a pair or CTA: tiles of the row product one by one, then gradients, `chunk` neighbours at a time, beginning
// with the pairs that the row product's last wave left without a tile.
template <int EPI>
struct ExpertWalk {
    int u, left, jump, pairs;
    int rows, pair, chunk;
    __device__ __forceinline__ ExpertWalk(int pair_, int pairs_, int rows_, int chunk_)
        : u(pair_), left(1), jump(1 + (pairs_ - 1) * chunk_), pairs(pairs_), rows(rows_), pair(pair_), chunk(chunk_) {
        if (EPI == kExpertGrad) begin_grads(pair);
        if (EPI == kExpertBoth && u >= rows) behind_rows();
    }
    __device__ __forceinline__ void begin_grads(int at) {
        u = at * chunk;
        left = chunk;
    }
    __device__ __forceinline__ void behind_rows() {
        const int rest = rows % pairs;
        begin_grads(pair >= rest ? pair - rest : pair - rest + pairs);
        u += rows;
    }
    __device__ __forceinline__ void next() {
        if (!expert_grads(EPI) || (EPI == kExpertBoth && u < rows)) {
            u += pairs;
            if (EPI == kExpertBoth && u >= rows) behind_rows();
        } else if (--left > 0) {
            ++u;
        } else {
            u += jump;
            left = chunk;
        }
    }
};

// Rows of a row product's tile on a pair, as the MMA takes them.
__device__ __forceinline__ int expert_width(const ExpertUnit& w) { return (w.end - w.row0 + 31) / 32 * 32; }

template <int CG, int EPI>
__device__ __forceinline__ ExpertUnit expert_unit(const ExpertGroup<EPI>& g, int u, int n_tiles, int4 cut, int row_units) {
    ExpertUnit r;
    r.split = -1;
    r.part = r.k_first = 0;
    int mb;
    if (expert_grads(EPI) && (EPI == kExpertGrad || u >= row_units)) {
        u -= row_units;
        if (CG == 1 && EPI == kExpertGrad && g.ways > 1) {
            r.split = u / g.ways;
            r.part = u - r.split * g.ways;
            u = r.split;
        }
        r.prob = expert_first_grad(EPI);
        while (r.prob + 1 < g.n && u >= g.prob[r.prob + 1].unit_start) ++r.prob;
        const ExpertProblem& b = g.prob[r.prob];
        const int t = u - b.unit_start, per = b.tiles_m * b.tiles_n;
        r.expert = t / per;
        tile_coords(t - r.expert * per, TileOrder{b.tiles_m, b.tiles_n, 8, 0}, mb, r.nb);
        r.row0 = mb * kBM * CG;
        r.end = b.rows;
        const int run = __ldcg(g.offsets + r.expert + 1) - __ldcg(g.offsets + r.expert);
        r.k_end = run > 0 ? (run + kBK - 1) / kBK : 0;
        const int past = r.k_end > 0 ? r.k_end : 1;
        if (CG == 1 && EPI == kExpertGrad && g.ways > 1) {
            const int kb = r.k_end;
            r.k_first = static_cast<int>(static_cast<int64_t>(kb) * r.part / g.ways);
            r.k_end = static_cast<int>(static_cast<int64_t>(kb) * (r.part + 1) / g.ways);
        }
        if (r.k_end == r.k_first) r.k_first = r.k_end = past;  // one slice of zeros
    } else {
        const ExpertProblem& b = g.prob[0];
        r.prob = 0;
        r.k_end = b.kb[0] + b.kb[1];
        int t = u;
        if (u >= cut.x) {
            const int s = u - cut.x, kb = r.k_end;
            r.split = s / cut.y;
            r.part = s - r.split * cut.y;
            r.k_first = static_cast<int>(static_cast<int64_t>(kb) * r.part / cut.y);
            r.k_end = static_cast<int>(static_cast<int64_t>(kb) * (r.part + 1) / cut.y);
            t = cut.x + r.split;
        }
        tile_coords(t, TileOrder{n_tiles, b.tiles_n, 8, 0}, mb, r.nb);
        const int4 at = __ldcg(g.tiles + mb);
        r.expert = at.x;
        r.row0 = at.y;
        r.end = at.z;
    }
    return r;
}

// ---------------------------------------------------------------- row products on pairs
// The weights are the MMA's A (256 columns of the result, 128 a CTA) and the rows its B, whose width is any multiple
// of 32: the last tile of a run is as wide as the run's rest, not as a whole tile.  Against rows as A in tiles of 256, with
// maps of the runs (us): gated forward 2048 rows of 8 experts, 4096/14336, 769 to 693; 8192 of 64, 2048/1408, 236 to 220;
// linear forward 4637 of 6, 80 x 7224, 42.6 to 27.4.  With long runs the tensor pipe is 65-71 % active (4096 rows of 8,
// 4096 x 4096; 32768 of 64, 2048/1408).
//
// A warp's lanes are columns of the result and the accumulator's columns its rows, 32 at a time; results (and G and U on
// their way in) change sides in the warp's 4 KiB of shared memory, 32 rows of 64 bytes at a time, where both sides' accesses
// are free of conflicts.

__device__ __forceinline__ void st_shared_b16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_b16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A block of up to 32 rows x 32 columns of a matrix [.., ld] in memory: this warp's columns from col on.
struct ExpertBlock {
    uint32_t buf;      // 2 KiB of shared memory: row j's 32 columns at 64 j
    int row, rows;     // first row, and one past the last that there is
    int col, ld;
    // The block's first N rows out of shared memory (every lane's writes done).
    template <int N>
    __device__ __forceinline__ void write(uint16_t* to) const {
        const int lane = static_cast<int>(threadIdx.x & 31u), c = 8 * (lane & 3);
#pragma unroll
        for (int k = 0; k < N / 8; ++k) {
            const int r = (lane >> 2) + 8 * k;
            uint32_t v[4];
            ld_shared_v4(buf + static_cast<uint32_t>(r * 64 + 2 * c), v);
            if (row + r < rows && col + c < ld) st_v4(to + static_cast<size_t>(row + r) * ld + col + c, v);
        }
    }
    __device__ __forceinline__ void read(const uint16_t* from, uint32_t (&v)[4][4]) const {
        const int lane = static_cast<int>(threadIdx.x & 31u), c = 8 * (lane & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = (lane >> 2) + 8 * k;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = 0u;
            if (row + r < rows && col + c < ld) ld_v4(from + static_cast<size_t>(row + r) * ld + col + c, v[k]);
        }
    }
    __device__ __forceinline__ void keep(const uint32_t (&v)[4][4]) const {
        const int lane = static_cast<int>(threadIdx.x & 31u), c = 8 * (lane & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) st_shared_v4(buf + static_cast<uint32_t>(((lane >> 2) + 8 * k) * 64 + 2 * c), v[k][0], v[k][1], v[k][2], v[k][3]);
    }
    // This lane's column of row j.
    __device__ __forceinline__ uint32_t at(int j) const { return buf + static_cast<uint32_t>(64 * j + 2 * (threadIdx.x & 31)); }
    __device__ __forceinline__ void put(int j, float v) const { st_shared_b16(at(j), pack_bf16x2_rn(__float_as_uint(v), 0u)); }
};

// rows: of the tile; blocks of 32 of them go to the two warps of a lane quarter in turn
struct ExpertTile {
    int row0, rows, col, cols;
    int first, step;  // this warp's first row of the tile, and from block to block
};

template <class Acc>
__device__ __forceinline__ void epi_rows_store(const ExpertTile& t, const Acc& acc, uint16_t* to, uint32_t buf) {
    if (t.col >= t.cols) return;
#pragma unroll 1
    for (int j = t.first; j < t.rows; j += t.step) {
        uint32_t g[32];
        acc.load(j, g);
        const ExpertBlock b{buf, t.row0 + j, t.row0 + t.rows, t.col, t.cols};
        __syncwarp();  // the last block has been read
#pragma unroll
        for (int i = 0; i < 32; ++i) b.put(i, __uint_as_float(g[i]));
        __syncwarp();
        b.template write<32>(to);
    }
}

// The activation is the same for a launch: code of its own for each leaves a branch a block instead of one an element
// (gated forward, 4096 rows of 16 experts, 1024/2816: 94 us with it, 105 without).
template <class F>
__device__ __forceinline__ auto with_act(int act, F&& f) {
    if (act == kActSilu) return f(std::integral_constant<int, kActSilu>{});
    if (act == kActGeluTanh) return f(std::integral_constant<int, kActGeluTanh>{});
    return f(std::integral_constant<int, kActRelu>{});
}

template <int ACT, class Acc>
__device__ __forceinline__ void epi_rows_gated_bwd(const ExpertTile& t, const Acc& acc, const uint16_t* g_in, const uint16_t* u_in,
                                                   uint16_t* dg, uint16_t* du, uint16_t* h, uint32_t buf) {
    if (t.col >= t.cols) return;
#pragma unroll 1
    for (int j = t.first; j < t.rows; j += t.step) {
        const ExpertBlock a{buf, t.row0 + j, t.row0 + t.rows, t.col, t.cols}, b{buf + 2048u, t.row0 + j, t.row0 + t.rows, t.col, t.cols};
        uint32_t g[4][4], u[4][4];
        a.read(g_in, g);
        b.read(u_in, u);
        uint32_t d[32], hs[16];
        acc.load(j, d);
        __syncwarp();  // the last block has been read
        a.keep(g);
        b.keep(u);
        __syncwarp();
        // each lane's places in the two buffers are its own from here on: dG and dU take those of G and U
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float gv = __uint_as_float(ld_shared_b16(a.at(i)) << 16), uv = __uint_as_float(ld_shared_b16(b.at(i)) << 16);
            const float dh = __uint_as_float(d[i]);
            float value, slope;
            act_both(gv, ACT, value, slope);
            a.put(i, dh * uv * slope);
            b.put(i, dh * value);
            const uint32_t r = pack_bf16x2_rn(__float_as_uint(value * uv), 0u);
            hs[i / 2] = i % 2 == 0 ? r : hs[i / 2] | r << 16;
        }
        __syncwarp();
        a.template write<32>(dg);
        b.template write<32>(du);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) st_shared_b16(a.at(i), hs[i / 2] >> (16 * (i % 2)));
        __syncwarp();
        a.template write<32>(h);
    }
}

// Two warps' barrier.
__device__ __forceinline__ void meet(int number) { asm volatile("bar.sync %0, 64;" ::"r"(number) : "memory"); }

// Whether two warps that meet inside a tile's epilogue both run it: the first to come to tile `no` decides for both, so that
// neither waits for one that has given up.  The word counts the tiles that are to be run (a warp with no columns to make may be
// some ahead of the other: it meets nobody), or says that the rest are left.  Each warp calls it once a tile until it answers 0.
__device__ __forceinline__ int expert_agree(uint32_t* word, uint32_t no, int ok) {
    const uint32_t run = no + 1, leave = 0xFFFFFFFFu;
    const uint32_t before = atomicCAS(word, no, ok ? run : leave);
    return before == no ? ok : before != leave;
}

// G and U of the same columns are in the lanes of two warps (quarters 0 and 2, 1 and 3), which trade 16 rows of each
// block and make H of 16 rows each.  They meet on a barrier of theirs (`meeting`) when their rows are in shared memory and
// again when they have read the other's; that both run the tile is settled before (expert_agree).
template <int ACT, class Acc>
__device__ __forceinline__ void epi_rows_gated_fwd(const ExpertTile& t, const Acc& acc, bool is_up, bool keep, uint16_t* own,
                                                   uint16_t* h, uint32_t buf, uint32_t other, int meeting) {
    const uint32_t lane = threadIdx.x & 31u, mine = buf + 2048u + 4u * lane, theirs = other + 2048u + 4u * lane;
    const bool inside = t.col < t.cols;  // the same for both warps
#pragma unroll 1
    for (int j = t.first; j < t.rows; j += t.step) {
        uint32_t v[32];
        acc.load(j, v);
        const ExpertBlock b{buf, t.row0 + j, t.row0 + t.rows, t.col, t.cols};
#pragma unroll
        for (int i = 0; i < 16; ++i) st_shared_f32(mine + 128u * i, __uint_as_float(is_up ? v[i] : v[16 + i]));
        meet(meeting);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = ld_shared_f32(theirs + 128u * i);
        meet(meeting);
        if (!inside) continue;
        if (keep) {
            __syncwarp();  // the last block has been read
#pragma unroll
            for (int i = 0; i < 32; ++i) b.put(i, __uint_as_float(v[i]));
            __syncwarp();
            b.template write<32>(own);
        }
        // H is rounded to bfloat16, the type of the next product's operand
        const ExpertBlock c{buf, b.row + (is_up ? 16 : 0), b.rows, t.col, t.cols};
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            c.put(i, is_up ? act_value(x[i], ACT) * __uint_as_float(v[16 + i]) : act_value(__uint_as_float(v[i]), ACT) * x[i]);
        __syncwarp();
        c.template write<16>(h);
    }
}

// The weights' gradients on pairs leave in boxes of 32 rows x 64 columns, whole 128-byte lines: what a store's copy
// engine takes a row of a box, not a byte, sets the pace of tiles with few slices (2048 rows of 32 experts, 1024 x 2048
// weights, 134 MB of results: 39 us in boxes of 32 columns).
template <int BN, class Acc>
__device__ __forceinline__ void epi_expert_grad(const BlockProblem& b, const Acc& acc, int row, int nb, int h, const CUtensorMap* map,
                                                int expert, uint32_t buf) {
    const int row0 = warp_row0(row);
    if (row0 >= b.rows) return;
    const uint32_t lane = threadIdx.x & 31u;
#pragma unroll 1
    for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 64) {
        const int col = nb * BN + c;
        if (b.cols - col <= 0) break;  // the same for the whole warp
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t g[32];
            acc.load(c + 32 * i, g);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[16 * i + j] = pack_bf16x2_rn(g[2 * j], g[2 * j + 1]);
        }
        if (lane == 0) bulk_wait_read<0>();  // the last box has left the buffer
        __syncwarp();
        // the 128-byte swizzle: 16-byte piece j of row r lies at piece j ^ (r mod 8)
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            st_shared_v4(buf + lane * 128u + ((j ^ (lane & 7u)) << 4), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, buf, col, row0, expert);
            bulk_commit();
        }
    }
}

template <int BN, int CG, int EPI>
__global__ void __launch_bounds__(ExpertCfg<BN, CG, EPI>::kThreads, 1)
    forge_expert_kernel(const __grid_constant__ ExpertGroup<EPI> grp) {
    using C = ExpertCfg<BN, CG, EPI>;
    constexpr bool kGated = EPI == kBlockGatedFwd, kGrads = expert_grads(EPI), kRows = EPI != kExpertGrad;
    constexpr bool kMeets = kGated && CG == 2;  // two warps meet in an epilogue
    constexpr bool kCuts = CG == 1 ? EPI != kExpertBoth : EPI == kBlockStore;  // tiles may be cut
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
    uint32_t* agreed = reinterpret_cast<uint32_t*>(peer_count + 1);  // by the two warps that hold G and U of the same columns
    uint32_t* tmem_slot = agreed + 4;
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
        for (int i = 0; i < 4; ++i) agreed[i] = 0u;
        *abort_flag = 0;
        fence_mbar_init();
        if constexpr (kRows) {
            tma_prefetch_desc(&grp.maps[0]);
            if constexpr (kGated) tma_prefetch_desc(&grp.maps[1]);
            tma_prefetch_desc(&grp.maps[2]);
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
    const uint32_t tmem_base = *tmem_slot;
    const AbortCtx ab{abort_flag, grp.status, grp.wait_limit_ns};
    uint64_t n_issued = 0;
    int64_t withheld = -1;

    stream_wait();
    const int n_tiles = kRows ? __ldcg(grp.n_tiles) : 0;
    const int4 cut = kRows ? __ldcg(grp.cut) : make_int4(0, 1, 0, 0);
    const int row_units = cut.z, n_units = row_units + (kGrads ? grp.n_units : 0);
    const int chunk = kGrads ? grp.chunk : 1;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint64_t keep = policy_evict_last();
            const uint64_t pol_b = grp.stream_b ? policy_evict_first() : keep;
            const bool leader = rank == 0;
            const bool withhold = grp.withhold_first_stage && leader;
            const uint32_t bars = CG == 2 ? map_to_rank(smem_addr(full), 0) : smem_addr(full);
            const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * 128u;
            const uint32_t a_ring = smem_addr(sA), b_ring = smem_addr(sB);
            // one slice: waits for its slot, arms it and copies into it
            auto slice = [&](auto&& copies) {
                if (!wait_bounded(&empty[stage], phase ^ 1u, ab)) return false;
                if (leader) mbar_arrive_expect_tx(&full[stage], CG * stage_bytes);
                if (withhold && n_issued == 0) {
                    withheld = 0;  // test switch: arm this stage but never copy into it
                } else {
                    copies(bars + 8u * static_cast<uint32_t>(stage), a_ring + static_cast<uint32_t>(stage) * a_bytes,
                           b_ring + static_cast<uint32_t>(stage) * C::kBBytes);
                }
                ++n_issued;
                if (++stage == n_stages) { stage = 0; phase ^= 1u; }
                return true;
            };
            int seen_prob = -1, seen_expert = -1;
            for (ExpertWalk<EPI> at(pair, pairs, row_units, chunk); ok && at.u < n_units; at.next()) {
                const ExpertUnit w = expert_unit<CG, EPI>(grp, at.u, n_tiles, cut, row_units);
                const ExpertProblem& b = grp.prob[w.prob];
                const int row_a = w.row0 + static_cast<int>(rank) * kBM;
                const int col_b = kGated ? w.nb * kColsPerTile : w.nb * BN + static_cast<int>(rank) * C::kBLoad;
                if (kGrads && (!kRows || at.u >= row_units)) {
                    const CUtensorMap* ma = grp.runs + static_cast<size_t>(b.map_a) * grp.experts + w.expert;
                    const CUtensorMap* mb = grp.runs + static_cast<size_t>(b.map_b) * grp.experts + w.expert;
                    if (w.prob != seen_prob || w.expert != seen_expert) {
                        tensormap_acquire(ma);
                        tensormap_acquire(mb);
                        seen_prob = w.prob;
                        seen_expert = w.expert;
                    }
                    // a part of no slices takes one past its run (a run of no rows: past the one row that its maps have)
                    int k0 = w.k_first * kBK;
                    const bool a_flat = b.a_flat != 0, b_flat = b.b_flat != 0;
                    const int a0 = a_flat ? row_a : 0, a2 = a_flat ? 0 : row_a / 64;
                    const int b0 = b_flat ? col_b : 0, b2 = b_flat ? 0 : col_b / 64;
                    for (int n = w.k_end == w.k_first ? 1 : w.k_end - w.k_first; ok && n > 0; --n, k0 += kBK)
                        ok = slice([&](uint32_t bar, uint32_t a_dst, uint32_t b_dst) {
                            tma_load_3d_cg<CG>(a_dst, ma, bar, a0, k0, a2, keep);
                            tma_load_3d_cg<CG>(b_dst, mb, bar, b0, k0, b2, keep);
                            if (a_flat) tma_load_3d_cg<CG>(a_dst + kBK * 128, ma, bar, a0 + 64, k0, 0, keep);
                            if (b_flat) tma_load_3d_cg<CG>(b_dst + kBK * 128, mb, bar, b0 + 64, k0, 0, keep);
                        });
                } else if constexpr (CG == 2) {
                    // the weights' 128 columns of the result, or 64 of the gate's rows and 64 of the up projection's
                    const bool wmn = EPI == kBlockGatedBwd || (!kGated && b.b_mn != 0), w_flat = wmn && b.b_flat != 0;
                    const int col = w.nb * kColsPerTile + static_cast<int>(rank) * (kColsPerTile / 2);
                    const int row = w.row0 + static_cast<int>(rank) * (expert_width(w) / 2);
#pragma unroll 1
                    for (int seg = 0; seg < (EPI == kBlockStore || kGrads ? 2 : 1) && ok; ++seg) {
                        // the unit's slices of this operand pair
                        const int base = seg == 0 ? 0 : b.kb[0];
                        const int from = w.k_first > base ? w.k_first - base : 0;
                        const int to = (w.k_end < base + b.kb[seg] ? w.k_end : base + b.kb[seg]) - base;
                        const CUtensorMap* mr = &grp.maps[2 + seg];
                        const CUtensorMap* mw = &grp.maps[seg];
                        const CUtensorMap* mu = &grp.maps[1];
                        int k0 = from * kBK, w0 = wmn ? (w_flat ? col : 0) : k0, w1 = wmn ? k0 : col;
                        const int w2 = wmn && !w_flat ? col / 64 : 0, dw0 = wmn ? 0 : kBK, dw1 = wmn ? kBK : 0;
#pragma unroll 1
                        for (int n = to - from; ok && n > 0; --n, k0 += kBK, w0 += dw0, w1 += dw1)
                            ok = slice([&](uint32_t bar, uint32_t a_dst, uint32_t b_dst) {
                                tma_load_4d_cg<CG>(a_dst, mw, bar, w0, w1, w2, w.expert, pol_b);
                                tma_load_3d_cg<CG>(b_dst, mr, bar, k0, row, 0, keep);
                                if (kGated) tma_load_4d_cg<CG>(a_dst + 64 * 128, mu, bar, w0, w1, 0, w.expert, pol_b);
                                if (!kGated && w_flat) tma_load_4d_cg<CG>(a_dst + kBK * 128, mw, bar, w0 + 64, w1, 0, w.expert, pol_b);
                            });
                    }
                } else {
                    const bool bmn = EPI == kBlockGatedBwd || (!kGated && b.b_mn != 0);
                    const bool b_flat = bmn && b.b_flat != 0;
#pragma unroll 1
                    for (int seg = 0; seg < (EPI == kBlockStore || kGrads ? 2 : 1) && ok; ++seg) {
                        // the unit's slices of this operand pair
                        const int base = seg == 0 ? 0 : b.kb[0];
                        const int from = w.k_first > base ? w.k_first - base : 0;
                        const int to = (w.k_end < base + b.kb[seg] ? w.k_end : base + b.kb[seg]) - base;
                        const CUtensorMap* ma = &grp.maps[2 + seg];
                        // gated forward: the first half of the columns holds the gate's rows, the other the up
                        // projection's, of the same d_ff columns
                        const CUtensorMap* mb = &grp.maps[seg];
                        const CUtensorMap* mu = &grp.maps[1];
                        int k0 = from * kBK;
                        int b0 = bmn ? (b_flat ? col_b : 0) : k0, b1 = bmn ? k0 : col_b;
                        const int b2 = bmn && !b_flat ? col_b / 64 : 0;
                        const int db0 = bmn ? 0 : kBK, db1 = bmn ? kBK : 0;
#pragma unroll 1
                        for (int n = to - from; ok && n > 0; --n, k0 += kBK, b0 += db0, b1 += db1)
                            ok = slice([&](uint32_t bar, uint32_t a_dst, uint32_t b_dst) {
                                tma_load_3d_cg<CG>(a_dst, ma, bar, k0, row_a, 0, keep);
                                tma_load_4d_cg<CG>(b_dst, mb, bar, b0, b1, b2, w.expert, pol_b);
                                if (kGated) tma_load_4d_cg<CG>(b_dst + BN / 2 * 128, mu, bar, b0, b1, 0, w.expert, pol_b);
                                if (!kGated && b_flat)
                                    tma_load_4d_cg<CG>(b_dst + kBK * 128, mb, bar, b0 + 64, b1, 0, w.expert, pol_b);
                            });
                    }
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
        if (lane == 0 && rank == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued_any = false;
            for (ExpertWalk<EPI> at(pair, pairs, row_units, chunk); ok && at.u < n_units; at.next()) {
                const ExpertUnit w = expert_unit<CG, EPI>(grp, at.u, n_tiles, cut, row_units);
                const bool grad = kGrads && (!kRows || at.u >= row_units), swapped = CG == 2 && !grad;
                const bool wmn = EPI == kBlockGatedBwd || (!kGated && grp.prob[0].b_mn != 0);  // the weights' order
                const bool amn = grad || (swapped && wmn), bmn = grad || (!swapped && wmn);
                const uint32_t idesc = idesc_bf16_f32(kBM * CG, swapped ? expert_width(w) : BN, amn, bmn);
                const uint32_t a_step = (amn ? 2048u : 32u) >> 4, b_step = (bmn ? 2048u : 32u) >> 4;
                const uint64_t a_desc = smem_desc_sw128(smem_addr(sA), amn ? kBK * 128u : 16u, 1024);
                const uint64_t b_desc = smem_desc_sw128(smem_addr(sB), bmn ? kBK * 128u : 16u, 1024);
                if (!wait_bounded(&acc_empty[acc], acc_phase ^ 1u, ab)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                const int slices = w.k_end == w.k_first ? 1 : w.k_end - w.k_first;
#pragma unroll 1
                for (int kb = 0; kb < slices; ++kb) {
                    if (!wait_bounded(&full[stage], phase, ab)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = a_desc + static_cast<uint32_t>(stage) * (static_cast<uint32_t>(a_rows) * 128u >> 4);
                    const uint64_t bd = b_desc + static_cast<uint32_t>(stage) * (C::kBBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk)
                        tc_mma_bf16<CG>(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, (kb | kk) != 0 ? 1u : 0u);
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
        WarpOut<false> out{nullptr, grp.to, 0, 0, 0, 0};
        uint16_t* grad_to[1];
        const uint32_t buf = smem_addr(staging) + static_cast<uint32_t>(e) * 4096u;
        uint32_t tile_no = 0;
        for (ExpertWalk<EPI> at(pair, pairs, row_units, chunk); at.u < n_units; at.next()) {
            const ExpertUnit w = expert_unit<CG, EPI>(grp, at.u, n_tiles, cut, row_units);
            const ExpertProblem& p = grp.prob[w.prob];
            const int row = w.row0 + static_cast<int>(rank) * kBM + quarter * 32 + lane;
            BlockProblem b;
            b.rows = w.end;
            b.cols = p.cols;
            b.ld = p.ld;
            b.add = nullptr;
            b.unit = nullptr;
            b.sum_in = b.sum_out = 0;
            b.act = grp.act;
            b.keep = grp.keep;
            b.g_in = grp.g_in;
            b.u_in = grp.u_in;
            out.ld = p.ld;
            out.rows = w.end;
            const bool grad = kGrads && (!kRows || at.u >= row_units);
            if constexpr (kGrads) {
                const size_t each = static_cast<size_t>(p.rows) * static_cast<size_t>(p.ld);
                grad_to[0] = grp.to[w.prob] + (grad ? each * static_cast<size_t>(w.expert) : 0);
                out.to = grad_to;
            }
            int ok = 1;
            if (lane == 0) {
                ok = wait_bounded(&acc_full[acc], acc_phase, ab_acc) ? 1 : 0;
                if constexpr (kMeets) ok = expert_agree(&agreed[2 * half + (quarter & 1)], tile_no, ok);
            }
            ++tile_no;
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const AccTmem tm{tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN)};
            const int meeting = 2 * half + (quarter & 1);  // kMeets: which two warps
            const int col = w.nb * kColsPerTile + static_cast<int>(rank) * (kColsPerTile / 2) + (kGated ? quarter & 1 : quarter) * 32;
            const ExpertTile t{w.row0, w.end - w.row0, col, p.cols, half * 32, 64};  // on pairs
            auto epilogue = [&](const auto& acc_from) {
                if constexpr (CG == 2 && EPI == kBlockGatedFwd) {
                    const bool is_up = quarter >= 2;
                    const uint32_t other = smem_addr(staging) + static_cast<uint32_t>(half * 4 + quarter) * 4096u;
                    with_act(grp.act, [&](auto a) {
                        epi_rows_gated_fwd<decltype(a)::value>(t, acc_from, is_up, grp.keep != 0, grp.to[is_up ? 1 : 0], grp.to[2], buf,
                                                               other, 1 + meeting);
                    });
                } else if constexpr (CG == 2 && EPI == kBlockGatedBwd) {
                    with_act(grp.act, [&](auto a) {
                        epi_rows_gated_bwd<decltype(a)::value>(t, acc_from, grp.g_in, grp.u_in, grp.to[0], grp.to[1], grp.to[2], buf);
                    });
                } else if constexpr (CG == 2) {
                    epi_rows_store(t, acc_from, grp.to[0], buf);
                } else if constexpr (EPI == kBlockGatedFwd) {
                    epi_gated_fwd<BN>(b, acc_from, row, w.nb, half, out);
                } else if constexpr (EPI == kBlockGatedBwd) {
                    epi_gated_bwd<BN>(b, acc_from, row, w.nb, half, out);
                } else {
                    epi_store<BN>(b, acc_from, row, w.nb, half, out);
                }
            };
            // [cut tile][part][CTA][lane quarter][column][lane]; quarters past a single CTA's tile are not there
            const size_t step = static_cast<size_t>(CG) * (a_rows / 32) * BN * 32;
            const size_t own = (static_cast<size_t>(rank) * (a_rows / 32) + quarter) * BN * 32 + lane;
            const bool whole = !kCuts || w.split < 0;
            const int ways = kGrads ? grp.ways : cut.y;
            float* const part = grp.parts + (static_cast<size_t>(w.split) * ways + w.part) * step + own;  // of a cut tile
            if (CG == 2 && grad) {
                if constexpr (CG == 2 && kGrads) epi_expert_grad<BN>(b, tm, row, w.nb, half, grp.outs + w.prob, w.expert, buf);
            } else if (whole) {
                epilogue(tm);
            } else if constexpr (!kCuts) {
            } else if constexpr (CG == 2) {
#pragma unroll 1
                for (int j = t.first; t.col < t.cols && j < t.rows; j += t.step) {
                    uint32_t g[32];
                    tm.load(j, g);
#pragma unroll
                    for (int i = 0; i < 32; ++i) __stcg(part + static_cast<size_t>(j + i) * 32, __uint_as_float(g[i]));
                }
            } else if (warp_row0(row) < b.rows) {
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
                                __stcg(part + static_cast<size_t>(at + j) * 32, __uint_as_float(g[j]));
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
            if constexpr (kCuts) {
                if (whole) continue;
                // every lane's values are visible device-wide before the warp counts itself in; the last one to
                // arrive sees the other parts' values
                __threadfence();
                __syncwarp();
                uint32_t before = 0;
                uint32_t* count = grp.counts + (w.split * CG + static_cast<int>(rank)) * C::kEpiWarps + e;
                if (lane == 0) before = atomicAdd(count, 1u);
                before = __shfl_sync(0xFFFFFFFFu, before, 0);
                if (before + 1 == static_cast<uint32_t>(ways)) {
                    __threadfence();
                    if (lane == 0) *count = 0u;
                    epilogue(AccParts{grp.parts + static_cast<size_t>(w.split) * ways * step + own, step, ways, CG == 2 || row < b.rows});
                }
            }
        }
        if constexpr (kGrads && CG == 2) {
            if (lane == 0) bulk_wait_read<0>();  // shared memory stays until the last stores have read it
        }
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
