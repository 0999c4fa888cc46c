// expert_api.cu -- the C ABI of the products grouped by expert (include/forge.h): a linear layer and the gated
// feed-forward block with a weight for each expert.  Argument checks, the plan made from the offsets on the
// device, workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "block_host.h"
#include "expert_kernel.cuh"
#include "expert_launch.h"
#include "forge.h"
#include "host.h"

namespace {

namespace host = forge::host;
using namespace forge::host;
using forge::ExpertGroup;
using forge::ExpertProblem;
using forge::kBlockGatedBwd;
using forge::kBlockGatedFwd;
using forge::kBlockStore;
using forge::kExpertBoth;
using forge::kExpertGrad;

constexpr int kMaxExperts = 1024;  // the plan gives each a thread of its one block
constexpr int kMaxCuts = 2;        // row products of a call
constexpr int kMaxRuns = 5;        // operands of gradients, which end with a run of rows: dG, dU, dY, X, H

int slices(int64_t k) { return static_cast<int>(ceil_div(k, forge::kBK)); }

// ---------------------------------------------------------------- the plan, made on the device

struct RunOperand {
    CUtensorMap map;  // of 64 columns of one row: tensormap_set widens it
    const char* base;
    int64_t pitch;    // bytes from row to row
    uint32_t dim0, dim2;
};

struct PlanArgs {
    const int* offsets;
    int experts, rows, tile_rows;
    int* clean;     // [experts + 1]
    int* n_tiles;
    int4* tiles;
    CUtensorMap* runs;  // [n_runs][experts]
    int n_runs;
    int4* cuts;     // of each row product
    int n_cuts;
    forge::ExpertCut cut[kMaxCuts];
    uint32_t* counts;
    int n_counts;
    RunOperand run[kMaxRuns];
};

// Inclusive scan over the block's threads of values that are not negative; 0 is neutral.
template <class Op>
__device__ __forceinline__ int block_scan(int v, int* warps, Op op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v = op(v, n);
    }
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = lane < static_cast<int>(blockDim.x >> 5) ? warps[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int n = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w = op(w, n);
        }
        warps[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v = op(v, warps[warp - 1]);
    __syncthreads();
    return v;
}

// One block: thread e is expert e, and there are as many threads as there are experts, maps or tiles to deal out (up to
// 1024).  Offsets are brought into order and within the rows (an offset below the one
// before it, or past the last row, ends an empty or a shorter run), so that no later launch can leave the
// tensors whatever they hold.
__global__ void __launch_bounds__(1024) expert_plan_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ int warps[32], first[kMaxExperts], begin[kMaxExperts], end[kMaxExperts], total;
    forge::stream_wait();
    const int e = threadIdx.x;
    const bool mine = e < a.experts;
    auto inside = [&](int i) { return min(max(__ldcg(a.offsets + i), 0), a.rows); };
    const int from = block_scan(mine ? inside(e) : 0, warps, [](int x, int y) { return max(x, y); });
    const int to = mine ? max(from, inside(e + 1)) : from;
    if (mine) {
        a.clean[e] = from;
        if (e + 1 == a.experts) a.clean[a.experts] = to;
    }
    const int tiles = (to - from + a.tile_rows - 1) / a.tile_rows;
    const int last = block_scan(tiles, warps, [](int x, int y) { return x + y; });
    first[e] = last - tiles;
    begin[e] = from;
    end[e] = to;
    if (e + 1 == a.experts) total = *a.n_tiles = last;
    __syncthreads();
    const int threads = static_cast<int>(blockDim.x);
    for (int i = e; i < total; i += threads) {
        int lo = 0, hi = a.experts - 1;  // the last expert whose first tile is not behind tile i
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (first[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int row = begin[lo] + (i - first[lo]) * a.tile_rows;
        a.tiles[i] = make_int4(lo, row, min(row + a.tile_rows, end[lo]), 0);
    }
    if (e < a.n_cuts) {
        const forge::ExpertCut& c = a.cut[e];
        const int all = total * c.tiles_n, rest = all % c.width;
        const int parts = forge::expert_parts(c, rest);
        const int from = parts > 1 ? all - rest : all;
        a.cuts[e] = make_int4(from, parts, from + (all - from) * parts, 0);
    }
    for (int i = e; i < a.n_counts; i += threads) a.counts[i] = 0u;
    for (int i = e; i < a.n_runs * a.experts; i += threads) {
        const int o = i / a.experts, x = i - o * a.experts;
        const uint4* src = reinterpret_cast<const uint4*>(&a.run[o].map);
        uint4* dst = reinterpret_cast<uint4*>(a.runs + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = src[j];
        // a run of no rows: one row that is never read (its slice lies past it)
        const int n = end[x] - begin[x];
        forge::tensormap_set(a.runs + i, a.run[o].base + (n > 0 ? begin[x] * a.run[o].pitch : 0), a.run[o].dim0, n > 0 ? n : 1,
                             a.run[o].dim2);
    }
}

// ---------------------------------------------------------------- tiles

struct Tiling {
    int bn;         // tile columns: 256 on CTA pairs, 128 on single CTAs
    int tile_rows;  // rows of a row tile
};

// A call's rows, experts and plan in its workspace.
struct Call {
    Machine mc;
    int64_t rows;
    int experts;
    Tiling tiling;
    int64_t tiles;  // row tiles at most
    int n_runs;
    int64_t clean, n_tiles, list, runs, cuts, counts, parts;  // places in the workspace
    int n_counts;                    // of row products, then of gradients
    int grad_ways, grad_counts;      // parts of each gradient tile, and where their arrivals are counted
    int64_t grad_parts;
    forge::ExpertCut cut[kMaxCuts];  // of the call's row products, in the order of their launches
    int n_cuts;
    char* ws;
    cudaStream_t stream;
    const int* offsets;
};

// Row tiles, by the rows that an expert has on average: 256 on pairs, 128, 64 or 32 on single CTAs, whose copies of A
// are as many rows.  Gated forward, 2048/1408, 64 experts, us on 256 / 128 / 64 / 32 rows: 8 rows each 189 / 186 / 181 / 180;
// 32: 195 / 190 / 191 / 230; 64: 200 / 199 / 230; 128: 218 / 242; 256: 278 / 360.  4096/14336, 8 experts: 128 rows each 508 / 565;
// 16: 454 / 443 / 432 / 441; one row of two experts 174 / 169 / 132 / 120.
Tiling choose_rows(int64_t rows, int64_t experts) {
    const int64_t each = rows / std::min(rows, experts);
    if (each > 90) return Tiling{256, 256};
    return Tiling{128, each > 40 ? 128 : each > 4 ? 64 : 32};
}

// dW of up to three products: a and b, numbers of their run operands; each dW_e [d_out, d_in]
struct GradProduct {
    int a, b;
    int64_t d_out, d_in;
    void* out;
};

Tiling grad_tiling(const Machine& mc, int64_t experts, const GradProduct* p, int n) {
    int64_t pairs = 0;
    for (int i = 0; i < n; ++i) pairs += experts * ceil_div(p[i].d_out, 256) * ceil_div(p[i].d_in, 256);
    return pairs >= mc.pairs ? Tiling{256, 256} : Tiling{128, 128};
}

// The tiles of a linear layer's backward pass that wants dX and dW, and whether one launch makes both: dX's units first,
// the gradients' behind them and beside its last wave.  It does with short runs, where both have the same tiles;
// experts of over 40 rows take pairs for that.  us in two launches / in one: 2048 rows of 32 experts, 1024 x 2048 66 / 61;
// 1003 of 16, 1032 x 520 25 / 22; 200 of 3, 512 x 256 12.6 / 8.8; with long runs 30 / 33 (4096 of 4, 1024 x 1024).  The
// gated block's dX has long units (its two products), which are better cut in a launch of their own (1003 rows of 16
// experts, 520/1032: 60 us, 67 in one; 300 of 4, 1024/776 41 and 48).
struct BackwardTiles {
    Tiling rows, grads;
    bool together;
};
BackwardTiles linear_tiles(const Machine& mc, const forge_expert_linear_shape& s) {
    const GradProduct p{0, 0, s.d_out, s.d_in, nullptr};
    BackwardTiles t{choose_rows(s.rows, s.experts), grad_tiling(mc, s.experts, &p, 1), false};
    if (s.rows >= 256 * s.experts) return t;
    if (t.grads.bn == 256 && s.rows > 40 * std::min(s.rows, s.experts)) t.rows = Tiling{256, 256};
    t.together = t.rows.bn == t.grads.bn && t.rows.tile_rows >= 128;
    return t;
}

// A row product of a call: its columns, those of a tile, and its reduction.
struct RowSize {
    int64_t cols, k;
    bool gated, two;  // two: two operand pairs
    bool beside;      // in the gradients' launch, whose units fill its last wave: not cut
    // With a gated block's epilogue: not cut on pairs.  Its reduction is as long as the model is wide, and pairs gain from
    // a cut past 64 slices only; a second copy of the epilogue for joined parts slowed small calls (2000 rows of 8 experts,
    // 1408/2048, backward: 117.5 us with it, 115.3 without).
    bool block;
};

// Into how many parts each tile of gradients is cut along its run, where single CTAs have few tiles of long runs (by an
// expert's rows on average).  Cut / whole, us: linear backward 29994 rows of 2 experts, 440 x 200, 46 / 141; 9000 of 3,
// 256 x 256, 25 / 29; gated backward 29994 of 1, 200/440, 129 / 253; 9000 of 1, 512/512, 60 / 72.
int grad_ways(const Machine& mc, int64_t rows, int64_t experts, const Tiling& t, int64_t units) {
    if (t.bn == 256 || units * 2 > mc.dev.num_sms) return 1;
    return forge::expert_parts(forge::ExpertCut{0, slices(rows / experts), mc.dev.num_sms, 6, 5}, static_cast<int>(units));
}

int64_t grad_units(const Tiling& t, int64_t experts, const GradProduct* p, int n) {
    int64_t u = 0;
    for (int i = 0; i < n; ++i) u += experts * ceil_div(p[i].d_out, t.bn == 256 ? 256 : 128) * ceil_div(p[i].d_in, t.bn);
    return u;
}

// grads: the tiling and number of the gradients' tiles, if they have a launch of their own
struct GradSize {
    Tiling tiling;
    int64_t units;
};

Call make_call(const Machine& mc, int64_t rows, int64_t experts, const Tiling& tiling, int n_runs,
               std::initializer_list<RowSize> products, const GradSize& grads, Arena& a) {
    Call c{};
    c.mc = mc;
    c.rows = rows;
    c.experts = static_cast<int>(experts);
    c.tiling = tiling;
    const Tiling& t = c.tiling;
    c.tiles = rows / t.tile_rows + std::min(rows, experts);
    c.n_runs = n_runs;
    c.clean = a.take((experts + 1) * 4);
    c.n_tiles = a.take(4);
    c.list = a.take(c.tiles * 16);
    c.runs = a.take(n_runs * experts * static_cast<int64_t>(sizeof(CUtensorMap)));
    c.cuts = a.take(kMaxCuts * 16);
    const bool pair = t.bn == 256;
    const int width = pair ? mc.pairs : mc.dev.num_sms;
    bool cut = false;
    for (const RowSize& p : products) {
        const int kb = p.beside || (pair && p.block) ? 0 : slices(p.k) * (p.two ? 2 : 1);
        forge::ExpertCut& x = c.cut[c.n_cuts++];
        // joins as kTiles has them (block_api.cu).  Cut against whole on pairs, us: linear forward 1500 rows of 3 experts,
        // 14336 x 256, 34 / 70; gated backward 418 of 2, 232/14152, 101 / 237; calls that are not cut within 1 %
        x = forge::ExpertCut{static_cast<int>(ceil_div(p.cols, p.gated ? t.bn / 2 : t.bn)), kb, width, pair ? 8 : 6, pair ? 12 : 5};
        cut = cut || forge::expert_parts(x, 1) > 1;
    }
    c.n_counts = cut ? width * (pair ? 2 : 1) * 8 : 0;
    c.grad_ways = grads.units > 0 ? grad_ways(mc, rows, experts, grads.tiling, grads.units) : 1;
    c.grad_counts = c.n_counts;
    if (c.grad_ways > 1) c.n_counts += static_cast<int>(grads.units) * 8;
    c.counts = a.take(c.n_counts * 4ll);
    c.parts = a.take(cut ? static_cast<int64_t>(width) * t.tile_rows * t.bn * 4 : 0);
    c.grad_parts = a.take(c.grad_ways > 1 ? grads.units * c.grad_ways * (128 * 128 * 4) : 0);
    return c;
}

forge_status check_rows(int64_t rows, int64_t experts, int64_t d_in, int64_t d_out) {
    if (rows < 0 || rows > kMaxDim || experts < 1 || experts > kMaxExperts) return FORGE_ERR_INVALID_ARGUMENT;
    if (d_in < 8 || d_out < 8 || d_in > kMaxDim || d_out > kMaxDim || d_in % 8 != 0 || d_out % 8 != 0)
        return FORGE_ERR_INVALID_ARGUMENT;
    // tiles are counted in int
    if ((rows / 32 + experts) * (std::max(d_in, d_out) / 64 + 1) > kMaxDim ||
        3 * experts * (d_in / 128 + 1) * (d_out / 64 + 1) > kMaxDim || 3 * experts * (d_out / 128 + 1) * (d_in / 64 + 1) > kMaxDim)
        return FORGE_ERR_INVALID_ARGUMENT;
    return FORGE_OK;
}

// ---------------------------------------------------------------- operands

// Rows by expert: A [rows, cols], K-major.
forge_status rows_map(CUtensorMap* map, const Call& c, const void* base, int64_t cols) {
    const int extent = std::min(c.tiling.tile_rows, 128);  // of a CTA: on pairs half of the tile
    return kept_map(map, MapKey{base, cols, c.rows, cols, 0, extent}, [&] {
        const uint64_t k = static_cast<uint64_t>(cols), r = static_cast<uint64_t>(c.rows);
        return host::encode_map(map, base, {k, r, 1}, {2 * k, 2 * k}, {64, static_cast<uint32_t>(extent), 1});
    });
}

// The weights [experts, rows, cols], of which a CTA stages `extent` rows (K-major) or columns (MN-major) a slice.
forge_status weight_map(CUtensorMap* map, const void* base, int64_t experts, int64_t rows, int64_t cols, bool mn, int extent) {
    return kept_map(map, MapKey{base, cols, rows, cols, mn, extent, experts}, [&] {
        const uint64_t k = static_cast<uint64_t>(cols), r = static_cast<uint64_t>(rows), e = static_cast<uint64_t>(experts);
        if (mn && cols % 64 == 0)
            return host::encode_map(map, base, {64, r, k / 64, e}, {2 * k, 128, 2 * r * k},
                                    {64, 64, static_cast<uint32_t>(extent / 64), 1});
        return host::encode_map(map, base, {k, r, 1, e}, {2 * k, 2 * r * k, 2 * r * k},
                                {64, mn ? 64u : static_cast<uint32_t>(extent), 1, 1});
    });
}

// An operand of the weights' gradients, [rows, cols] and MN-major: its map, which the plan makes one of each run.  A
// slice of `extent` columns is one box of blocks of 64 columns, or (extent 64, and widths that are no multiple of 64) a
// box for each 64.
forge_status run_operand(RunOperand* o, const void* base, int64_t cols, int extent) {
    const bool blocks = extent > 64 && cols % 64 == 0;
    o->base = static_cast<const char*>(base);
    o->pitch = cols * 2;
    o->dim0 = blocks ? 64 : static_cast<uint32_t>(cols);
    o->dim2 = blocks ? static_cast<uint32_t>(cols / 64) : 1;
    return kept_map(&o->map, MapKey{base, cols, 1, cols, 2, extent}, [&] {
        const uint64_t pitch = static_cast<uint64_t>(cols) * 2;
        return host::encode_map(&o->map, base, {64, 1, 1}, {pitch, blocks ? 128 : pitch},
                                {64, 64, blocks ? static_cast<uint32_t>(extent / 64) : 1});
    });
}

// Gradient i, [experts, rows, cols].
template <int EPI>
forge_status set_gradient(ExpertGroup<EPI>& g, const Tiling& t, int i, void* base, int64_t experts, int64_t rows, int64_t cols) {
    g.to[i] = static_cast<uint16_t*>(base);
    if (t.bn != 256) return FORGE_OK;
    return kept_map(&g.outs[i], MapKey{base, cols, rows, cols, 4, 0, experts},
                    [&] { return host::encode_result_map(&g.outs[i], base, cols, rows, experts); });
}

// ---------------------------------------------------------------- launches

template <int EPI>
void begin_group(ExpertGroup<EPI>& g, const Call& c, int64_t kb_max) {
    std::memset(&g, 0, sizeof(g));
    g.n = 1;
    g.experts = c.experts;
    g.a_rows = forge::expert_grads(EPI) ? 128 : c.tiling.tile_rows;  // (row products beside gradients have tiles of 128 rows, or pairs)
    g.parts = reinterpret_cast<float*>(c.ws + c.parts);
    g.counts = reinterpret_cast<uint32_t*>(c.ws + c.counts);
    g.withhold_first_stage = host::take_withhold();
    g.n_tiles = reinterpret_cast<const int*>(c.ws + c.n_tiles);
    g.tiles = reinterpret_cast<const int4*>(c.ws + c.list);
    g.offsets = reinterpret_cast<const int*>(c.ws + c.clean);
    g.runs = reinterpret_cast<const CUtensorMap*>(c.ws + c.runs);
    g.status = c.mc.dev.status;
    g.wait_limit_ns = host::wait_limit_ns();
    g.acc_wait_limit_ns = host::acc_wait_limit_ns(kb_max);
}

template <int EPI>
forge_status launch(const ExpertGroup<EPI>& g, const Call& c, int bn, int64_t units) {
    const int width = bn == 256 ? c.mc.pairs : c.mc.dev.num_sms;
    host::count_launch();
    return cuda_status(forge::launch_expert<EPI>(&g, bn, static_cast<int>(std::min<int64_t>(width, units)), c.stream));
}

forge_status launch_plan(const Call& c, PlanArgs& a) {
    a.offsets = c.offsets;
    a.experts = c.experts;
    a.rows = static_cast<int>(c.rows);
    a.tile_rows = c.tiling.tile_rows;
    a.clean = reinterpret_cast<int*>(c.ws + c.clean);
    a.n_tiles = reinterpret_cast<int*>(c.ws + c.n_tiles);
    a.tiles = reinterpret_cast<int4*>(c.ws + c.list);
    a.runs = reinterpret_cast<CUtensorMap*>(c.ws + c.runs);
    a.cuts = reinterpret_cast<int4*>(c.ws + c.cuts);
    a.n_cuts = c.n_cuts;
    for (int i = 0; i < c.n_cuts; ++i) a.cut[i] = c.cut[i];
    a.counts = reinterpret_cast<uint32_t*>(c.ws + c.counts);
    a.n_counts = c.n_counts;
    const int64_t work = std::max({c.experts * std::max<int64_t>(a.n_runs, 1), std::min<int64_t>(c.tiles, 1024), int64_t{a.n_counts / 4}});
    const int64_t threads = std::min<int64_t>(1024, round_up(std::max<int64_t>(work, 64), 32));
    return cuda_status(host::launch_early(expert_plan_kernel, dim3(1), dim3(static_cast<unsigned>(threads)), 0, c.stream, a));
}

// cut: which of the call's row products this is
template <int EPI>
void set_rows(ExpertGroup<EPI>& g, const Call& c, int cut, int64_t cols, int64_t k0, int64_t k1) {
    g.cut = reinterpret_cast<const int4*>(c.ws + c.cuts) + cut;
    ExpertProblem& b = g.prob[0];
    b.cols = static_cast<int>(cols);
    b.ld = cols;
    b.tiles_n = static_cast<int>(ceil_div(cols, EPI == kBlockGatedFwd ? c.tiling.bn / 2 : c.tiling.bn));
    b.kb[0] = slices(k0);
    b.kb[1] = slices(k1);
    g.stream_b = c.tiling.tile_rows < 128;
}

// Of the weights, the rows or columns that a CTA stages a slice.
constexpr int kWeightExtent = 128, kGatedExtent = 64;

// out [rows, cols] = A0 W0 (+ A1 W1): W_e [cols, k] as it is read in y = x W^T, or [k, cols] (mn)
struct RowProduct {
    const void* a[2];
    const void* w[2];
    int64_t k, cols;
    bool mn;
    void* out;
};

// Units of a row product at most.
int64_t most_units(const Call& c, int cut) { return c.tiles * c.cut[cut].tiles_n + (c.n_counts > 0 ? c.cut[cut].width : 0); }

template <int EPI>
forge_status fill_rows(ExpertGroup<EPI>& g, const Call& c, int cut, const RowProduct& p) {
    set_rows(g, c, cut, p.cols, p.k, p.a[1] != nullptr ? p.k : 0);
    g.prob[0].b_mn = p.mn;
    g.prob[0].b_flat = p.mn && p.cols % 64 != 0;
    for (int i = 0; i < 2 && p.a[i] != nullptr; ++i) {
        FORGE_TRY(rows_map(&g.maps[2 + i], c, p.a[i], p.k));
        FORGE_TRY(weight_map(&g.maps[i], p.w[i], c.experts, p.mn ? p.k : p.cols, p.mn ? p.cols : p.k, p.mn,
                             kWeightExtent));
    }
    g.to[0] = static_cast<uint16_t*>(p.out);
    return FORGE_OK;
}

forge_status run_rows(const Call& c, int cut, const RowProduct& p) {
    ExpertGroup<kBlockStore> g;
    begin_group(g, c, 2 * slices(p.k));
    FORGE_TRY(fill_rows(g, c, cut, p));
    return launch(g, c, c.tiling.bn, most_units(c, cut));
}

// Neighbouring units of a pair or CTA.  A unit of another expert costs two fences on its maps: with short runs four units
// of one expert at a time (2048 rows of 64 experts, gated backward 2048/1408: 405 us, one at a time 432), where each still
// gets several such groups (1003 rows of 16 experts, 520/1032: 63.8 us so, 61.2 one at a time) and an expert has too few tiles to
// keep them on it anyway (16 rows of 8 experts, 4096/14336, 896 tiles each: 895 and 878).
int grad_chunk(const Call& c, int64_t units, int64_t each, int width) {
    return c.rows < 256ll * c.experts && units >= 16ll * width && each < 2ll * width ? 4 : 1;
}

// EPI: kExpertGrad, or kExpertBoth with dx, the call's first row product, in front of the gradients
template <int EPI>
forge_status run_grads(const Call& c, const Tiling& t, const GradProduct* p, int n, const RowProduct* dx) {
    ExpertGroup<EPI> g;
    begin_group(g, c, std::max(slices(c.rows), dx != nullptr ? 2 * slices(dx->k) : 0));
    constexpr int first = forge::expert_first_grad(EPI);
    g.n = first + n;
    if constexpr (EPI == kExpertBoth) FORGE_TRY(fill_rows(g, c, 0, *dx));
    int64_t u = 0;
    for (int i = 0; i < n; ++i) {
        ExpertProblem& b = g.prob[first + i];
        b.rows = static_cast<int>(p[i].d_out);
        b.cols = static_cast<int>(p[i].d_in);
        b.ld = p[i].d_in;
        b.tiles_m = static_cast<int>(ceil_div(p[i].d_out, t.bn == 256 ? 256 : 128));
        b.tiles_n = static_cast<int>(ceil_div(p[i].d_in, t.bn));
        b.unit_start = static_cast<int>(u);
        b.a_flat = p[i].d_out % 64 != 0;
        b.b_flat = p[i].d_in % 64 != 0;
        b.map_a = p[i].a;
        b.map_b = p[i].b;
        u += static_cast<int64_t>(c.experts) * b.tiles_m * b.tiles_n;
        FORGE_TRY(set_gradient(g, t, first + i, p[i].out, c.experts, p[i].d_out, p[i].d_in));
    }
    g.ways = EPI == kExpertGrad ? c.grad_ways : 1;
    if (g.ways > 1) {
        g.parts = reinterpret_cast<float*>(c.ws + c.grad_parts);
        g.counts = reinterpret_cast<uint32_t*>(c.ws + c.counts) + c.grad_counts;
    }
    u *= g.ways;
    g.n_units = static_cast<int>(u);
    g.chunk = g.ways > 1 ? 1 : grad_chunk(c, u, static_cast<int64_t>(g.prob[first].tiles_m) * g.prob[first].tiles_n, t.bn == 256 ? c.mc.pairs : c.mc.dev.num_sms);
    return launch(g, c, t.bn, u + (dx != nullptr ? c.tiles * g.prob[0].tiles_n : 0));
}

// ---------------------------------------------------------------- a linear layer for each expert

forge_status check_linear(const forge_expert_linear_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    return check_rows(s->rows, s->experts, s->d_in, s->d_out);
}

forge_status check_offsets(const int32_t* offsets) {
    if (offsets == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    return aligned(offsets, 4) ? FORGE_OK : FORGE_ERR_MISALIGNED;
}

forge_status check_gated(const forge_expert_gated_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->act != FORGE_ACT_SILU && s->act != FORGE_ACT_GELU_TANH && s->act != FORGE_ACT_RELU)
        return FORGE_ERR_INVALID_ARGUMENT;
    return check_rows(s->rows, s->experts, s->d_model, s->d_ff);
}

struct GatedSpace {
    Call c;
    int64_t dg, du, h, bytes;
};

GatedSpace layout_gated(const Machine& mc, const forge_expert_gated_shape& s, bool backward) {
    GatedSpace l{};
    Arena a;
    const Tiling rows = choose_rows(s.rows, s.experts);
    if (backward) {
        const GradProduct p[3] = {{0, 0, s.d_ff, s.d_model, nullptr}, {0, 0, s.d_ff, s.d_model, nullptr}, {0, 0, s.d_model, s.d_ff, nullptr}};
        const Tiling grads = grad_tiling(mc, s.experts, p, 3);
        l.c = make_call(mc, s.rows, s.experts, rows, kMaxRuns,
                        {{s.d_ff, s.d_model, false, false, false, true}, {s.d_model, s.d_ff, false, true, false, false}},
                        GradSize{grads, grad_units(grads, s.experts, p, 3)}, a);
    } else {
        l.c = make_call(mc, s.rows, s.experts, rows, 0,
                        {{s.d_ff, s.d_model, true, false, false, true}, {s.d_model, s.d_ff, false, false, false, false}},
                        GradSize{}, a);
    }
    const int64_t bytes = s.rows * s.d_ff * 2;
    if (backward) {
        l.dg = a.take(bytes);
        l.du = a.take(bytes);
    }
    l.h = a.take(bytes);
    l.bytes = a.used;
    return l;
}

int64_t linear_space(const Machine& mc, const forge_expert_linear_shape& s, bool backward, const Tiling& rows, bool together, Call* c) {
    Arena a;
    if (backward) {
        const GradProduct p{0, 0, s.d_out, s.d_in, nullptr};
        const Tiling grads = grad_tiling(mc, s.experts, &p, 1);
        *c = make_call(mc, s.rows, s.experts, rows, 2, {{s.d_in, s.d_out, false, false, together, false}},
                       GradSize{grads, together ? 0 : grad_units(grads, s.experts, &p, 1)}, a);
    } else {
        *c = make_call(mc, s.rows, s.experts, rows, 0, {{s.d_out, s.d_in, false, false, false, false}}, GradSize{}, a);
    }
    return a.used;
}

// The run operands of the gated backward pass; a and b: columns of the gradients' operands that a CTA stages
forge_status gated_runs(PlanArgs& plan, const GatedSpace& l, const forge_expert_gated_shape& s, const void* dY, const void* X, int a,
                        int b) {
    char* ws = l.c.ws;
    FORGE_TRY(run_operand(&plan.run[0], ws + l.dg, s.d_ff, a));
    FORGE_TRY(run_operand(&plan.run[1], ws + l.du, s.d_ff, a));
    FORGE_TRY(run_operand(&plan.run[2], dY, s.d_model, a));
    FORGE_TRY(run_operand(&plan.run[3], X, s.d_model, b));
    FORGE_TRY(run_operand(&plan.run[4], ws + l.h, s.d_ff, b));
    plan.n_runs = 5;
    return FORGE_OK;
}

// dH, and with it dG, dU and H in the workspace
forge_status run_gated_dh(const GatedSpace& l, const forge_expert_gated_shape& s, const void* dY, const void* G, const void* U,
                          const void* Wd) {
    const Call& c = l.c;
    ExpertGroup<kBlockGatedBwd> g;
    begin_group(g, c, slices(s.d_model));
    set_rows(g, c, 0, s.d_ff, s.d_model, 0);
    g.act = s.act;
    g.g_in = static_cast<const uint16_t*>(G);
    g.u_in = static_cast<const uint16_t*>(U);
    const int64_t outs[3] = {l.dg, l.du, l.h};
    for (int i = 0; i < 3; ++i) g.to[i] = reinterpret_cast<uint16_t*>(c.ws + outs[i]);
    g.prob[0].b_flat = s.d_ff % 64 != 0;
    FORGE_TRY(rows_map(&g.maps[2], c, dY, s.d_model));
    FORGE_TRY(weight_map(&g.maps[0], Wd, s.experts, s.d_model, s.d_ff, true, kWeightExtent));
    return launch(g, c, c.tiling.bn, most_units(c, 0));
}

RowProduct gated_dx(const GatedSpace& l, const forge_expert_gated_shape& s, const void* Wg, const void* Wu, void* dX) {
    return RowProduct{{l.c.ws + l.dg, l.c.ws + l.du}, {Wg, Wu}, s.d_ff, s.d_model, true, dX};
}

forge_status zero(std::initializer_list<void*> ps, int64_t bytes, cudaStream_t stream) {
    for (void* p : ps)
        if (p != nullptr && cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), stream) != cudaSuccess) return FORGE_ERR_CUDA;
    return FORGE_OK;
}

// The rows of all experts' weights are numbered as one matrix's.
forge_status check_stacked(int64_t experts, int64_t d_out) {
    return experts * d_out > kMaxDim ? FORGE_ERR_INVALID_ARGUMENT : FORGE_OK;
}

// The fused step of one layer; a and b: its run operands' numbers
forge_status run_step(const Call& c, int a, int b, const void* dY, const void* X, int64_t rows, int64_t experts, const forge_layer& w,
                      forge_opt_kind k, const forge_hparams* hp, int32_t state, int64_t step, cudaStream_t stream) {
    const CUtensorMap* runs = reinterpret_cast<const CUtensorMap*>(c.ws + c.runs);
    return host::expert_step(dY, X, reinterpret_cast<const int*>(c.ws + c.clean), runs + a * experts, runs + b * experts, rows,
                             experts, w.W, w.m, w.v, w.qscales, k, hp, w.d_out, w.d_in, state, step, w.seed, stream);
}

}  // namespace

extern "C" {

int64_t forge_expert_linear_workspace(const forge_expert_linear_shape* shape, int32_t backward) {
    if (check_linear(shape) != FORGE_OK) return -1;
    Machine mc;
    if (shape->rows == 0) return 0;
    if (machine(&mc) != FORGE_OK) return -1;
    Call c;
    const Tiling alone = choose_rows(shape->rows, shape->experts);
    const int64_t n = linear_space(mc, *shape, backward != 0, alone, false, &c);
    if (!backward) return n;
    const BackwardTiles t = linear_tiles(mc, *shape);
    return std::max(n, linear_space(mc, *shape, true, t.rows, t.together, &c));
}

forge_status forge_expert_linear(const void* X, const void* W, const int32_t* offsets, void* Y, void* workspace,
                                 int64_t workspace_bytes, const forge_expert_linear_shape* shape,
                                 struct CUstream_st* stream) {
    FORGE_TRY(check_linear(shape));
    const forge_expert_linear_shape& s = *shape;
    if (s.rows == 0) return FORGE_OK;
    FORGE_TRY(check_all({X, W, Y}));
    FORGE_TRY(check_offsets(offsets));
    Call c;
    Machine mc;
    FORGE_TRY(machine(&mc));
    FORGE_TRY(check_workspace(workspace, workspace_bytes, linear_space(mc, s, false, choose_rows(s.rows, s.experts), false, &c)));
    c.ws = static_cast<char*>(workspace);
    c.stream = stream;
    c.offsets = offsets;
    PlanArgs plan{};
    FORGE_TRY(launch_plan(c, plan));
    return run_rows(c, 0, RowProduct{{X, nullptr}, {W, nullptr}, s.d_in, s.d_out, false, Y});
}

forge_status forge_expert_linear_backward(const void* dY, const void* X, const void* W, const int32_t* offsets, void* dX,
                                          void* dW, void* workspace, int64_t workspace_bytes,
                                          const forge_expert_linear_shape* shape, struct CUstream_st* stream) {
    FORGE_TRY(check_linear(shape));
    const forge_expert_linear_shape& s = *shape;
    if (dX == nullptr && dW == nullptr && s.rows > 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (!aligned(dX, 32) || !aligned(dW, 32)) return FORGE_ERR_MISALIGNED;
    if (s.rows == 0) return zero({dW}, s.experts * s.d_out * s.d_in * 2, stream);
    FORGE_TRY(check_all({dY, X, W}));
    FORGE_TRY(check_offsets(offsets));
    Call c;
    Machine mc;
    FORGE_TRY(machine(&mc));
    const bool both = dX != nullptr && dW != nullptr;
    const GradProduct p{0, 1, s.d_out, s.d_in, dW};
    BackwardTiles t = linear_tiles(mc, s);
    if (!both) t = BackwardTiles{choose_rows(s.rows, s.experts), t.grads, false};
    FORGE_TRY(check_workspace(workspace, workspace_bytes, linear_space(mc, s, true, t.rows, t.together, &c)));
    c.ws = static_cast<char*>(workspace);
    c.stream = stream;
    c.offsets = offsets;
    PlanArgs plan{};
    FORGE_TRY(run_operand(&plan.run[0], dY, s.d_out, 128));
    FORGE_TRY(run_operand(&plan.run[1], X, s.d_in, 128));
    plan.n_runs = 2;
    FORGE_TRY(launch_plan(c, plan));
    const RowProduct dx{{dY, nullptr}, {W, nullptr}, s.d_out, s.d_in, true, dX};
    if (t.together) return run_grads<kExpertBoth>(c, t.grads, &p, 1, &dx);
    if (dX != nullptr) FORGE_TRY(run_rows(c, 0, dx));
    return dW != nullptr ? run_grads<kExpertGrad>(c, t.grads, &p, 1, nullptr) : FORGE_OK;
}

int64_t forge_expert_gated_mlp_workspace(const forge_expert_gated_shape* shape, int32_t backward) {
    if (check_gated(shape) != FORGE_OK) return -1;
    Machine mc;
    if (shape->rows == 0) return 0;
    if (machine(&mc) != FORGE_OK) return -1;
    return layout_gated(mc, *shape, backward != 0).bytes;
}

forge_status forge_expert_gated_mlp(const void* X, const void* Wg, const void* Wu, const void* Wd, const int32_t* offsets,
                                    void* Y, void* G, void* U, void* workspace, int64_t workspace_bytes,
                                    const forge_expert_gated_shape* shape, struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    const forge_expert_gated_shape& s = *shape;
    if (s.rows == 0) return FORGE_OK;
    FORGE_TRY(check_all({X, Wg, Wu, Wd, Y}));
    FORGE_TRY(check_offsets(offsets));
    if ((G == nullptr) != (U == nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    if (!aligned(G, 32) || !aligned(U, 32)) return FORGE_ERR_MISALIGNED;
    Machine mc;
    FORGE_TRY(machine(&mc));
    GatedSpace l = layout_gated(mc, s, false);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    Call& c = l.c;
    c.ws = static_cast<char*>(workspace);
    c.stream = stream;
    c.offsets = offsets;
    PlanArgs plan{};
    FORGE_TRY(launch_plan(c, plan));
    ExpertGroup<kBlockGatedFwd> g;
    begin_group(g, c, slices(s.d_model));
    set_rows(g, c, 0, s.d_ff, s.d_model, 0);
    g.act = s.act;
    g.keep = G != nullptr;
    if (g.keep) {
        g.to[0] = static_cast<uint16_t*>(G);
        g.to[1] = static_cast<uint16_t*>(U);
    }
    g.to[2] = reinterpret_cast<uint16_t*>(c.ws + l.h);
    FORGE_TRY(rows_map(&g.maps[2], c, X, s.d_model));
    const int extent = kGatedExtent;
    FORGE_TRY(weight_map(&g.maps[0], Wg, s.experts, s.d_ff, s.d_model, false, extent));
    FORGE_TRY(weight_map(&g.maps[1], Wu, s.experts, s.d_ff, s.d_model, false, extent));
    FORGE_TRY(launch(g, c, c.tiling.bn, most_units(c, 0)));
    return run_rows(c, 1, RowProduct{{c.ws + l.h, nullptr}, {Wd, nullptr}, s.d_ff, s.d_model, false, Y});
}

forge_status forge_expert_gated_mlp_backward(const void* dY, const void* X, const void* G, const void* U, const void* Wg,
                                             const void* Wu, const void* Wd, const int32_t* offsets, void* dX, void* dWg,
                                             void* dWu, void* dWd, void* workspace, int64_t workspace_bytes,
                                             const forge_expert_gated_shape* shape, struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    const forge_expert_gated_shape& s = *shape;
    FORGE_TRY(check_all({dWg, dWu, dWd}));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    if (s.rows == 0) return zero({dWg, dWu, dWd}, s.experts * s.d_ff * s.d_model * 2, stream);
    FORGE_TRY(check_all({dY, X, G, U, Wg, Wu, Wd}));
    FORGE_TRY(check_offsets(offsets));
    Machine mc;
    FORGE_TRY(machine(&mc));
    GatedSpace l = layout_gated(mc, s, true);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    Call& c = l.c;
    c.ws = static_cast<char*>(workspace);
    c.stream = stream;
    c.offsets = offsets;
    const GradProduct p[3] = {{0, 3, s.d_ff, s.d_model, dWg}, {1, 3, s.d_ff, s.d_model, dWu}, {2, 4, s.d_model, s.d_ff, dWd}};
    const Tiling t = grad_tiling(mc, s.experts, p, 3);
    PlanArgs plan{};
    FORGE_TRY(gated_runs(plan, l, s, dY, X, 128, 128));
    FORGE_TRY(launch_plan(c, plan));
    FORGE_TRY(run_gated_dh(l, s, dY, G, U, Wd));
    if (dX != nullptr) FORGE_TRY(run_rows(c, 1, gated_dx(l, s, Wg, Wu, dX)));
    return run_grads<kExpertGrad>(c, t, p, 3, nullptr);
}

forge_status forge_expert_linear_backward_step(const void* dY, const void* X, void* W, const int32_t* offsets, void* dX, void* m,
                                               void* v, float* qscales, void* workspace, int64_t workspace_bytes, int32_t state,
                                               forge_opt_kind opt_kind, const forge_hparams* hp,
                                               const forge_expert_linear_shape* shape, int64_t step, uint64_t seed,
                                               struct CUstream_st* stream) {
    FORGE_TRY(check_linear(shape));
    const forge_expert_linear_shape& s = *shape;
    FORGE_TRY(check_stacked(s.experts, s.d_out));
    FORGE_TRY(host::check_step(W, m, v, qscales, opt_kind, hp, s.d_out, s.d_in, state, step));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    Call c{};
    if (s.rows > 0) {
        FORGE_TRY(check_all({dY, X}));
        FORGE_TRY(check_offsets(offsets));
        Machine mc;
        FORGE_TRY(machine(&mc));
        FORGE_TRY(check_workspace(workspace, workspace_bytes, linear_space(mc, s, true, choose_rows(s.rows, s.experts), false, &c)));
        c.ws = static_cast<char*>(workspace);
        c.stream = stream;
        c.offsets = offsets;
        PlanArgs plan{};
        FORGE_TRY(run_operand(&plan.run[0], dY, s.d_out, 64));
        FORGE_TRY(run_operand(&plan.run[1], X, s.d_in, 64));
        plan.n_runs = 2;
        FORGE_TRY(launch_plan(c, plan));
        // dX reads the weights before the fused step replaces them: same stream, this order
        if (dX != nullptr) FORGE_TRY(run_rows(c, 0, RowProduct{{dY, nullptr}, {W, nullptr}, s.d_out, s.d_in, true, dX}));
    }
    return run_step(c, 0, 1, dY, X, s.rows, s.experts, forge_layer{nullptr, nullptr, W, m, v, qscales, 0, s.d_out, s.d_in, seed},
                    opt_kind, hp, state, step, stream);
}

forge_status forge_expert_gated_mlp_backward_step(const void* dY, const void* X, const void* G, const void* U,
                                                  const forge_layer* gate, const forge_layer* up, const forge_layer* down,
                                                  const int32_t* offsets, void* dX, void* workspace, int64_t workspace_bytes,
                                                  int32_t state, forge_opt_kind opt_kind, const forge_hparams* hp,
                                                  const forge_expert_gated_shape* shape, int64_t step, struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    const forge_expert_gated_shape& s = *shape;
    FORGE_TRY(check_stacked(s.experts, std::max(s.d_ff, s.d_model)));
    if (gate == nullptr || up == nullptr || down == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    for (const forge_layer* w : {gate, up})
        FORGE_TRY(host::check_step(w->W, w->m, w->v, w->qscales, opt_kind, hp, s.d_ff, s.d_model, state, step));
    FORGE_TRY(host::check_step(down->W, down->m, down->v, down->qscales, opt_kind, hp, s.d_model, s.d_ff, state, step));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    forge_layer layers[3] = {*gate, *up, *down};
    for (int i = 0; i < 3; ++i) {
        layers[i].d_out = i < 2 ? s.d_ff : s.d_model;
        layers[i].d_in = i < 2 ? s.d_model : s.d_ff;
    }
    GatedSpace l{};
    Call& c = l.c;
    if (s.rows > 0) {
        FORGE_TRY(check_all({dY, X, G, U}));
        FORGE_TRY(check_offsets(offsets));
        Machine mc;
        FORGE_TRY(machine(&mc));
        l = layout_gated(mc, s, true);
        FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
        c.ws = static_cast<char*>(workspace);
        c.stream = stream;
        c.offsets = offsets;
        PlanArgs plan{};
        FORGE_TRY(gated_runs(plan, l, s, dY, X, 64, 64));
        FORGE_TRY(launch_plan(c, plan));
        // the input gradients read the weights before the fused step replaces them: same stream, this order
        FORGE_TRY(run_gated_dh(l, s, dY, G, U, down->W));
        if (dX != nullptr) FORGE_TRY(run_rows(c, 1, gated_dx(l, s, gate->W, up->W, dX)));
    }
    FORGE_TRY(run_step(c, 0, 3, c.ws + l.dg, X, s.rows, s.experts, layers[0], opt_kind, hp, state, step, stream));
    FORGE_TRY(run_step(c, 1, 3, c.ws + l.du, X, s.rows, s.experts, layers[1], opt_kind, hp, state, step, stream));
    return run_step(c, 2, 4, dY, c.ws + l.h, s.rows, s.experts, layers[2], opt_kind, hp, state, step, stream);
}

}  // extern "C"
