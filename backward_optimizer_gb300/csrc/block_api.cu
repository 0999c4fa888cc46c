// block_api.cu -- the C ABI of the operators around the fused layers that are made of matrix products
// (include/forge.h): the gated feed-forward block and the cross entropy of a linear head.  Argument
// checks, the cutting of the products into units, workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "block_host.h"
#include "block_kernel.cuh"
#include "block_launch.h"
#include "forge.h"
#include "host.h"
#include "rows_kernel.cuh"

namespace {

using forge::BlockGroup;
using forge::BlockProblem;
using forge::PairGroup;
using forge::kMaxProducts;
namespace host = forge::host;
using namespace forge::host;

// ---------------------------------------------------------------- cutting products into units

// One product as the plan sees it: the output's rows and columns, columns per 256-wide tile (128 for
// the gated forward, whose tile holds gate and up), and its reduction slices.
struct Cut {
    int64_t rows, cols;
    int kb;
    int parts;        // units per split tile
    int split_from;   // tiles before this one are whole
    int tiles_m, tiles_n;
    int64_t part_base;
    int count_base;
    int units() const { return split_from + (tiles_m * tiles_n - split_from) * parts; }
};

struct Plan {
    int bn;      // tile columns: 256 on CTA pairs, 128 or 64 on single CTAs
    int width;   // pairs or CTAs
    int a_rows;  // rows of A per stage (BlockGroup::a_rows)
    int n;
    Cut cut[kMaxProducts];
    int64_t part_floats;
    int counts;
};

// A unit shorter than this many slices costs more in its fill, its partial sums and their join than
// it saves.
constexpr int kMinSlices = 8;
constexpr int kMaxParts = 16;
// the epilogue of a tile, in slices of the mainloop: only to weigh units against one another
constexpr int kEpiSlices = 8;

// Tile shapes and what they cost, in slices (some 0.27 us whatever the tile: the copies set the pace):
// `epi`: a tile's epilogue and change of accumulator, which run beside the next tile's slices and are its
// least time; `last`: the last tile's epilogue, beyond the narrowest tile's; a split tile's join: `join` and
// `per_part` for each part.  Wide tiles need fewer slices for the same product, narrow ones fill the GPU with
// less and end sooner.  The numbers are a fit to 1200 timings of products from 5 to 5366 rows, each with
// every shape and several cuts; the plan below then comes within 1 % of the best shape and cut on average.
// 256 tokens, 4096/14336, down product: 89 us on 256, 99 on 128, 123 on 64 columns.  256 tokens,
// 1024/2816, dX and the weight gradients: 41.5 / 35.1 / 41.  256 tokens, 256/512: 24.5 / 20 / 18.
struct TileCost {
    int bn, epi, last, join, per_part;
};
constexpr TileCost kTiles[] = {{256, 8, 13, 8, 12}, {128, 8, 3, 6, 5}, {64, 6, 1, 10, 2}};

int64_t tiles_of(const Cut& c, int bn, bool gated) {
    return ceil_div(c.rows, bn == 256 ? 256 : 128) * ceil_div(c.cols, bn / (gated ? 2 : 1));
}

struct Choice {
    double t;
    int bn, parts, length;
    void offer(double time, int width, int n_parts, int part_length) {
        // equal times: the wider tile and fewer parts, which come first, read less
        if (bn == 0 || time < 0.98 * t) *this = Choice{time, width, n_parts, part_length};
    }
};

// One product: its full waves, then the last one's tiles, whole or cut into parts that fill the GPU.
Choice choose_one(const Cut& c, const Machine& mc, bool gated) {
    Choice best{};
    for (const TileCost& k : kTiles) {
        const int64_t width = k.bn == 256 ? mc.pairs : mc.dev.num_sms;
        const int64_t tiles = tiles_of(c, k.bn, gated), full = tiles / width, rest = tiles % width;
        const int64_t wave = std::max(c.kb, k.epi);
        best.offer(static_cast<double>((ceil_div(tiles, width) - 1) * wave + c.kb + k.last), k.bn, 1, c.kb);
        for (int parts = 2; rest > 0 && parts <= kMaxParts && c.kb >= kMinSlices * parts && rest * parts <= width; ++parts)
            best.offer(static_cast<double>(full * wave + ceil_div(c.kb, parts) + k.last + k.join + k.per_part * parts),
                       k.bn, parts, c.kb);
    }
    return best;
}

int parts_of(const Cut& c, int length) {
    return std::max(1, std::min({static_cast<int>(ceil_div(c.kb, length)), kMaxParts, c.kb / kMinSlices}));
}

// Several products: the call lasts as long as its longest unit, or as an even share of all work.  For each
// tile shape, units are cut to the length at which the larger of the two is smallest; a unit's time: its slices,
// or its epilogue where that is longer; a part's sums cost it a little more.
Choice choose_many(const Cut* cut, int n, const Machine& mc) {
    Choice best{};
    int kb_max = 0;
    for (int i = 0; i < n; ++i) kb_max = std::max(kb_max, cut[i].kb);
    for (const TileCost& k : kTiles) {
        const int width = k.bn == 256 ? mc.pairs : mc.dev.num_sms;
        double least = 0, time = 0;
        int cut_to = kb_max;
        for (int cuts : {1, 2, 3, 4, 6, 8, 12, 16}) {
            const int length = static_cast<int>(ceil_div(kb_max, cuts));
            double longest = 0, work = 0;
            int most = 1;
            for (int i = 0; i < n; ++i) {
                const int parts = parts_of(cut[i], length);
                const double unit = std::max<double>(static_cast<double>(cut[i].kb) / parts, kEpiSlices) + (parts > 1 ? 3 : 1);
                longest = std::max(longest, unit);
                work += unit * parts * tiles_of(cut[i], k.bn, false);
                most = std::max(most, parts);
            }
            const double t = std::max(longest, work / width);
            if (cuts == 1 || t < 0.97 * least) {
                // joins run beside other units' slices, but not all the way
                const double join = most > 1 ? k.join + k.per_part * most : 0;
                least = t;
                time = std::max(longest + join / 2, work / width) + k.last;
                cut_to = length;
            }
        }
        best.offer(time, k.bn, 0, cut_to);
    }
    return best;
}

// Choices of recent sizes, per host thread: working one out takes as much host time as a small kernel, and
// the sizes alone determine it.
struct ChoiceSlot {
    int64_t key[3 * kMaxProducts + 3];
    Choice choice;
    bool used;
};
constexpr int kChoiceSlots = 64;
thread_local ChoiceSlot t_choices[kChoiceSlots];

Choice choose(const Plan& p, const Machine& mc, bool gated) {
    int64_t key[3 * kMaxProducts + 3] = {p.n * 2 + gated, mc.pairs, mc.dev.num_sms};
    uint64_t h = static_cast<uint64_t>(key[0]);
    for (int i = 0; i < p.n; ++i) {
        const int64_t size[3] = {p.cut[i].rows, p.cut[i].cols, p.cut[i].kb};
        for (int j = 0; j < 3; ++j) {
            key[3 + 3 * i + j] = size[j];
            h = (h ^ static_cast<uint64_t>(size[j])) * 0x9E3779B97F4A7C15ull;
        }
    }
    ChoiceSlot& slot = t_choices[(h >> 32) % kChoiceSlots];
    if (!slot.used || std::memcmp(slot.key, key, sizeof key) != 0) {
        slot.choice = p.n == 1 ? choose_one(p.cut[0], mc, gated) : choose_many(p.cut, p.n, mc);
        std::memcpy(slot.key, key, sizeof key);
        slot.used = true;
    }
    return slot.choice;
}

void plan_products(Plan& p, const Machine& mc, bool gated, bool a_k_major) {
    const Choice choice = choose(p, mc, gated);
    p.bn = choice.bn;
    const bool pair = p.bn == 256;
    p.width = pair ? mc.pairs : mc.dev.num_sms;
    p.a_rows = 128;
    if (p.n == 1 && !pair && a_k_major && p.cut[0].rows <= 64) p.a_rows = static_cast<int>(round_up(p.cut[0].rows, 8));
    const int64_t tm = pair ? 256 : 128, tn = p.bn / (gated ? 2 : 1);
    for (int i = 0; i < p.n; ++i) {
        Cut& c = p.cut[i];
        c.tiles_m = static_cast<int>(ceil_div(c.rows, tm));
        c.tiles_n = static_cast<int>(ceil_div(c.cols, tn));
        c.parts = p.n == 1 ? choice.parts : parts_of(c, choice.length);
        const int tiles = c.tiles_m * c.tiles_n;
        c.split_from = c.parts == 1 ? tiles : p.n == 1 ? tiles - tiles % p.width : 0;
    }
    p.part_floats = 0;
    p.counts = 0;
    const int cg = pair ? 2 : 1;
    for (int i = 0; i < p.n; ++i) {
        Cut& c = p.cut[i];
        const int split = c.parts > 1 ? c.tiles_m * c.tiles_n - c.split_from : 0;
        c.part_base = p.part_floats;
        c.count_base = p.counts;
        p.part_floats += static_cast<int64_t>(split) * c.parts * tm * p.bn;
        p.counts += split * cg * 8;
    }
}

Plan plan_one(const Machine& mc, int64_t rows, int64_t cols, int kb, bool gated = false) {
    Plan p{};
    p.n = 1;
    p.cut[0].rows = rows;
    p.cut[0].cols = cols;
    p.cut[0].kb = kb;
    plan_products(p, mc, gated, true);
    return p;
}

int slices(int64_t k) { return static_cast<int>(ceil_div(k, forge::kBK)); }

// The split tiles' regions that the launches of a call share, each big enough for any of them: FP32
// parts, and arrival counters, which are zero between launches once the call has cleared them.
struct SplitSpace {
    int64_t parts, counts;
    int n_counts;
};

SplitSpace take_split(Arena& a, std::initializer_list<const Plan*> plans) {
    int64_t floats = 0;
    int counts = 0;
    for (const Plan* p : plans) {
        floats = std::max(floats, p->part_floats);
        counts = std::max(counts, p->counts);
    }
    return SplitSpace{a.take(floats * 4), a.take(counts * 4ll), counts};
}

// The schedule and everything of a launch that does not depend on the epilogue.  The products come
// longest first.
template <int NP>
forge_status fill_group(BlockGroup<NP>& g, const Plan& p, const Machine& mc, char* ws, const SplitSpace& sp) {
    g.n = p.n;
    g.a_rows = p.a_rows;
    int u = 0, kb_max = 0;
    int longest = 0;
    for (int i = 0; i < p.n; ++i) {
        BlockProblem& b = g.prob[i];
        const Cut& c = p.cut[i];
        b.rows = static_cast<int>(c.rows);
        b.cols = static_cast<int>(c.cols);
        const int group = c.tiles_m < 8 ? c.tiles_m : 8;
        b.order = forge::TileOrder{c.tiles_m, c.tiles_n, group, 0};
        b.unit_start = u;
        b.split_from = c.split_from;
        b.parts = c.parts;
        b.part_base = c.part_base;
        b.count_base = c.count_base;
        u += c.units();
        kb_max = std::max(kb_max, c.kb);
        longest = std::max(longest, c.split_from > 0 ? c.kb : c.kb / c.parts);
    }
    // units at the front that take at least three quarters of the longest one's time are the long ones
    int n_long = 0, short_kb = 0;
    bool front = true;
    for (int i = 0; i < p.n; ++i) {
        const Cut& c = p.cut[i];
        const int whole = c.split_from, rest = c.units() - c.split_from;
        const int kb_part = c.kb / c.parts;
        if (whole > 0) {
            if (front && 4 * c.kb >= 3 * longest) n_long += whole;
            else { front = false; short_kb = std::max(short_kb, c.kb); }
        }
        if (rest > 0) {
            if (front && 4 * kb_part >= 3 * longest) n_long += rest;
            else { front = false; short_kb = std::max(short_kb, kb_part); }
        }
    }
    g.units = forge::plan_units(u, n_long, std::min(p.width, u), longest + kEpiSlices, short_kb + kEpiSlices);
    g.parts = reinterpret_cast<float*>(ws + sp.parts);
    g.counts = reinterpret_cast<uint32_t*>(ws + sp.counts);
    g.status = mc.dev.status;
    g.wait_limit_ns = host::wait_limit_ns();
    g.acc_wait_limit_ns = host::acc_wait_limit_ns(kb_max);
    g.withhold_first_stage = host::take_withhold();
    return FORGE_OK;
}

// The map of an operand of which a CTA stages `extent` rows (K-major) or columns (MN-major) per slice, one
// box a slice; or two boxes of 64 columns where the operand's width is no multiple of 64 (flat).
forge_status operand_map(CUtensorMap* map, const Operand& o, bool mn, int extent) {
    const MapKey key{o.base, o.cols, o.rows, o.ld, mn, extent};
    return kept_map(map, key, [&] {
        const uint64_t cols = static_cast<uint64_t>(o.cols), rows = static_cast<uint64_t>(o.rows);
        const uint64_t pitch = static_cast<uint64_t>(o.ld) * 2;
        if (mn && o.cols % 64 == 0)
            return host::encode_map(map, o.base, {64, rows, cols / 64}, {pitch, 128}, {64, 64, static_cast<uint32_t>(extent / 64)});
        return host::encode_map(map, o.base, {cols, rows, 1}, {pitch, pitch}, {64, mn ? 64u : static_cast<uint32_t>(extent), 1});
    });
}

// Map i of product l of a group (BlockGroup::maps).
template <int NP>
forge_status set_map(BlockGroup<NP>& g, const Plan& p, int l, int i, const Operand& o, bool mn, bool gated = false) {
    const int extent = i % 2 == 0 ? p.a_rows : p.bn == 256 ? 128 : gated ? p.bn / 2 : p.bn;
    int& flat = i % 2 == 0 ? g.prob[l].a_flat : g.prob[l].b_flat;
    flat = flat || (mn && o.cols % 64 != 0);
    return operand_map(&g.maps[4 * l + i], o, mn, extent);
}

// Result i of a group, [rows, cols] in one piece (PairGroup::outs; an operand's extent is never 0).
template <int EPI>
forge_status set_result(PairGroup<EPI>& g, const Plan& p, int i, void* base, int64_t cols, int64_t rows) {
    g.to[i] = static_cast<uint16_t*>(base);
    if (!forge::staged(EPI) || p.bn != 256) return FORGE_OK;
    return kept_map(&g.outs[i], MapKey{base, cols, rows, cols, 0, 0},
                    [&] { return host::encode_result_map(&g.outs[i], base, cols, rows); });
}

template <int EPI>
forge_status launch(const PairGroup<EPI>& g, const Plan& p, cudaStream_t stream) {
    host::count_launch();
    return cuda_status(forge::launch_block<EPI>(&g, p.bn, std::min(p.width, g.units.n_units), stream));
}

// One product of a kBlockStore launch.
struct Product {
    int64_t rows, cols;
    Operand a[2], b[2];
    int64_t k[2];
    int a_mn, b_mn;
    uint16_t* out;
    const uint16_t* add;
    float* sum;
    int sum_in, sum_out;
    const float* unit;
};

Plan plan_store(const Machine& mc, Product* pr, int n) {
    std::stable_sort(pr, pr + n, [](const Product& x, const Product& y) {
        return slices(x.k[0]) + slices(x.k[1]) > slices(y.k[0]) + slices(y.k[1]);
    });
    Plan p{};
    p.n = n;
    for (int i = 0; i < n; ++i) {
        p.cut[i].rows = pr[i].rows;
        p.cut[i].cols = pr[i].cols;
        p.cut[i].kb = slices(pr[i].k[0]) + slices(pr[i].k[1]);
    }
    plan_products(p, mc, false, pr[0].a_mn == 0);
    return p;
}

// pr: in the order that plan_store left them in
forge_status run_store(const Machine& mc, const Plan& p, const Product* pr, char* ws, const SplitSpace& sp,
                       cudaStream_t stream) {
    PairGroup<forge::kBlockStore> g;
    std::memset(&g, 0, sizeof(g));
    FORGE_TRY(fill_group(g, p, mc, ws, sp));
    for (int i = 0; i < p.n; ++i) {
        BlockProblem& b = g.prob[i];
        for (int s = 0; s < 2; ++s) {
            b.kb[s] = slices(pr[i].k[s]);
            if (b.kb[s] == 0) continue;
            FORGE_TRY(set_map(g, p, i, 2 * s, pr[i].a[s], pr[i].a_mn != 0));
            FORGE_TRY(set_map(g, p, i, 2 * s + 1, pr[i].b[s], pr[i].b_mn != 0));
        }
        b.a_mn = pr[i].a_mn;
        b.b_mn = pr[i].b_mn;
        if (!pr[i].sum_out) FORGE_TRY(set_result(g, p, i, pr[i].out, pr[i].cols, pr[i].rows));
        b.add = pr[i].add;
        b.sum = pr[i].sum;
        b.sum_in = pr[i].sum_in;
        b.sum_out = pr[i].sum_out;
        b.unit = pr[i].unit;
        b.ld = pr[i].cols;
    }
    return launch<forge::kBlockStore>(g, p, stream);
}

__global__ void __launch_bounds__(256) zero_counts_kernel(uint32_t* counts, int n) {
    forge::stream_wait();
    for (int i = threadIdx.x; i < n; i += 256) counts[i] = 0u;
}

// Clears the call's counters: the first launch does it for those behind it unless it needs them itself.
template <int NP>
forge_status clear_counts(BlockGroup<NP>& first, const Plan& p, char* ws, const SplitSpace& sp, cudaStream_t stream) {
    if (sp.n_counts == 0) return FORGE_OK;
    uint32_t* at = reinterpret_cast<uint32_t*>(ws + sp.counts);
    if (p.counts == 0) {
        first.zero_at = at;
        first.zero_n = sp.n_counts;
        return FORGE_OK;
    }
    return cuda_status(host::launch_early(zero_counts_kernel, dim3(1), dim3(256), 0, stream, at, sp.n_counts));
}

// y [rows, n] = a [rows, k] w [n, k]^T (+ add)
Product product_nt(const void* a, const void* w, int64_t rows, int64_t n, int64_t k, void* y, const void* add) {
    Product p{};
    p.rows = rows;
    p.cols = n;
    p.a[0] = Operand{a, k, rows, k};
    p.b[0] = Operand{w, k, n, k};
    p.k[0] = k;
    p.out = static_cast<uint16_t*>(y);
    p.add = static_cast<const uint16_t*>(add);
    return p;
}

// dX [T, d_in] = dY [T, d_out] W [d_out, d_in]; dY's rows ld apart
Product product_dx(const void* dY, int64_t ld, const void* W, int64_t T, int64_t d_out, int64_t d_in, void* dX) {
    Product p{};
    p.rows = T;
    p.cols = d_in;
    p.a[0] = Operand{dY, d_out, T, ld};
    p.b[0] = Operand{W, d_in, d_out, d_in};
    p.k[0] = d_out;
    p.b_mn = 1;
    p.out = static_cast<uint16_t*>(dX);
    return p;
}

// dW [d_out, d_in] = dY [T, d_out]^T X [T, d_in]; dY's rows ld apart
Product product_dw(const void* dY, int64_t ld, const void* X, int64_t T, int64_t d_out, int64_t d_in, void* dW) {
    Product p{};
    p.rows = d_out;
    p.cols = d_in;
    p.a[0] = Operand{dY, d_out, T, ld};
    p.b[0] = Operand{X, d_in, T, d_in};
    p.k[0] = T;
    p.a_mn = p.b_mn = 1;
    p.out = static_cast<uint16_t*>(dW);
    return p;
}

// ---------------------------------------------------------------- gated feed-forward block

forge_status check_gated(const forge_gated_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->T < 0 || s->T > kMaxDim || s->d_model < 8 || s->d_ff < 8 || s->d_model > kMaxDim || s->d_ff > kMaxDim)
        return FORGE_ERR_INVALID_ARGUMENT;
    if (s->d_model % 8 != 0 || s->d_ff % 8 != 0) return FORGE_ERR_INVALID_ARGUMENT;
    // tiles are counted in int
    if ((s->T / 128 + 1) * (std::max(s->d_model, s->d_ff) / 64 + 1) > kMaxDim ||
        (s->d_ff / 128 + 1) * (s->d_model / 128 + 1) > kMaxDim)
        return FORGE_ERR_INVALID_ARGUMENT;
    if (s->act != FORGE_ACT_SILU && s->act != FORGE_ACT_GELU_TANH && s->act != FORGE_ACT_RELU)
        return FORGE_ERR_INVALID_ARGUMENT;
    return FORGE_OK;
}

struct GatedForward {
    bool few;  // one to four tokens: rows_kernel.cuh
    Plan up, down;
    Product y;
    int64_t h, bytes;
    SplitSpace split;
};

GatedForward layout_gated_forward(const Machine& mc, const forge_gated_shape& s) {
    GatedForward l{};
    Arena a;
    l.few = forge::rows_fit(s.T, s.d_model, true) && forge::rows_fit(s.T, s.d_ff, false);
    if (l.few) {
        l.h = a.take(s.T * s.d_ff * 2);
        l.bytes = a.used;
        return l;
    }
    l.up = plan_one(mc, s.T, s.d_ff, slices(s.d_model), true);
    l.y = product_nt(nullptr, nullptr, s.T, s.d_model, s.d_ff, nullptr, nullptr);
    l.down = plan_store(mc, &l.y, 1);
    l.split = take_split(a, {&l.up, &l.down});
    l.h = a.take(s.T * s.d_ff * 2);
    l.bytes = a.used;
    return l;
}

struct GatedBackward {
    Plan dh, grads;
    Product pr[4];
    int n;
    int64_t dg, du, h, bytes;
    SplitSpace split;
};

// dw: the weights' gradients are wanted (else the fused step makes them its own way)
GatedBackward layout_gated_backward(const Machine& mc, const forge_gated_shape& s, const void* dY, const void* X,
                                    const void* Wg, const void* Wu, void* dX, void* dWg, void* dWu, void* dWd, bool dw,
                                    bool dx, char* ws) {
    GatedBackward l;
    Arena a;
    l.dg = a.take(s.T * s.d_ff * 2);
    l.du = a.take(s.T * s.d_ff * 2);
    l.h = a.take(s.T * s.d_ff * 2);
    l.dh = plan_one(mc, s.T, s.d_ff, slices(s.d_model));
    l.n = 0;
    if (dx) {
        Product p = product_dx(ws + l.dg, s.d_ff, Wg, s.T, s.d_ff, s.d_model, dX);
        p.a[1] = Operand{ws + l.du, s.d_ff, s.T, s.d_ff};
        p.b[1] = Operand{Wu, s.d_model, s.d_ff, s.d_model};
        p.k[1] = s.d_ff;
        l.pr[l.n++] = p;
    }
    if (dw) {
        l.pr[l.n++] = product_dw(ws + l.dg, s.d_ff, X, s.T, s.d_ff, s.d_model, dWg);
        l.pr[l.n++] = product_dw(ws + l.du, s.d_ff, X, s.T, s.d_ff, s.d_model, dWu);
        l.pr[l.n++] = product_dw(dY, s.d_model, ws + l.h, s.T, s.d_model, s.d_ff, dWd);
    }
    l.grads = Plan{};
    if (l.n > 0) l.grads = plan_store(mc, l.pr, l.n);
    l.split = take_split(a, {&l.dh, &l.grads});
    l.bytes = a.used;
    return l;
}

forge_status run_gated_dh(const Machine& mc, const GatedBackward& l, const void* dY, const void* Wd, const void* G,
                          const void* U, char* ws, const forge_gated_shape& s, cudaStream_t stream) {
    PairGroup<forge::kBlockGatedBwd> g;
    std::memset(&g, 0, sizeof(g));
    FORGE_TRY(fill_group(g, l.dh, mc, ws, l.split));
    FORGE_TRY(clear_counts(g, l.dh, ws, l.split, stream));
    BlockProblem& b = g.prob[0];
    b.kb[0] = slices(s.d_model);
    b.ld = s.d_ff;
    b.g_in = static_cast<const uint16_t*>(G);
    b.u_in = static_cast<const uint16_t*>(U);
    const int64_t outs[3] = {l.dg, l.du, l.h};
    for (int i = 0; i < 3; ++i) FORGE_TRY(set_result(g, l.dh, i, ws + outs[i], s.d_ff, s.T));
    b.act = s.act;
    FORGE_TRY(set_map(g, l.dh, 0, 0, Operand{dY, s.d_model, s.T, s.d_model}, false));
    FORGE_TRY(set_map(g, l.dh, 0, 1, Operand{Wd, s.d_ff, s.d_model, s.d_ff}, true));
    return launch<forge::kBlockGatedBwd>(g, l.dh, stream);
}

// ---------------------------------------------------------------- cross entropy of a linear head

forge_status check_loss(const forge_loss_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->T < 0 || s->T > kMaxDim || s->vocab < 1 || s->vocab > kMaxDim || s->d_model < 8 || s->d_model > kMaxDim ||
        s->d_model % 8 != 0)
        return FORGE_ERR_INVALID_ARGUMENT;
    if ((s->T / 128 + 1) * (std::max(s->vocab, s->d_model) / 128 + 1) > kMaxDim ||
        (s->vocab / 128 + 1) * (s->d_model / 128 + 1) > kMaxDim)
        return FORGE_ERR_INVALID_ARGUMENT;
    return FORGE_OK;
}

struct LossForward {
    Plan plan;
    int64_t stats, bytes;
    int stat_parts;
    SplitSpace split;
};

LossForward layout_loss_forward(const Machine& mc, const forge_loss_shape& s) {
    LossForward l;
    Arena a;
    l.plan = plan_one(mc, s.T, s.vocab, slices(s.d_model));
    l.split = take_split(a, {&l.plan});
    l.stat_parts = 2 * l.plan.cut[0].tiles_n;
    l.stats = a.take(static_cast<int64_t>(l.stat_parts) * s.T * 8);
    l.bytes = a.used;
    return l;
}

// Vocabulary entries per piece of the backward pass: g of one piece is [T, piece] bfloat16, at most
// 256 MiB unless T alone asks for more than 2048 entries' worth.
int64_t loss_piece(const forge_loss_shape& s) {
    const int64_t fit = (256ll << 20) / (2 * std::max<int64_t>(s.T, 1)) / 256 * 256;
    return std::min(round_up(s.vocab, 64), std::max<int64_t>(fit, 2048));
}

struct LossBackward {
    int64_t piece, pieces;
    int64_t g, sum, unit, bytes;
    SplitSpace split;
};

struct LossPiece {
    int64_t v0, n, ld;
    Plan grad, out;
    Product pr[2];
    int np;
};

LossPiece loss_piece_of(const Machine& mc, const forge_loss_shape& s, const LossBackward& l, int64_t i, const void* X,
                        const void* W, void* dX, void* dW, bool dx, bool dw, char* ws) {
    LossPiece p{};
    p.v0 = i * l.piece;
    p.n = std::min(l.piece, s.vocab - p.v0);
    p.ld = round_up(p.n, 64);  // whole blocks of 64 columns for the copies of dW's operand
    p.grad = plan_one(mc, s.T, p.n, slices(s.d_model));
    const size_t row = static_cast<size_t>(p.v0) * s.d_model * 2;
    if (dx) {
        Product x = product_dx(ws + l.g, p.ld, static_cast<const char*>(W) + row, s.T, p.n, s.d_model, dX);
        x.sum = reinterpret_cast<float*>(ws + l.sum);
        x.sum_in = i > 0;
        x.sum_out = i + 1 < l.pieces;
        p.pr[p.np++] = x;
    }
    if (dw) {
        Product w = product_dw(ws + l.g, p.ld, X, s.T, p.n, s.d_model, static_cast<char*>(dW) + row);
        w.a[0].cols = p.ld;  // g's padding (exp(-lse), which may be infinite) ends in rows of dW that are not stored
        p.pr[p.np++] = w;
    }
    for (int j = 0; j < p.np; ++j) p.pr[j].unit = reinterpret_cast<const float*>(ws + l.unit);
    if (p.np > 0) p.out = plan_store(mc, p.pr, p.np);
    return p;
}

LossBackward layout_loss_backward(const Machine& mc, const forge_loss_shape& s, bool dx, bool dw) {
    LossBackward l{};
    Arena a;
    l.unit = a.take(4);
    l.piece = loss_piece(s);
    l.pieces = ceil_div(s.vocab, l.piece);
    l.g = a.take(s.T * l.piece * 2);
    l.sum = a.take(dx && l.pieces > 1 ? s.T * s.d_model * 4 : 0);
    // pieces are alike but for the last one
    const LossPiece p = loss_piece_of(mc, s, l, 0, nullptr, nullptr, nullptr, nullptr, dx, dw, nullptr);
    const LossPiece q = loss_piece_of(mc, s, l, l.pieces - 1, nullptr, nullptr, nullptr, nullptr, dx, dw, nullptr);
    l.split = take_split(a, {&p.grad, &p.out, &q.grad, &q.out});
    l.bytes = a.used;
    return l;
}

// Whether a launch of its own finds the largest dloss and clears the counters (loss_begin_kernel), or the first
// piece's gradient does: it can where it is not cut itself, and where a warp's look at every dloss ends before
// the first tile does.  In turn on one GPU: 130 tokens over 4099 x 512 24.6 us with the launch, 22.6 without; 1024 over
// 4096 x 256 27.9 and 26.3; 2048 38.8 and 39.7.
constexpr int64_t kOwnUnitRows = 1024;

bool loss_begins(const LossPiece& p, const forge_loss_shape& s) { return p.grad.counts > 0 || s.T > kOwnUnitRows; }

// g of one piece of the vocabulary
forge_status run_loss_grad(const Machine& mc, const LossBackward& l, const LossPiece& p, const forge_loss_shape& s,
                           const void* X, const void* W, const int64_t* target, const float* lse, const float* dloss,
                           char* ws, cudaStream_t stream) {
    const bool first = p.v0 == 0 && !loss_begins(p, s);
    PairGroup<forge::kBlockLossGrad> g;
    std::memset(&g, 0, sizeof(g));
    FORGE_TRY(fill_group(g, p.grad, mc, ws, l.split));
    BlockProblem& b = g.prob[0];
    b.kb[0] = slices(s.d_model);
    FORGE_TRY(set_result(g, p.grad, 0, ws + l.g, p.ld, s.T));
    b.ld = p.ld;
    b.target = target;
    b.v0 = p.v0;
    b.vocab = s.vocab;
    b.ignore = s.ignore_index;
    b.lse = lse;
    b.dloss = dloss;
    b.unit = reinterpret_cast<const float*>(ws + l.unit);
    if (first) {
        b.own_unit = reinterpret_cast<float*>(ws + l.unit);
        FORGE_TRY(clear_counts(g, p.grad, ws, l.split, stream));
    }
    FORGE_TRY(set_map(g, p.grad, 0, 0, Operand{X, s.d_model, s.T, s.d_model}, false));
    FORGE_TRY(set_map(g, p.grad, 0, 1, Operand{static_cast<const char*>(W) + static_cast<size_t>(p.v0) * s.d_model * 2,
                                            s.d_model, p.n, s.d_model}, false));
    return launch<forge::kBlockLossGrad>(g, p.grad, stream);
}

forge_status run_loss_products(const Machine& mc, const LossBackward& l, const LossPiece& p, char* ws,
                               cudaStream_t stream) {
    if (p.np == 0) return FORGE_OK;
    return run_store(mc, p.out, p.pr, ws, l.split, stream);
}

// Joins the tiles' maxima and sums of one row: lse, and the loss of the target's logit that one tile's
// epilogue left in `loss`.  A block takes kRows rows (32 with many rows, so that loads of a part are
// whole lines; fewer with few rows, so that more blocks and threads share the parts).
constexpr int kFinishThreads = 512;

__device__ __forceinline__ void join(float& m, float& s, float vm, float vs) {
    const float mn = fmaxf(m, vm), base = forge::stats_base(mn);
    s = s * forge::exp2_fast(m - base) + vs * forge::exp2_fast(vm - base);
    m = mn;
}

template <int kRows>
__global__ void __launch_bounds__(kFinishThreads)
    loss_finish_kernel(const float2* stats, int parts, int rows, const int64_t* target, int64_t vocab, int64_t ignore,
                       float* loss, float* lse) {
    constexpr int kShares = kFinishThreads / kRows;
    __shared__ float2 part[kShares][kRows];
    forge::stream_wait();
    const int r = threadIdx.x % kRows, share = threadIdx.x / kRows;
    const int row = blockIdx.x * kRows + r;
    float m = -INFINITY, s = 0.0f;
    if (row < rows) {
        for (int first = share; first < parts; first += 8 * kShares) {
            float2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = first + i * kShares;
                v[i] = at < parts ? __ldcg(stats + static_cast<size_t>(at) * rows + row) : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) join(m, s, v[i].x, v[i].y);
        }
    }
    part[share][r] = make_float2(m, s);
    for (int n = kShares / 2; n > 0; n /= 2) {
        __syncthreads();
        if (share < n) {
            const float2 v = part[share + n][r];
            join(m, s, v.x, v.y);
            part[share][r] = make_float2(m, s);
        }
    }
    if (share != 0 || row >= rows) return;
    const float l = m == -INFINITY && s == 0.0f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(s));
    lse[row] = l;
    const int64_t t = target[row];
    loss[row] = t == ignore ? 0.0f : t >= 0 && t < vocab ? l - loss[row] : NAN;
}

// The largest finite |dloss| of the tokens that count, or 1 where there is none above 0; and the counters of the
// call's split tiles cleared: one block.
__global__ void __launch_bounds__(1024)
    loss_begin_kernel(const float* dloss, const int64_t* target, int64_t ignore, int rows, float* unit, uint32_t* counts,
                      int n_counts) {
    __shared__ float part[32];
    forge::stream_wait();
    for (int i = threadIdx.x; i < n_counts; i += 1024) counts[i] = 0u;
    float m = 0.0f;
    for (int i = threadIdx.x; i < rows; i += 1024) m = fmaxf(m, forge::loss_weight(dloss[i], target[i], ignore));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    m = part[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (threadIdx.x == 0) *unit = m > 0.0f ? m : 1.0f;
}

forge_status run_loss_begin(const LossBackward& l, const forge_loss_shape& s, const int64_t* target, const float* dloss,
                            char* ws, cudaStream_t stream) {
    return cuda_status(host::launch_early(loss_begin_kernel, dim3(1), dim3(1024), 0, stream, dloss, target,
                                          s.ignore_index, static_cast<int>(s.T), reinterpret_cast<float*>(ws + l.unit),
                                          reinterpret_cast<uint32_t*>(ws + l.split.counts), l.split.n_counts));
}

void describe(const Plan& p, int32_t* tile_cols, int32_t* whole, int32_t* cut, int32_t* parts) {
    *tile_cols = p.bn;
    for (int i = 0; i < p.n; ++i) {
        const Cut& c = p.cut[i];
        *whole += c.split_from;
        *cut += c.tiles_m * c.tiles_n - c.split_from;
        *parts = std::max(*parts, c.parts);
    }
}

}  // namespace

extern "C" {

int64_t forge_gated_mlp_workspace(const forge_gated_shape* shape, int32_t backward) {
    if (check_gated(shape) != FORGE_OK) return -1;
    Machine mc;
    if (shape->T == 0) return 0;
    if (machine(&mc) != FORGE_OK) return -1;
    if (!backward) return layout_gated_forward(mc, *shape).bytes;
    // with and without the weights' gradients and dX
    int64_t most = 0;
    for (int i = 0; i < 4; ++i)
        most = std::max(most, layout_gated_backward(mc, *shape, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                    nullptr, nullptr, i & 1, i >> 1, nullptr).bytes);
    return most;
}

forge_status forge_gated_mlp(const void* X, const void* Wg, const void* Wu, const void* Wd, const void* residual,
                             void* Y, void* G, void* U, void* workspace, int64_t workspace_bytes,
                             const forge_gated_shape* shape, struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    if (shape->T == 0) return FORGE_OK;
    FORGE_TRY(check_all({X, Wg, Wu, Wd, Y}));
    if ((G == nullptr) != (U == nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    if (!aligned(G, 32) || !aligned(U, 32) || !aligned(residual, 32)) return FORGE_ERR_MISALIGNED;
    Machine mc;
    FORGE_TRY(machine(&mc));
    const forge_gated_shape& s = *shape;
    GatedForward l = layout_gated_forward(mc, s);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    char* ws = static_cast<char*>(workspace);
    if (l.few) {
        forge::RowsArgs r{};
        r.x = static_cast<const uint16_t*>(X);
        r.w = static_cast<const uint16_t*>(Wg);
        r.w2 = static_cast<const uint16_t*>(Wu);
        r.y = reinterpret_cast<uint16_t*>(ws + l.h);
        r.g_out = static_cast<uint16_t*>(G);
        r.u_out = static_cast<uint16_t*>(U);
        r.T = static_cast<int>(s.T);
        r.N = static_cast<int>(s.d_ff);
        r.K = static_cast<int>(s.d_model);
        r.act = s.act;
        r.withhold = host::take_withhold() ? 16 : 0;
        r.status = mc.dev.status;
        r.wait_limit_ns = host::wait_limit_ns();
        FORGE_TRY(cuda_status(forge::launch_rows(r, true, mc.dev.num_sms, stream)));
        forge::RowsArgs d = r;
        d.x = r.y;
        d.w = static_cast<const uint16_t*>(Wd);
        d.w2 = nullptr;
        d.add = static_cast<const uint16_t*>(residual);
        d.y = static_cast<uint16_t*>(Y);
        d.N = static_cast<int>(s.d_model);
        d.K = static_cast<int>(s.d_ff);
        d.weights_ready = 1;
        d.withhold = 0;
        return cuda_status(forge::launch_rows(d, false, mc.dev.num_sms, stream));
    }
    PairGroup<forge::kBlockGatedFwd> g;
    std::memset(&g, 0, sizeof(g));
    FORGE_TRY(fill_group(g, l.up, mc, ws, l.split));
    FORGE_TRY(clear_counts(g, l.up, ws, l.split, stream));
    BlockProblem& b = g.prob[0];
    b.kb[0] = slices(s.d_model);
    b.ld = s.d_ff;
    b.keep = G != nullptr;
    if (b.keep) {
        FORGE_TRY(set_result(g, l.up, 0, G, s.d_ff, s.T));
        FORGE_TRY(set_result(g, l.up, 1, U, s.d_ff, s.T));
    }
    FORGE_TRY(set_result(g, l.up, 2, ws + l.h, s.d_ff, s.T));
    b.act = s.act;
    FORGE_TRY(set_map(g, l.up, 0, 0, Operand{X, s.d_model, s.T, s.d_model}, false));
    FORGE_TRY(set_map(g, l.up, 0, 1, Operand{Wg, s.d_model, s.d_ff, s.d_model}, false, true));
    FORGE_TRY(set_map(g, l.up, 0, 3, Operand{Wu, s.d_model, s.d_ff, s.d_model}, false, true));
    FORGE_TRY(launch<forge::kBlockGatedFwd>(g, l.up, stream));
    const Product y = product_nt(ws + l.h, Wd, s.T, s.d_model, s.d_ff, Y, residual);
    return run_store(mc, l.down, &y, ws, l.split, stream);
}

forge_status forge_gated_mlp_backward(const void* dY, const void* X, const void* G, const void* U, const void* Wg,
                                      const void* Wu, const void* Wd, void* dX, void* dWg, void* dWu, void* dWd,
                                      void* workspace, int64_t workspace_bytes, const forge_gated_shape* shape,
                                      struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    const forge_gated_shape& s = *shape;
    FORGE_TRY(check_all({dWg, dWu, dWd}));
    if (s.T > 0) FORGE_TRY(check_all({dY, X, G, U, Wg, Wu, Wd}));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    Machine mc;
    FORGE_TRY(machine(&mc));
    if (s.T == 0) {  // no tokens: the gradients are zero
        for (void* p : {dWg, dWu, dWd})
            if (cudaMemsetAsync(p, 0, static_cast<size_t>(s.d_ff) * s.d_model * 2, stream) != cudaSuccess)
                return FORGE_ERR_CUDA;
        return FORGE_OK;
    }
    char* ws = static_cast<char*>(workspace);
    const GatedBackward l = layout_gated_backward(mc, s, dY, X, Wg, Wu, dX, dWg, dWu, dWd, true, dX != nullptr, ws);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    FORGE_TRY(run_gated_dh(mc, l, dY, Wd, G, U, ws, s, stream));
    return run_store(mc, l.grads, l.pr, ws, l.split, stream);
}

forge_status forge_gated_mlp_backward_step(const void* dY, const void* X, const void* G, const void* U,
                                           const forge_layer* gate, const forge_layer* up, const forge_layer* down,
                                           void* dX, void* workspace, int64_t workspace_bytes, int32_t state,
                                           forge_opt_kind opt_kind, const forge_hparams* hp,
                                           const forge_gated_shape* shape, int64_t step, struct CUstream_st* stream) {
    FORGE_TRY(check_gated(shape));
    const forge_gated_shape& s = *shape;
    if (gate == nullptr || up == nullptr || down == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    for (const forge_layer* w : {gate, up})
        FORGE_TRY(host::check_step(w->W, w->m, w->v, w->qscales, opt_kind, hp, s.d_ff, s.d_model, state, step));
    FORGE_TRY(host::check_step(down->W, down->m, down->v, down->qscales, opt_kind, hp, s.d_model, s.d_ff, state, step));
    if (s.T > 0) FORGE_TRY(check_all({dY, X, G, U}));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    Machine mc;
    FORGE_TRY(machine(&mc));
    char* ws = static_cast<char*>(workspace);
    forge_layer layers[3] = {*gate, *up, *down};
    for (forge_layer& w : layers) {
        w.T = s.T;
        w.X = X;
        w.d_out = s.d_ff;
        w.d_in = s.d_model;
    }
    layers[2].d_out = s.d_model;
    layers[2].d_in = s.d_ff;
    if (s.T > 0) {
        const GatedBackward l = layout_gated_backward(mc, s, dY, X, gate->W, up->W, dX, nullptr, nullptr, nullptr, false,
                                                      dX != nullptr, ws);
        FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
        // the input gradients read the weights before the fused step replaces them: same stream, this order
        FORGE_TRY(run_gated_dh(mc, l, dY, down->W, G, U, ws, s, stream));
        if (dX != nullptr) FORGE_TRY(run_store(mc, l.grads, l.pr, ws, l.split, stream));
        layers[0].dY = ws + l.dg;
        layers[1].dY = ws + l.du;
        layers[2].dY = dY;
        layers[2].X = ws + l.h;
    }
    return forge_fused_dw_step_layers(layers, 3, state, opt_kind, hp, step, stream);
}

int64_t forge_linear_cross_entropy_workspace(const forge_loss_shape* shape, int32_t backward) {
    if (check_loss(shape) != FORGE_OK) return -1;
    Machine mc;
    if (shape->T == 0) return 0;
    if (machine(&mc) != FORGE_OK) return -1;
    if (!backward) return layout_loss_forward(mc, *shape).bytes;
    int64_t most = 0;
    for (int i = 0; i < 4; ++i) most = std::max(most, layout_loss_backward(mc, *shape, i & 1, i >> 1).bytes);
    return most;
}

forge_status forge_linear_cross_entropy(const void* X, const void* W, const int64_t* target, float* loss, float* lse,
                                        void* workspace, int64_t workspace_bytes, const forge_loss_shape* shape,
                                        struct CUstream_st* stream) {
    FORGE_TRY(check_loss(shape));
    const forge_loss_shape& s = *shape;
    if (s.T == 0) return FORGE_OK;
    FORGE_TRY(check_all({X, W}));
    if (target == nullptr || loss == nullptr || lse == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    if (!aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4)) return FORGE_ERR_MISALIGNED;
    Machine mc;
    FORGE_TRY(machine(&mc));
    const LossForward l = layout_loss_forward(mc, s);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    char* ws = static_cast<char*>(workspace);
    PairGroup<forge::kBlockLossStats> g;
    std::memset(&g, 0, sizeof(g));
    FORGE_TRY(fill_group(g, l.plan, mc, ws, l.split));
    FORGE_TRY(clear_counts(g, l.plan, ws, l.split, stream));
    BlockProblem& b = g.prob[0];
    b.kb[0] = slices(s.d_model);
    b.target = target;
    b.vocab = s.vocab;
    b.ignore = s.ignore_index;
    b.stats = reinterpret_cast<float2*>(ws + l.stats);
    b.target_logit = loss;
    FORGE_TRY(set_map(g, l.plan, 0, 0, Operand{X, s.d_model, s.T, s.d_model}, false));
    FORGE_TRY(set_map(g, l.plan, 0, 1, Operand{W, s.d_model, s.vocab, s.d_model}, false));
    FORGE_TRY(launch<forge::kBlockLossStats>(g, l.plan, stream));
    // as many rows a block as still give half of the SMs a block
    const int rows = s.T >= 16 * mc.dev.num_sms ? 32 : s.T >= 4 * mc.dev.num_sms ? 8 : 1;
    return cuda_status(host::launch_early(rows == 32  ? loss_finish_kernel<32>
                                          : rows == 8 ? loss_finish_kernel<8>
                                                      : loss_finish_kernel<1>,
                                          dim3(static_cast<unsigned>(ceil_div(s.T, rows))),
                                          dim3(kFinishThreads), 0, stream, b.stats, l.stat_parts, static_cast<int>(s.T),
                                          target, s.vocab, s.ignore_index, loss, lse));
}

forge_status forge_linear_cross_entropy_backward(const void* X, const void* W, const int64_t* target, const float* lse,
                                                 const float* dloss, void* dX, void* dW, void* workspace,
                                                 int64_t workspace_bytes, const forge_loss_shape* shape,
                                                 struct CUstream_st* stream) {
    FORGE_TRY(check_loss(shape));
    const forge_loss_shape& s = *shape;
    if (dX == nullptr && dW == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    if (!aligned(dX, 32) || !aligned(dW, 32)) return FORGE_ERR_MISALIGNED;
    if (s.T > 0) {
        FORGE_TRY(check_all({X, W}));
        if (target == nullptr || lse == nullptr || dloss == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
        if (!aligned(target, 8) || !aligned(lse, 4) || !aligned(dloss, 4)) return FORGE_ERR_MISALIGNED;
    }
    Machine mc;
    FORGE_TRY(machine(&mc));
    if (s.T == 0)
        return dW == nullptr ? FORGE_OK
                             : cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(s.vocab) * s.d_model * 2, stream));
    const bool dx = dX != nullptr, dw = dW != nullptr;
    const LossBackward l = layout_loss_backward(mc, s, dx, dw);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    char* ws = static_cast<char*>(workspace);
    for (int64_t i = 0; i < l.pieces; ++i) {
        const LossPiece p = loss_piece_of(mc, s, l, i, X, W, dX, dW, dx, dw, ws);
        if (i == 0 && loss_begins(p, s)) FORGE_TRY(run_loss_begin(l, s, target, dloss, ws, stream));
        FORGE_TRY(run_loss_grad(mc, l, p, s, X, W, target, lse, dloss, ws, stream));
        FORGE_TRY(run_loss_products(mc, l, p, ws, stream));
    }
    return FORGE_OK;
}

forge_status forge_linear_cross_entropy_step(const void* X, void* W, const int64_t* target, const float* lse,
                                             const float* dloss, void* dX, void* m, void* v, float* qscales,
                                             void* workspace, int64_t workspace_bytes, int32_t state,
                                             forge_opt_kind opt_kind, const forge_hparams* hp,
                                             const forge_loss_shape* shape, int64_t step, uint64_t seed,
                                             struct CUstream_st* stream) {
    FORGE_TRY(check_loss(shape));
    const forge_loss_shape& s = *shape;
    FORGE_TRY(host::check_step(W, m, v, qscales, opt_kind, hp, s.vocab, s.d_model, state, step));
    if (!aligned(dX, 32)) return FORGE_ERR_MISALIGNED;
    if (s.T > 0) {
        FORGE_TRY(check_all({X, W}));
        if (target == nullptr || lse == nullptr || dloss == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
        if (!aligned(target, 8) || !aligned(lse, 4) || !aligned(dloss, 4)) return FORGE_ERR_MISALIGNED;
    }
    Machine mc;
    FORGE_TRY(machine(&mc));
    if (s.T == 0)
        return host::fused_rows(nullptr, 0, X, 0, 0, s.vocab, W, m, v, qscales, opt_kind, hp, s.vocab, s.d_model, state,
                                step, seed, nullptr, stream);
    const bool dx = dX != nullptr;
    const LossBackward l = layout_loss_backward(mc, s, dx, false);
    FORGE_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    char* ws = static_cast<char*>(workspace);
    for (int64_t i = 0; i < l.pieces; ++i) {
        const LossPiece p = loss_piece_of(mc, s, l, i, X, W, dX, nullptr, dx, false, ws);
        if (i == 0 && loss_begins(p, s)) FORGE_TRY(run_loss_begin(l, s, target, dloss, ws, stream));
        // logits and dX read the piece's rows before the fused step replaces them
        FORGE_TRY(run_loss_grad(mc, l, p, s, X, W, target, lse, dloss, ws, stream));
        FORGE_TRY(run_loss_products(mc, l, p, ws, stream));
        // each piece numbers its elements from 0: a seed of its own keeps its random bits its own
        FORGE_TRY(host::fused_rows(ws + l.g, p.ld, X, s.T, p.v0, p.n, W, m, v, qscales, opt_kind, hp, s.vocab, s.d_model,
                                   state, step, seed ^ (static_cast<uint64_t>(i) << 40),
                                   reinterpret_cast<const float*>(ws + l.unit), stream));
    }
    return FORGE_OK;
}

forge_status forge_gated_mlp_launch_shape(const forge_gated_shape* shape, int32_t launch, int32_t* tile_cols,
                                          int32_t* whole, int32_t* cut, int32_t* parts) {
    FORGE_TRY(check_gated(shape));
    if (tile_cols == nullptr || whole == nullptr || cut == nullptr || parts == nullptr || launch < 0 || launch > 3)
        return FORGE_ERR_INVALID_ARGUMENT;
    *tile_cols = *whole = *cut = *parts = 0;
    if (shape->T == 0) return FORGE_OK;
    Machine mc;
    FORGE_TRY(machine(&mc));
    if (launch < 2) {
        const GatedForward l = layout_gated_forward(mc, *shape);
        if (!l.few) describe(launch == 0 ? l.up : l.down, tile_cols, whole, cut, parts);
    } else {
        const GatedBackward l = layout_gated_backward(mc, *shape, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                      nullptr, nullptr, true, true, nullptr);
        describe(launch == 2 ? l.dh : l.grads, tile_cols, whole, cut, parts);
    }
    return FORGE_OK;
}

forge_status forge_linear_cross_entropy_launch_shape(const forge_loss_shape* shape, int32_t launch, int32_t* tile_cols,
                                                     int32_t* whole, int32_t* cut, int32_t* parts) {
    FORGE_TRY(check_loss(shape));
    if (tile_cols == nullptr || whole == nullptr || cut == nullptr || parts == nullptr || launch < 0 || launch > 2)
        return FORGE_ERR_INVALID_ARGUMENT;
    *tile_cols = *whole = *cut = *parts = 0;
    if (shape->T == 0) return FORGE_OK;
    Machine mc;
    FORGE_TRY(machine(&mc));
    if (launch == 0) {
        describe(layout_loss_forward(mc, *shape).plan, tile_cols, whole, cut, parts);
    } else {
        const LossBackward l = layout_loss_backward(mc, *shape, true, true);
        const LossPiece p = loss_piece_of(mc, *shape, l, 0, nullptr, nullptr, nullptr, nullptr, true, true, nullptr);
        describe(launch == 1 ? p.grad : p.out, tile_cols, whole, cut, parts);
    }
    return FORGE_OK;
}

}  // extern "C"
