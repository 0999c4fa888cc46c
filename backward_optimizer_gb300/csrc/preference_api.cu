// preference_api.cu -- the C ABI of the preference loss (include/forge.h), and its kernels.
//
// Sequence i of 2 P (chosen ones 0 .. P-1, rejected ones P .. 2P-1) owns tokens offsets[i] .. offsets[i+1]-1.
//   score_i = sum over its tokens of (ref - nll) (mean: divided by their number),
//   z_p = beta (score_p - score_{P+p}) - margin, loss_p = f(z_p).
//
// The sums are the work.  Sequences are ragged, from none to all of the tokens, so they are not what is dealt out:
// tokens are, `chunk` to a warp.  A warp finds the first sequence that reaches into its tokens (two or three steps
// of a 32-way search) and leaves one partial sum for each sequence it meets.  Chunk c and sequence i meet at most
// once and both grow along the tokens, so c + i numbers the meetings without a gap for two: that is the partial's
// place, and it needs no counter.  A second launch adds a sequence's partials in their order, so results do not
// depend on timing; up to 4096 tokens one block does both.
//
// Over long sequences the policy's and the reference's sums nearly cancel, so they are kept to some 48 bits: a value
// is a pair of binary32, each addition exact up to the pair's second part (Knuth's two-sum).  Binary64 would do the
// same, but the chip has few units for it (262144 tokens of 256 pairs: 21.2 us with it).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "forge.h"
#include "host.h"
#include "ptx.cuh"

namespace {

namespace host = forge::host;

constexpr int kThreads = 256, kWarps = kThreads / 32;

// hi + lo
struct Wide {
    float hi, lo;
};

// a + b, and what its rounding left out
__device__ __forceinline__ Wide two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return Wide{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ void add(Wide& a, Wide b) {
    const Wide s = two_sum(a.hi, b.hi);
    a.hi = s.hi;
    a.lo = __fadd_rn(a.lo, __fadd_rn(s.lo, b.lo));
}
// An infinite sum has no second part (two_sum leaves a NaN there).
__device__ __forceinline__ Wide settled(Wide a) {
    if (!(fabsf(a.hi) < INFINITY)) return Wide{a.hi, 0.0f};
    const Wide s = two_sum(a.hi, a.lo);
    return s;
}
// a / n
__device__ __forceinline__ Wide divided(Wide a, int n) {
    const float by = static_cast<float>(n), rest = static_cast<float>(n - static_cast<int>(by));
    const float q = a.hi / by;
    return settled(Wide{q, (__fmaf_rn(-q, by, a.hi) + a.lo - q * rest) / by});
}

struct Partial {
    float hi, lo;
    int count, unused;
};

struct PrefArgs {
    const float* nll;
    const float* ref;      // or null
    const uint8_t* mask;   // or null
    const int* offsets;    // [2 pairs + 1]
    float* loss;
    float* reward;         // or null
    float* slope;          // or null
    Partial* parts;
    int tokens, pairs, chunk;
    int kind, mean;
    float beta, smoothing, margin;
    const float* dloss;    // backward
    float* dnll;
};

// An offset, within the tokens whatever it holds.
__device__ __forceinline__ int offset_at(const PrefArgs& a, int i) { return min(max(__ldcg(a.offsets + i), 0), a.tokens); }

// The last sequence that starts at or before token t, or -1: a warp's search, 32 offsets at a time.
__device__ __forceinline__ int sequence_of(const PrefArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = 2 * a.pairs;  // as many offsets as are at or before t
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool at = i < hi && offset_at(a, i) <= t;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, at));
        if (n == 0) break;
        const int next = lo + n * step;  // offsets lo .. lo + (n - 1) step are at or before t, that at `next` is not
        lo += (n - 1) * step + 1;
        hi = min(hi, next);
    }
    return lo - 1;
}

// f(sequence, its first token, one past its last) for each sequence that has tokens among t0 .. t1-1, these tokens only,
// by the whole warp.  Any number of empty sequences in between costs one search (one by one they would take a trip to memory
// each, seconds for millions of them).  Offsets out of order take no more steps than those in order can: a sequence for
// each token, and an empty one in front of it.
template <class F>
__device__ __forceinline__ void each_sequence(const PrefArgs& a, int t0, int t1, F&& f) {
    int i = max(sequence_of(a, t0), 0), begin = offset_at(a, i);
    for (int left = 2 * (t1 - t0) + 2; left > 0 && i < 2 * a.pairs && begin < t1; --left) {
        const int end = offset_at(a, i + 1);
        if (begin < end) {
            const int from = max(begin, t0), to = min(end, t1);
            if (from < to) f(i, from, to);
            ++i;
            begin = end;
        } else {  // the last sequence that starts where this empty one does
            i = max(sequence_of(a, begin), i + 1);
            begin = offset_at(a, i);
        }
    }
}

// f and its slope
__device__ __forceinline__ void pair_loss(const PrefArgs& a, float z, float& loss, float& slope) {
    if (a.kind == FORGE_PREF_SIGMOID) {
        const float e = expf(-fabsf(z)), l = log1pf(e);        // log(1 + exp(-|z|))
        const float small = e / (1.0f + e), large = 1.0f / (1.0f + e);  // of sigmoid(z), sigmoid(-z)
        const float pos = z >= 0.0f ? large : small, neg = z >= 0.0f ? small : large;
        const float lose = l + (z < 0.0f ? -z : 0.0f), win = l + (z > 0.0f ? z : 0.0f);  // -log sigmoid(z), -log sigmoid(-z)
        loss = (1.0f - a.smoothing) * lose + a.smoothing * win;
        slope = a.smoothing * pos - (1.0f - a.smoothing) * neg;
        if (a.smoothing == 0.0f) loss = lose;  // not 0 times an infinite term
        if (z != z) loss = slope = z;
    } else if (a.kind == FORGE_PREF_HINGE) {
        loss = z >= 1.0f ? 0.0f : 1.0f - z;
        slope = z < 1.0f ? -1.0f : z != z ? z : 0.0f;
    } else {
        const float d = (z - 0.5f) / a.beta;
        loss = d * d;
        slope = 2.0f * d / a.beta;
    }
}

__device__ __forceinline__ void sum_all(Wide& v, int& n) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        add(v, Wide{__shfl_xor_sync(0xFFFFFFFFu, v.hi, o), __shfl_xor_sync(0xFFFFFFFFu, v.lo, o)});
        n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
}

// The partial sums of one chunk of tokens: a warp.
__device__ __forceinline__ void chunk_sums(const PrefArgs& a, int c) {
    const int lane = threadIdx.x & 31;
    const int t0 = c * a.chunk, t1 = static_cast<int>(min(static_cast<int64_t>(t0) + a.chunk, static_cast<int64_t>(a.tokens)));
    each_sequence(a, t0, t1, [&](int i, int from, int to) {
        Wide s{0.0f, 0.0f};
        int n = 0;
        constexpr int kAhead = 8;
        for (int t = from + lane; t < to; t += 32 * kAhead) {
            float x[kAhead], r[kAhead];
            bool counts[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const bool in = t + 32 * j < to;
                counts[j] = in && (a.mask == nullptr || a.mask[t + 32 * j] != 0);
                x[j] = in ? a.nll[t + 32 * j] : 0.0f;
                r[j] = in && a.ref != nullptr ? a.ref[t + 32 * j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                // a masked token's values are left out, whatever they are
                if (counts[j]) {
                    add(s, two_sum(r[j], -x[j]));
                    ++n;
                }
            }
        }
        sum_all(s, n);
        if (lane == 0) a.parts[c + i] = Partial{s.hi, s.lo, n, 0};
    });
}

// One pair from its sequences' partials: a warp.
__device__ __forceinline__ void finish_pair(const PrefArgs& a, int p) {
    const int lane = threadIdx.x & 31;
    Wide score[2];
    float per[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = p + h * a.pairs, begin = offset_at(a, i), end = offset_at(a, i + 1);
        Wide s{0.0f, 0.0f};
        int n = 0;
        if (begin < end) {
            const int last = (end - 1) / a.chunk;
#pragma unroll 4
            for (int c = begin / a.chunk + lane; c <= last; c += 32) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.parts + c + i));
                add(s, Wide{v.x, v.y});
                n += __float_as_int(v.z);
            }
        }
        sum_all(s, n);
        const bool several = a.mean && n > 1;
        score[h] = several ? divided(settled(s), n) : settled(s);
        per[h] = several ? 1.0f / static_cast<float>(n) : 1.0f;
    }
    if (lane != 0) return;
    auto times_beta = [&](Wide v, float less) {
        return v.lo == 0.0f ? __fmaf_rn(a.beta, v.hi, -less) : __fmaf_rn(a.beta, v.hi, __fmaf_rn(a.beta, v.lo, -less));
    };
    Wide d = two_sum(score[0].hi, -score[1].hi);
    d.lo += score[0].lo - score[1].lo;
    float loss, g;
    pair_loss(a, times_beta(settled(d), a.margin), loss, g);
    a.loss[p] = loss;
    if (a.reward != nullptr) {
        a.reward[p] = times_beta(score[0], 0.0f);
        a.reward[a.pairs + p] = times_beta(score[1], 0.0f);
    }
    if (a.slope != nullptr) {  // of a token's nll: it counts -1 in its score
        a.slope[p] = -g * a.beta * per[0];
        a.slope[a.pairs + p] = g * a.beta * per[1];
    }
}

// kAll: one block makes the sums and finishes the pairs itself.
template <bool kAll>
__global__ void __launch_bounds__(kAll ? 1024 : kThreads) pref_sums_kernel(const PrefArgs a) {
    forge::stream_wait();
    const int warp = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int chunks = (a.tokens + a.chunk - 1) / a.chunk;
    if constexpr (kAll) {
        for (int c = warp; c < chunks; c += 32) chunk_sums(a, c);
        __threadfence_block();
        __syncthreads();
        for (int p = warp; p < a.pairs; p += 32) finish_pair(a, p);
    } else if (warp < chunks) {
        chunk_sums(a, warp);
    }
}

__global__ void __launch_bounds__(kThreads) pref_finish_kernel(const PrefArgs a) {
    forge::stream_wait();
    const int p = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (p < a.pairs) finish_pair(a, p);
}

// dnll of one chunk of tokens: a warp.  A token of no sequence has gradient 0, and so has a masked one.
__global__ void __launch_bounds__(kThreads) pref_grad_kernel(const PrefArgs a) {
    forge::stream_wait();
    const int lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int chunks = (a.tokens + a.chunk - 1) / a.chunk;
    if (c >= chunks) return;
    const int t0 = c * a.chunk, t1 = static_cast<int>(min(static_cast<int64_t>(t0) + a.chunk, static_cast<int64_t>(a.tokens)));
    const int first = a.pairs > 0 ? offset_at(a, 0) : a.tokens, end = a.pairs > 0 ? offset_at(a, 2 * a.pairs) : 0;
    for (int t = t0 + lane; t < min(t1, first); t += 32) a.dnll[t] = 0.0f;
    for (int t = max(t0, max(first, end)) + lane; t < t1; t += 32) a.dnll[t] = 0.0f;
    if (a.pairs == 0) return;
    each_sequence(a, t0, t1, [&](int i, int from, int to) {
        const float g = a.slope[i] * a.dloss[i < a.pairs ? i : i - a.pairs];
        for (int t = from + lane; t < to; t += 32) a.dnll[t] = a.mask == nullptr || a.mask[t] != 0 ? g : 0.0f;
    });
}

constexpr int kOneBlock = 4096, kOneBlockPairs = 64;  // tokens and pairs that one block takes by itself

// Tokens of a warp: as many as a few sequences have, between 32 and 256 (128 where one block does it all), more only
// where the partials of one long sequence would be too many for the warp that adds them.
int chunk_of(int64_t tokens, int64_t pairs) {
    const int64_t most = tokens <= kOneBlock ? 128 : 256;
    int64_t chunk = 32;
    while (chunk < most && chunk < 4 * (tokens / std::max<int64_t>(2 * pairs, 1))) chunk *= 2;
    while (chunk * 8192 < tokens) chunk *= 2;
    return static_cast<int>(chunk);
}

forge_status check(const forge_preference_shape* s) {
    if (s == nullptr || s->reserved != 0) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->tokens < 0 || s->tokens > (1ll << 30) || s->pairs < 0 || s->pairs > (1ll << 24)) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->kind != FORGE_PREF_SIGMOID && s->kind != FORGE_PREF_HINGE && s->kind != FORGE_PREF_IPO) return FORGE_ERR_INVALID_ARGUMENT;
    if (!(s->beta > 0.0f) || !std::isfinite(s->beta) || !std::isfinite(s->margin)) return FORGE_ERR_INVALID_ARGUMENT;
    if (!(s->smoothing >= 0.0f && s->smoothing < 1.0f)) return FORGE_ERR_INVALID_ARGUMENT;
    if (s->smoothing != 0.0f && s->kind != FORGE_PREF_SIGMOID) return FORGE_ERR_INVALID_ARGUMENT;
    return FORGE_OK;
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

PrefArgs args_of(const forge_preference_shape& s) {
    PrefArgs a{};
    a.tokens = static_cast<int>(s.tokens);
    a.pairs = static_cast<int>(s.pairs);
    a.chunk = chunk_of(s.tokens, s.pairs);
    a.kind = s.kind;
    a.mean = s.mean;
    a.beta = s.beta;
    a.smoothing = s.smoothing;
    a.margin = s.margin;
    return a;
}

unsigned blocks(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

}  // namespace

extern "C" {

int64_t forge_preference_loss_workspace(const forge_preference_shape* shape) {
    if (check(shape) != FORGE_OK) return -1;
    if (shape->pairs == 0) return 0;
    const int64_t chunk = chunk_of(shape->tokens, shape->pairs);
    return ((shape->tokens + chunk - 1) / chunk + 2 * shape->pairs) * static_cast<int64_t>(sizeof(Partial));
}

forge_status forge_preference_loss(const float* nll, const float* ref, const uint8_t* mask, const int32_t* offsets, float* loss,
                                   float* reward, float* slope, void* workspace, int64_t workspace_bytes,
                                   const forge_preference_shape* shape, struct CUstream_st* stream) {
    const forge_status bad = check(shape);
    if (bad != FORGE_OK) return bad;
    if (shape->pairs == 0) return FORGE_OK;
    if (offsets == nullptr || loss == nullptr || (shape->tokens > 0 && nll == nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    if (workspace == nullptr || workspace_bytes < forge_preference_loss_workspace(shape)) return FORGE_ERR_INVALID_ARGUMENT;
    for (const void* p : {static_cast<const void*>(nll), static_cast<const void*>(ref), static_cast<const void*>(offsets),
                          static_cast<const void*>(loss), static_cast<const void*>(reward), static_cast<const void*>(slope)})
        if (off(p, 4)) return FORGE_ERR_MISALIGNED;
    if (off(workspace, 256)) return FORGE_ERR_MISALIGNED;
    host::Device dev;
    const forge_status st = host::device(&dev);
    if (st != FORGE_OK) return st;
    PrefArgs a = args_of(*shape);
    a.nll = nll;
    a.ref = ref;
    a.mask = mask;
    a.offsets = offsets;
    a.loss = loss;
    a.reward = reward;
    a.slope = slope;
    a.parts = static_cast<Partial*>(workspace);
    const dim3 block(kThreads);
    if (shape->tokens <= kOneBlock && shape->pairs <= kOneBlockPairs)
        return host::launch_early(pref_sums_kernel<true>, dim3(1), dim3(1024), 0, stream, a) == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
    if (a.tokens > 0 && host::launch_early(pref_sums_kernel<false>, dim3(blocks((a.tokens + a.chunk - 1) / a.chunk)), block, 0,
                                           stream, a) != cudaSuccess)
        return FORGE_ERR_CUDA;
    return host::launch_early(pref_finish_kernel, dim3(blocks(a.pairs)), block, 0, stream, a) == cudaSuccess ? FORGE_OK
                                                                                                            : FORGE_ERR_CUDA;
}

forge_status forge_preference_loss_backward(const float* dloss, const float* slope, const uint8_t* mask, const int32_t* offsets,
                                            float* dnll, const forge_preference_shape* shape, struct CUstream_st* stream) {
    const forge_status bad = check(shape);
    if (bad != FORGE_OK) return bad;
    if (shape->tokens == 0) return FORGE_OK;
    if (dnll == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    if (shape->pairs > 0 && (dloss == nullptr || slope == nullptr || offsets == nullptr)) return FORGE_ERR_INVALID_ARGUMENT;
    for (const void* p : {static_cast<const void*>(dloss), static_cast<const void*>(slope), static_cast<const void*>(offsets),
                          static_cast<const void*>(dnll)})
        if (off(p, 4)) return FORGE_ERR_MISALIGNED;
    host::Device dev;
    const forge_status st = host::device(&dev);
    if (st != FORGE_OK) return st;
    PrefArgs a = args_of(*shape);
    a.dloss = dloss;
    a.slope = const_cast<float*>(slope);
    a.mask = mask;
    a.offsets = offsets;
    a.dnll = dnll;
    return host::launch_early(pref_grad_kernel, dim3(blocks((a.tokens + a.chunk - 1) / a.chunk)), dim3(kThreads), 0, stream, a) ==
                   cudaSuccess
               ? FORGE_OK
               : FORGE_ERR_CUDA;
}

}  // extern "C"
