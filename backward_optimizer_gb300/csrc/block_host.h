// block_host.h -- what the host side of the operators made of matrix products has in common (internal):
// argument checks, workspace layout, the machine, and encoded tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "block_launch.h"
#include "forge.h"
#include "host.h"

#define FORGE_TRY(expr)                      \
    do {                                     \
        const forge_status st_ = (expr);     \
        if (st_ != FORGE_OK) return st_;     \
    } while (0)

namespace forge {
namespace host {

constexpr int64_t kMaxDim = 1ll << 30;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline forge_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA; }

struct Machine {
    Device dev;
    int pairs;  // CTA pairs resident at once
};

inline forge_status machine(Machine* m) {
    forge_status st = device(&m->dev);
    if (st != FORGE_OK) return st;
    static std::atomic<int> pairs[64];
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) return FORGE_ERR_CUDA;
    d &= 63;
    int n = pairs[d].load();
    if (n == 0) {
        if (block_pairs(m->dev.num_sms, &n) != cudaSuccess || n < 1) return FORGE_ERR_CUDA;
        pairs[d].store(n);
    }
    m->pairs = n;
    return FORGE_OK;
}

// Non-null and 32-byte aligned.
inline forge_status check_all(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (p == nullptr) return FORGE_ERR_INVALID_ARGUMENT;
    for (const void* p : ps)
        if (!aligned(p, 32)) return FORGE_ERR_MISALIGNED;
    return FORGE_OK;
}

inline forge_status check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need == 0) return FORGE_OK;
    if (ws == nullptr || have < need) return FORGE_ERR_INVALID_ARGUMENT;
    return aligned(ws, 256) ? FORGE_OK : FORGE_ERR_MISALIGNED;
}

// Workspace: regions one after another, each 256-byte aligned.
struct Arena {
    int64_t used = 0;
    int64_t take(int64_t bytes) {
        const int64_t at = used;
        used += round_up(bytes, 256);
        return at;
    }
};

struct Operand {
    const void* base;
    int64_t cols, rows, ld;  // as it lies in memory
};

// Encoded tensor maps of recent calls, per host thread, as forge_api.cu keeps them for the weight-gradient
// kernels: a map is plain host data determined by its key.
struct MapKey {
    const void* base;
    int64_t cols, rows, ld;
    int mn, extent;
    int64_t experts = 0;  // of operands that a matrix for each expert makes up (expert_api.cu)
    bool operator==(const MapKey& o) const {
        return base == o.base && cols == o.cols && rows == o.rows && ld == o.ld && mn == o.mn && extent == o.extent &&
               experts == o.experts;
    }
};
struct MapSlot {
    MapKey key;
    CUtensorMap map;
    bool used;
};
constexpr int kMapSlots = 128;
inline thread_local MapSlot t_maps[kMapSlots];

template <class Encode>
forge_status kept_map(CUtensorMap* map, const MapKey& key, Encode&& encode) {
    uint64_t h = reinterpret_cast<uintptr_t>(key.base) * 0x9E3779B97F4A7C15ull;
    h ^= static_cast<uint64_t>(key.cols) * 0xC2B2AE3D27D4EB4Full ^ static_cast<uint64_t>(key.rows) * 0x165667B19E3779F9ull;
    h ^= static_cast<uint64_t>(key.ld * 1024 + key.extent * 2 + key.mn) * 0x85EBCA77C2B2AE63ull;
    MapSlot& slot = t_maps[(h >> 32) % kMapSlots];
    if (slot.used && slot.key == key) {
        *map = slot.map;
        return FORGE_OK;
    }
    const forge_status st = encode();
    if (st == FORGE_OK) slot = MapSlot{key, *map, true};
    return st;
}

}  // namespace host
}  // namespace forge
