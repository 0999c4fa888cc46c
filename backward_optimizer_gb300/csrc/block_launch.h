// block_launch.h -- host-side launchers of the matrix-product kernel (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace forge {

struct RowsArgs;

constexpr int kMaxProducts = 4;  // products of one kBlockStore launch

// One launch of EPI on CTA pairs with 256 x 256 tiles (bn = 256) or single CTAs with 128 x bn tiles (128,
// 64); group: a PairGroup<EPI>; units: pairs or CTAs.
template <int EPI> cudaError_t launch_block(const void* group, int bn, int units, cudaStream_t stream);

// CTA pairs that the current device runs at once.
cudaError_t block_pairs(int num_sms, int* pairs);

// Whether the few-token kernel (rows_kernel.cuh) takes T tokens and rows of K weights.
bool rows_fit(int64_t T, int64_t K, bool gated);
cudaError_t launch_rows(RowsArgs a, bool gated, int num_sms, cudaStream_t stream);

}  // namespace forge
