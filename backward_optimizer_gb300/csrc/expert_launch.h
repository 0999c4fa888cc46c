// expert_launch.h -- host-side launchers of the products grouped by expert (internal).
#pragma once

#include <cuda_runtime.h>

namespace forge {

// One launch of EPI on CTA pairs with 256 x 256 tiles (bn = 256) or single CTAs with a_rows x 128 tiles;
// group: an ExpertGroup<EPI>; units: pairs or CTAs.
template <int EPI> cudaError_t launch_expert(const void* group, int bn, int units, cudaStream_t stream);

}  // namespace forge
