// The product kernel grouped by expert with the epilogue kBlockGatedBwd.
#include "expert_instantiate.cuh"

template cudaError_t forge::launch_expert<forge::kBlockGatedBwd>(const void*, int, int, cudaStream_t);
