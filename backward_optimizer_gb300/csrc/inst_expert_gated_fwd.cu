// The product kernel grouped by expert with the epilogue kBlockGatedFwd.
#include "expert_instantiate.cuh"

template cudaError_t forge::launch_expert<forge::kBlockGatedFwd>(const void*, int, int, cudaStream_t);
