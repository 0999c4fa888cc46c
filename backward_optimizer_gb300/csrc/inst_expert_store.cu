// The product kernel grouped by expert with the epilogue kBlockStore.
#include "expert_instantiate.cuh"

template cudaError_t forge::launch_expert<forge::kBlockStore>(const void*, int, int, cudaStream_t);
