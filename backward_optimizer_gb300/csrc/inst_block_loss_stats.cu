// The matrix-product kernel with the epilogue kBlockLossStats.
#include "block_instantiate.cuh"

template cudaError_t forge::launch_block<forge::kBlockLossStats>(const void*, int, int, cudaStream_t);
