// The matrix-product kernel with the epilogue kBlockGatedFwd.
#include "block_instantiate.cuh"

template cudaError_t forge::launch_block<forge::kBlockGatedFwd>(const void*, int, int, cudaStream_t);
