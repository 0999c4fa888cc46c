// The matrix-product kernel with the epilogue kBlockGatedBwd.
#include "block_instantiate.cuh"

template cudaError_t forge::launch_block<forge::kBlockGatedBwd>(const void*, int, int, cudaStream_t);
