// The matrix-product kernel with the epilogue kBlockLossGrad.
#include "block_instantiate.cuh"

template cudaError_t forge::launch_block<forge::kBlockLossGrad>(const void*, int, int, cudaStream_t);
