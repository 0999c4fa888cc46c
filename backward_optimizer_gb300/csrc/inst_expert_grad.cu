// The product kernel grouped by expert with the epilogue kExpertGrad.
#include "expert_instantiate.cuh"

template cudaError_t forge::launch_expert<forge::kExpertGrad>(const void*, int, int, cudaStream_t);
