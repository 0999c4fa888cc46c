// The product kernel grouped by expert with a row product and weights' gradients.
#include "expert_instantiate.cuh"

template cudaError_t forge::launch_expert<forge::kExpertBoth>(const void*, int, int, cudaStream_t);
