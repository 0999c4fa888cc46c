// Kernel instantiations with a weight for each expert for one optimizer (sgd).
#include "instantiate.cuh"
FORGE_INSTANTIATE_RAGGED(forge::kSGD, forge::kEpiOptFP32)
