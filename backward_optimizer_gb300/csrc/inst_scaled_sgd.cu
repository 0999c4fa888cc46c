// Kernel instantiations with a scaled dY for one optimizer (sgd).
#include "instantiate.cuh"
FORGE_INSTANTIATE_SCALED(forge::kSGD, forge::kEpiOptFP32)
