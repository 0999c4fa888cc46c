// Kernel instantiations with a scaled dY for one optimizer (adagrad).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kAdaGrad)
