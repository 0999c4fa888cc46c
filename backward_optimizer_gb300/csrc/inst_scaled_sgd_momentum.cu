// Kernel instantiations with a scaled dY for one optimizer (sgd_momentum).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kSGDMomentum)
