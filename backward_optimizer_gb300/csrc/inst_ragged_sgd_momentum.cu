// Kernel instantiations with a weight for each expert for one optimizer (sgd_momentum).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_RAGGED(forge::kSGDMomentum)
