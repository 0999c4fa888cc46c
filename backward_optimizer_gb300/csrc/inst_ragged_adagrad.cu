// Kernel instantiations with a weight for each expert for one optimizer (adagrad).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_RAGGED(forge::kAdaGrad)
