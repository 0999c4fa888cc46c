// Kernel instantiations with a weight for each expert for one optimizer (rmsprop).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_RAGGED(forge::kRMSprop)
