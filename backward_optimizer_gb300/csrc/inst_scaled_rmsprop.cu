// Kernel instantiations with a scaled dY for one optimizer (rmsprop).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kRMSprop)
