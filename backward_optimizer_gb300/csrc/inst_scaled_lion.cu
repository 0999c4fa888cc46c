// Kernel instantiations with a scaled dY for one optimizer (lion).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kLion)
