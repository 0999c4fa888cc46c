// Kernel instantiations with a scaled dY for one optimizer (nadam).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kNAdam)
