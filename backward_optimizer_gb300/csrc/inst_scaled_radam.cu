// Kernel instantiations with a scaled dY for one optimizer (radam).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kRAdam)
