// Kernel instantiations with a scaled dY for one optimizer (adamw).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_SCALED(forge::kAdamW)
