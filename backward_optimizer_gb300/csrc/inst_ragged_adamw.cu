// Kernel instantiations with a weight for each expert for one optimizer (adamw).
#include "instantiate.cuh"
FORGE_INSTANTIATE_OPT_RAGGED(forge::kAdamW)
