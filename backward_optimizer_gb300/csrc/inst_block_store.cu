// The matrix-product kernel with the epilogue kBlockStore.
#include "block_instantiate.cuh"

template cudaError_t forge::launch_block<forge::kBlockStore>(const void*, int, int, cudaStream_t);

cudaError_t forge::block_pairs(int num_sms, int* pairs) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cudaError_t err = block_config<256, 2, kBlockStore>(cfg, attr, num_sms, nullptr);
    if (err != cudaSuccess) return err;
    // every epilogue has one CTA per SM, so one count serves all
    return cudaOccupancyMaxActiveClusters(pairs, forge_block_kernel<256, 2, kBlockStore>, &cfg);
}
