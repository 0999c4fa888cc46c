// block_instantiate.cuh -- defines the launchers of block_launch.h for one epilogue.
#pragma once

#include <atomic>

#include "block_kernel.cuh"
#include "block_launch.h"

namespace forge {

template <int BN, int CG, int EPI>
cudaError_t block_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int units, cudaStream_t stream) {
    using C = BlockCfg<BN, CG, EPI>;
    static std::atomic<uint64_t> configured{0};  // one bit per device ordinal
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        err = cudaFuncSetAttribute(forge_block_kernel<BN, CG, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   C::kSmemBytes);
        if (err != cudaSuccess) return err;
        configured.fetch_or(bit);
    }
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(units * CG, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cudaSuccess;
}

template <int BN, int CG, int EPI>
cudaError_t launch_block_as(const void* group, int units, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cudaError_t err = block_config<BN, CG, EPI>(cfg, attr, units, stream);
    if (err != cudaSuccess) return err;
    return cudaLaunchKernelEx(&cfg, forge_block_kernel<BN, CG, EPI>, static_cast<const GroupOf<CG, EPI>&>(*static_cast<const PairGroup<EPI>*>(group)));
}

template <int EPI>
cudaError_t launch_block(const void* group, int bn, int units, cudaStream_t stream) {
    if (bn == 256) return launch_block_as<256, 2, EPI>(group, units, stream);
    return bn == 128 ? launch_block_as<128, 1, EPI>(group, units, stream) : launch_block_as<64, 1, EPI>(group, units, stream);
}

}  // namespace forge
