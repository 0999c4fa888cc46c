// expert_instantiate.cuh -- defines the launchers of expert_launch.h for one epilogue.
#pragma once

#include <atomic>

#include "expert_kernel.cuh"
#include "expert_launch.h"

namespace forge {

template <int BN, int CG, int EPI>
cudaError_t launch_expert_as(const void* group, int units, cudaStream_t stream) {
    using C = ExpertCfg<BN, CG, EPI>;
    static std::atomic<uint64_t> configured{0};  // one bit per device ordinal
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        err = cudaFuncSetAttribute(forge_expert_kernel<BN, CG, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   C::kSmemBytes);
        if (err != cudaSuccess) return err;
        configured.fetch_or(bit);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * CG, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, forge_expert_kernel<BN, CG, EPI>, *static_cast<const ExpertGroup<EPI>*>(group));
}

template <int EPI>
cudaError_t launch_expert(const void* group, int bn, int units, cudaStream_t stream) {
    return bn == 256 ? launch_expert_as<256, 2, EPI>(group, units, stream) : launch_expert_as<128, 1, EPI>(group, units, stream);
}

}  // namespace forge
