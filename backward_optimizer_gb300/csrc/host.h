// host.h -- host-side services of forge_api.cu for the library's other translation units (internal;
// not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "forge.h"

namespace forge {
namespace host {

struct Device {
    int num_sms;
    int* status;  // device status word
};

// The current device, checked to be sm_103a.
forge_status device(Device* out);

// Tensor map of a bfloat16 array of three dimensions (strides in bytes, of the second and third), read in
// boxes with the 128-byte swizzle: the box's innermost extent is 64 elements.
forge_status encode_map(CUtensorMap* map, const void* base, const uint64_t (&dims)[3], const uint64_t (&strides)[2],
                        const uint32_t (&box)[3]);

// Tensor map of a row-major bfloat16 result [rows, cols] in one piece, written in boxes of 32 x 32 with the
// 64-byte swizzle.
forge_status encode_result_map(CUtensorMap* map, void* base, int64_t cols, int64_t rows);

uint64_t wait_limit_ns();
uint64_t acc_wait_limit_ns(int64_t k_blocks);
int take_withhold();  // the test switch, consumed by the launch that takes it
void count_launch();

// Launches `kernel` so that it may start while the kernel before it on the stream is still running: for
// kernels that call stream_wait() (ptx.cuh) before they touch memory.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The fused step's argument checks for a layer.
forge_status check_step(const void* W, const void* m, const void* v, const float* qscales, forge_opt_kind k,
                        const forge_hparams* hp, int64_t d_out, int64_t d_in, int32_t state, int64_t step);

// The fused step on rows row0 .. row0 + rows - 1 of a layer's weights [d_out, d_in]: dY [T, rows] with
// rows `dy_ld` elements apart (a multiple of 8), X [T, d_in]; W, m, v and qscales are the whole layer's.  unit (device
// memory, or null): dY is the gradient divided by it.
forge_status fused_rows(const void* dY, int64_t dy_ld, const void* X, int64_t T, int64_t row0, int64_t rows, void* W,
                        void* m, void* v, float* qscales, forge_opt_kind k, const forge_hparams* hp, int64_t d_out,
                        int64_t d_in, int32_t state, int64_t step, uint64_t seed, const float* unit,
                        cudaStream_t stream);

}  // namespace host
}  // namespace forge
