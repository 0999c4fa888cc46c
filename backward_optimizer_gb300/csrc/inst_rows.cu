// The few-token product kernel: shapes, dispatch, launch.
#include <algorithm>

#include "block_launch.h"
#include "host.h"
#include "rows_kernel.cuh"

namespace forge {

namespace {

template <int T, int ROWS, int VECS, bool GATED>
cudaError_t launch_rows_as(const RowsArgs& a, int blocks, int smem, cudaStream_t stream) {
    auto kernel = forge_rows_kernel<T, ROWS, VECS, GATED>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsRing);
    if (err != cudaSuccess) return err;
    return host::launch_early(kernel, dim3(blocks), dim3(kRowsThreads), static_cast<size_t>(smem), stream, a);
}

// Weight rows per group by the length of a row: about 32 KB a group, so that its join is small beside its
// copies; a gated group has at least two.
constexpr int rows_for(int vecs, bool gated) { return vecs == 1 ? 4 : vecs == 2 || gated ? 2 : 1; }

template <int T, int VECS>
cudaError_t launch_rows_at(const RowsArgs& a, bool gated, int blocks, int smem, cudaStream_t stream) {
    return gated ? launch_rows_as<T, rows_for(VECS, true), VECS, true>(a, blocks, smem, stream)
                 : launch_rows_as<T, rows_for(VECS, false), VECS, false>(a, blocks, smem, stream);
}

int vecs_of(int64_t K) { return static_cast<int>((K / 8 + kRowsLanes - 1) / kRowsLanes); }

// Slots of the ring, at least three; 0: the rows are too long for it.
int slots_for(int64_t K, bool gated) {
    const int64_t fit = kRowsRing / (rows_for(vecs_of(K), gated) * K * 2);
    return fit < 3 ? 0 : static_cast<int>(std::min<int64_t>(fit, kRowsMaxSlots));
}

}  // namespace

bool rows_fit(int64_t T, int64_t K, bool gated) {
    // Three and four tokens' parts of x leave the registers for rows of up to 8192 weights: with longer ones
    // the kernel spills and loses to the tensor core's tiles (four tokens, 4096/14336: 125 us against 73;
    // 2048/5632: 25 us against 32).
    return T >= 1 && T <= 4 && vecs_of(K) <= (T > 2 ? 2 : kRowsMaxVecs) && slots_for(K, gated) > 0;
}

namespace {

template <int T>
cudaError_t launch_rows_for(const RowsArgs& a, int vecs, bool gated, int blocks, int smem, cudaStream_t stream) {
    if (vecs == 1) return launch_rows_at<T, 1>(a, gated, blocks, smem, stream);
    if (vecs == 2) return launch_rows_at<T, 2>(a, gated, blocks, smem, stream);
    if constexpr (T <= 2) {
        if (vecs == 3) return launch_rows_at<T, 3>(a, gated, blocks, smem, stream);
        if (vecs == 4) return launch_rows_at<T, 4>(a, gated, blocks, smem, stream);
        return launch_rows_at<T, 5>(a, gated, blocks, smem, stream);
    }
    return cudaErrorInvalidValue;  // rows_fit
}

}  // namespace

cudaError_t launch_rows(RowsArgs a, bool gated, int num_sms, cudaStream_t stream) {
    const int vecs = vecs_of(a.K), rows = rows_for(vecs, gated);
    a.slots = slots_for(a.K, gated);
    const int groups = a.N / (gated ? rows / 2 : rows), smem = a.slots * rows * a.K * 2;
    const int blocks = std::min(groups, num_sms);
    if (a.T == 1) return launch_rows_for<1>(a, vecs, gated, blocks, smem, stream);
    return a.T == 2 ? launch_rows_for<2>(a, vecs, gated, blocks, smem, stream)
                    : launch_rows_for<4>(a, vecs, gated, blocks, smem, stream);
}

}  // namespace forge
