// launch.h -- how kernels that wait for the one before them in the stream are launched.
#pragma once

#include <cuda_runtime.h>

#include "../../include/attn.h"

namespace attn {

// A launch.  `early`: its blocks may start while the kernel before it in the stream still runs (they wait for that
// kernel's end before they touch memory), so that the start of a call, barriers, tensor memory and instructions, overlaps
// the end of the call before: 2.4 -> 2.1 us for a short read, 13.4 -> 13.0 for one token of 32 heads.  Not the wide
// cache kernel, which leaves SMs without blocks when there is little work: its blocks then gather on the SMs that end
// first (4 x 64 tokens over 2000 keys: 33 -> 36 us).
template <typename K, typename... Args>
int launch(K kernel, int grid, int threads, size_t smem, bool early, cudaStream_t st, const Args&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(grid);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = st;
    config.attrs = &attr;
    config.numAttrs = early ? 1 : 0;
    if (cudaLaunchKernelEx(&config, kernel, args...) == cudaSuccess) return ATTN_OK;
    cudaGetLastError();  // reported here, not by a later call
    return ATTN_ERR_LAUNCH;
}

}  // namespace attn
