// mt_decoder.cuh -- what the kernels of the decoder's row operators share
// (rotary positions, quantised cache, logits); their C entry points are in
// decoder.cpp.
#pragma once

#include "mt_kernels.cuh"
#include "mt_decoder_internal.h"

namespace mt {

// A launch as a programmatic dependent of the previous kernel on the stream:
// the kernel may start while that one finishes and waits for it
// (grid_wait_prerequisites) before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int64_t grid, int threads,
                             size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mt
