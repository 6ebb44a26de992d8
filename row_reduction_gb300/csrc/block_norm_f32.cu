// Norms around a block: f32 storage.
#include "block_norm.cuh"
namespace mt {
MT_DEFINE_BLOCK_NORM(float, f32)
}  // namespace mt

namespace mt {

// A weight's gradient: the sum of the CTAs' partial sums of a column.  A CTA
// adds 32 columns: 32 threads wide, kRows rows deep, then the rows in order.
namespace {
constexpr int kRows = 32;
__global__ void __launch_bounds__(32 * kRows)
    norm_sums_kernel(const float *partial, int cols, int blocks, float *d0,
                     float *d1, float *d2) {
    __shared__ float sums[kRows][33];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int k = (int)blockIdx.y;
    float *d = k == 0 ? d0 : k == 1 ? d1 : d2;
    if (d == nullptr) return;
    const int i = (int)blockIdx.x * 32 + (threadIdx.x & 31);
    const int y = threadIdx.x >> 5;
    float v = 0.f;
    if (i < cols) {
#pragma unroll 8
        for (int b = y; b < blocks; b += kRows)
            v += partial[((int64_t)b * 3 + k) * cols + i];
    }
    sums[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && i < cols) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += sums[r][threadIdx.x & 31];
        d[i] = s;
    }
}
}  // namespace

cudaError_t launch_norm_sums(const float *partial, int cols, int blocks,
                             float *d0, float *d1, float *d2,
                             cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + 31) / 32), 3);
    cfg.blockDim = dim3(32 * kRows);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_sums_kernel, partial, cols, blocks,
                              d0, d1, d2);
}

}  // namespace mt
