// Rotary positions: f32 storage.
#include "rotary.cuh"
namespace mt {
MT_DEFINE_ROTARY(float, f32)
}  // namespace mt

namespace mt {

// dweight[d] = sum over a tensor's rows of partial sums.  A CTA adds 32
// columns: 32 threads wide, kRows rows deep, then the rows in order.
namespace {
constexpr int kRows = 32;
__global__ void __launch_bounds__(32 * kRows)
    rotary_dweight_kernel(const float *partial, int dim, int blocks0,
                          int blocks1, float *dw0, float *dw1) {
    __shared__ float sums[kRows][33];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int per = (dim + 31) / 32;
    const int i = (int)blockIdx.x / per;
    float *dw = i ? dw1 : dw0;
    if (dw == nullptr) return;
    const int d = ((int)blockIdx.x % per) * 32 + (threadIdx.x & 31);
    const int y = threadIdx.x >> 5;
    const int lo = i ? blocks0 : 0, n = i ? blocks1 : blocks0;
    float v = 0.f;
    if (d < dim) {
#pragma unroll 8
        for (int b = y; b < n; b += kRows)
            v += partial[(int64_t)(lo + b) * dim + d];
    }
    sums[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && d < dim) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += sums[r][threadIdx.x & 31];
        dw[d] = s;
    }
}
}  // namespace

cudaError_t launch_rotary_dweight(const float *partial, int dim,
                                  const int32_t blocks[2], float *dw0,
                                  float *dw1, cudaStream_t s) {
    return launch_dependent(rotary_dweight_kernel, 2 * ((dim + 31) / 32),
                            32 * kRows, 0, s, partial, dim, (int)blocks[0],
                            (int)blocks[1], dw0, dw1);
}

}  // namespace mt
