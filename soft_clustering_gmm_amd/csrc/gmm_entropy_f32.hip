// The cross entropy's kernels for float operands, and those without a type.
#include "gmm_entropy_kernels.hpp"

namespace gmm {

GMM_ENTROPY_TYPE(float)

__global__ void __launch_bounds__(256) entropy_fold_kernel(const float* parts, int64_t count, int64_t rows, int V,
                                                           float* out, int across) {
  __shared__ float red[4][64];
  const int group = blockIdx.x / across, t = threadIdx.x % 64, slice = threadIdx.x / 64;
  const int col = (blockIdx.x % across) * 64 + t;
  const int64_t r1 = min(count, (group + 1) * rows);
  float sum = 0.f;
  if (col < V)
#pragma unroll 8
    for (int64_t r = group * rows + slice; r < r1; r += 4) sum += parts[r * V + col];
  red[slice][t] = sum;
  __syncthreads();
  if (slice == 0 && col < V) out[group * (int64_t)V + col] = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
}

hipError_t launch_entropy_fold(const float* parts, int64_t count, int64_t most, int V, float* out, hipStream_t s) {
  const int64_t rows = fold_rows(count, most);
  const int across = (V + 63) / 64;
  entropy_fold_kernel<<<(unsigned)(across * ((count + rows - 1) / rows)), 256, 0, s>>>(parts, count, rows, V, out, across);
  return hipGetLastError();
}

}  // namespace gmm
