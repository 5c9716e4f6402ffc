// The linear layer's kernels for _Float16 operands.
#include "gmm_linear_kernels.hpp"

namespace gmm {
GMM_LINEAR_TYPE(_Float16)
template hipError_t launch_dz_range<_Float16>(int, const float*, const float*, int64_t, float*, hipStream_t);
}  // namespace gmm
