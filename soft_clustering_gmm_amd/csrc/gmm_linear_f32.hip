// The linear layer's kernels for float operands.
#include "gmm_linear_kernels.hpp"

namespace gmm {
GMM_LINEAR_TYPE(float)
}  // namespace gmm
