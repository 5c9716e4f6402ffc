// The linear layer's kernels for _Float16 operands.
#include "gmm_linear_kernels.hpp"

namespace gmm {
GMM_LINEAR_TYPE(_Float16)
}  // namespace gmm
