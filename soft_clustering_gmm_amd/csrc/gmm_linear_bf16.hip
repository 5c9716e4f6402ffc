// The linear layer's kernels for __bf16 operands.
#include "gmm_linear_kernels.hpp"

namespace gmm {
GMM_LINEAR_TYPE(__bf16)
}  // namespace gmm
