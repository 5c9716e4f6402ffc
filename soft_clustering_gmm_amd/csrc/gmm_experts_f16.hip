// The layer of experts' kernels for _Float16 operands.
#include "gmm_experts_kernels.hpp"

namespace gmm {
GMM_EXPERTS_TYPE(_Float16)

}  // namespace gmm
