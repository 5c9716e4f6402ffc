// The layer of experts' kernels for __bf16 operands.
#include "gmm_experts_kernels.hpp"

namespace gmm {
GMM_EXPERTS_TYPE(__bf16)

}  // namespace gmm
