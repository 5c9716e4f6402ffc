// The cross entropy's kernels for __bf16 operands.
#include "gmm_entropy_kernels.hpp"

namespace gmm {
GMM_ENTROPY_TYPE(__bf16)
}
