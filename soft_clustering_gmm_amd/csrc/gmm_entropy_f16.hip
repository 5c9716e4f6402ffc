// The cross entropy's kernels for _Float16 operands.
#include "gmm_entropy_kernels.hpp"

namespace gmm {
GMM_ENTROPY_TYPE(_Float16)
}
