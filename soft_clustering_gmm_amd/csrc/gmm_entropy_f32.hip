// The cross entropy's kernels for float operands.
#include "gmm_entropy_kernels.hpp"

namespace gmm {
GMM_ENTROPY_TYPE(float)
}
