// Layer norm with X and Y in this type.
#include "gmm_norm_kernels.hpp"

namespace gmm {
GMM_NORM_TYPES(_Float16, _Float16)
}
