// Layer norm with X in float and Y in each type.
#include "gmm_norm_kernels.hpp"

namespace gmm {
GMM_NORM_TYPES(float, float)
GMM_NORM_TYPES(float, _Float16)
GMM_NORM_TYPES(float, __bf16)
}
