// Forward kernels of the gated linear recurrence for __half elements.
#include "linrec_kernels.cuh"

namespace chol {

CHOL_LINREC(__half, false)

}  // namespace chol
