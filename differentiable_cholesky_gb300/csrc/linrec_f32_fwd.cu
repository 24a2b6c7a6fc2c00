// Forward kernels of the gated linear recurrence for float elements.
#include "linrec_kernels.cuh"

namespace chol {

CHOL_LINREC(float, false)

}  // namespace chol
