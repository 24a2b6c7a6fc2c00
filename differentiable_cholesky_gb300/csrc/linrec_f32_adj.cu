// Adjoint kernels of the gated linear recurrence for float elements.
#include "linrec_kernels.cuh"

namespace chol {

CHOL_LINREC(float, true)

}  // namespace chol
