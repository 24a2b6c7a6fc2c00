// Adjoint kernels of the gated linear recurrence for __nv_bfloat16 elements.
#include "linrec_kernels.cuh"

namespace chol {

CHOL_LINREC(__nv_bfloat16, true)

}  // namespace chol
