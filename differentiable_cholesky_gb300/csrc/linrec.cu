// Gated linear recurrence h_t = a_t h_{t-1} + b_t for every channel, and its
// reverse mode; the kernels are in linrec_kernels.cuh.
//
//   a = g, exp(g) or 1 / (1 + exp(-g));   b = x or (1 - a) x
//   lambda_t = adj_h_t + a_{t+1} lambda_{t+1}
//   adj_a = lambda_t (h_{t-1} - x_t, with b = (1 - a) x),   adj_g = adj_a da/dg
//   adj_x = lambda_t or (1 - a_t) lambda_t,   adj_s0 = a_1 lambda_1

#include <initializer_list>

#include "checks.h"
#include "learn.h"
#include "linrec_kernels.cuh"

namespace chol {

template <> cudaError_t linrec_typed<float, false>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);
template <> cudaError_t linrec_typed<float, true>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);
template <> cudaError_t linrec_typed<__half, false>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);
template <> cudaError_t linrec_typed<__half, true>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);
template <> cudaError_t linrec_typed<__nv_bfloat16, false>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);
template <> cudaError_t linrec_typed<__nv_bfloat16, true>(const LinrecArgs&, int32_t, bool, bool, cudaStream_t);

cudaError_t linrec(const LinrecArgs& a, int32_t dtype, int32_t gate, bool complement, bool adjoint,
                   cudaStream_t stream) {
    return model_dispatch(dtype, [&](auto t) {
        using T = typename decltype(t)::type;
        constexpr int V = 16 / (int)sizeof(T);
        // 16-byte vectors of channels: every row of every array begins on one
        bool vec = a.d % V == 0;
        for (const void* p : {a.g, a.x, (const void*)a.h, a.adj_h, (const void*)a.adj_g,
                              (const void*)a.adj_x})
            vec = vec && (p == nullptr || aligned(p, 16));
        for (int64_t s : {a.g_ts, a.x_ts, a.dh_ts}) vec = vec && (a.time <= 1 || s % V == 0);
        for (int64_t s : {a.g_bs, a.x_bs, a.dh_bs}) vec = vec && (a.batch <= 1 || s % V == 0);
        return adjoint ? linrec_typed<T, true>(a, gate, complement, vec, stream)
                       : linrec_typed<T, false>(a, gate, complement, vec, stream);
    });
}

}  // namespace chol
