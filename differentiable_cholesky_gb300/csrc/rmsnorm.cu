// Root-mean-square norm with the residual's addition, and its reverse mode.
//
//   r = x + res,  rstd = 1 / sqrt(sum(r^2) / d + eps),  y = r rstd w
//   n = r rstd,   u = adj_y w
//   adj_in = rstd (u - n mean(u n)) + adj_r,   adj_w = sum over rows of adj_y n
//
// Sums are float32; r is rounded only when it is written, y and the 8-bit
// scales come from the unrounded r.

#include <algorithm>

#include "learn.cuh"
#include "learn.h"

namespace chol {
namespace {

constexpr int kThreads = 256;

enum OutKind { OUT_MODEL, OUT_E4M3, OUT_I8 };

template <int OUT> __device__ __forceinline__ float code_max() { return OUT == OUT_E4M3 ? 448.0f : 127.0f; }
template <int OUT> __device__ __forceinline__ uint8_t to_code8(float x) {
    return OUT == OUT_E4M3 ? to_e4m3(x) : to_i8(x);
}
// The scale of a group whose largest |y| has these bits, and its inverse.  A
// group whose scale would not be a normal number counts as zeros (scale 0),
// since the inverse may overflow.
template <int OUT> __device__ __forceinline__ float scale_of(uint32_t top) {
    const float s = __fmul_rn(__uint_as_float(top), 1.0f / code_max<OUT>());
    return s < 0x1p-126f ? 0.0f : s;
}
__device__ __forceinline__ float inverse_of(float scale) {
    return scale > 0.0f ? __frcp_rn(scale) : 0.0f;
}

// Any d and any alignment: a block goes over its row two or three times (sum
// of squares; for 8-bit output the largest |y|; the output).  r is written in
// the last pass only, since it may replace res.
template <typename T, typename R, int OUT>
__global__ void __launch_bounds__(kThreads) rms_norm_loop_kernel(RmsArgs a) {
    __shared__ float tmp[32];
    __shared__ uint32_t tmp_max[32];
    const T* w = static_cast<const T*>(a.w);
    const int d = (int)a.d, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const R* res = a.res != nullptr ? static_cast<const R*>(a.res) + row * a.ldr : nullptr;
        R* r = a.r != nullptr ? static_cast<R*>(a.r) + row * a.d : nullptr;
        auto sum_at = [&](int j) {
            return res != nullptr ? to_f32(x[j]) + to_f32(res[j]) : to_f32(x[j]);
        };
        float ss = 0.0f;
        for (int j = threadIdx.x; j < d; j += kThreads) {
            const float v = sum_at(j);
            ss = fmaf(v, v, ss);
        }
        __syncthreads();
        ss = block_sum<kThreads>(ss, tmp);
        const float rstd = rsqrtf(ss / (float)d + a.eps);
        if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
        auto y_of = [&](float v, int j) {
            return w != nullptr ? v * rstd * to_f32(w[j]) : v * rstd;
        };
        if constexpr (OUT == OUT_MODEL) {
            T* y = static_cast<T*>(a.y) + row * a.d;
            for (int j = threadIdx.x; j < d; j += kThreads) {
                const float v = sum_at(j);
                y[j] = from_f32<T>(y_of(v, j));
                if (r != nullptr) r[j] = from_f32<R>(v);
            }
        } else {
            uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.d;
            if (a.group == 0) {
                uint32_t top = 0;
                for (int j = threadIdx.x; j < d; j += kThreads)
                    top = max(top, abs_bits(y_of(sum_at(j), j)));
                top = block_max<kThreads>(top, tmp_max);
                const float scale = scale_of<OUT>(top), inv = inverse_of(scale);
                if (threadIdx.x == 0) a.scale[row] = scale;
                for (int j = threadIdx.x; j < d; j += kThreads) {
                    const float v = sum_at(j);
                    y[j] = to_code8<OUT>(y_of(v, j) * inv);
                    if (r != nullptr) r[j] = from_f32<R>(v);
                }
            } else {
                // a warp per group of 128 columns, four columns a lane
                const int groups = (d + 127) / 128;
                for (int g = warp; g < groups; g += kThreads / 32) {
                    float v[4], yv[4];
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = g * 128 + i * 32 + lane;
                        v[i] = j < d ? sum_at(j) : 0.0f;
                        yv[i] = j < d ? y_of(v[i], j) : 0.0f;
                        top = max(top, abs_bits(yv[i]));
                    }
                    const float scale = scale_of<OUT>(warp_max(top)), inv = inverse_of(scale);
                    if (lane == 0) a.scale[row * groups + g] = scale;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = g * 128 + i * 32 + lane;
                        if (j >= d) continue;
                        y[j] = to_code8<OUT>(yv[i] * inv);
                        if (r != nullptr) r[j] = from_f32<R>(v[i]);
                    }
                }
            }
        }
    }
}

// Rows of the adjoint that one partial sum of adj_w covers: few enough
// partial sums that writing and adding them stays small beside the rows.
inline int64_t adj_w_parts(int64_t rows) {
    return std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)device_sm_count() * 2));
}

// One block per part: rows part, part + parts, ...; their adj_y n summed into
// part's row of `work` in row order.
template <typename T, typename R>
__global__ void __launch_bounds__(kThreads) rms_norm_adj_loop_kernel(RmsAdjArgs a) {
    __shared__ float tmp[32];
    const T* w = static_cast<const T*>(a.w);
    const int d = (int)a.d;
    float* part = a.work + (int64_t)blockIdx.x * a.d;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* dy = static_cast<const T*>(a.adj_y) + row * a.ldy;
        const R* r = static_cast<const R*>(a.r) + row * a.ldr;
        const R* dr = a.adj_r != nullptr ? static_cast<const R*>(a.adj_r) + row * a.d : nullptr;
        const float rstd = a.rstd[row];
        float c = 0.0f;
        for (int j = threadIdx.x; j < d; j += kThreads) {
            const float u = w != nullptr ? to_f32(dy[j]) * to_f32(w[j]) : to_f32(dy[j]);
            c = fmaf(u, to_f32(r[j]) * rstd, c);
        }
        __syncthreads();
        c = block_sum<kThreads>(c, tmp) / (float)d;
        for (int j = threadIdx.x; j < d; j += kThreads) {
            const float g = to_f32(dy[j]), n = to_f32(r[j]) * rstd;
            const float u = w != nullptr ? g * to_f32(w[j]) : g;
            float v = rstd * (u - n * c);
            if (dr != nullptr) v += to_f32(dr[j]);
            if (a.adj_in != nullptr) static_cast<R*>(a.adj_in)[row * a.d + j] = from_f32<R>(v);
            if (a.adj_x != nullptr) static_cast<T*>(a.adj_x)[row * a.d + j] = from_f32<T>(v);
            if (a.adj_w != nullptr) part[j] = row == blockIdx.x ? g * n : fmaf(g, n, part[j]);
        }
    }
}

// adj_w[j] = sum over parts, in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
column_sum_kernel(const float* __restrict__ work, int64_t parts, int64_t d, T* __restrict__ out) {
    for (int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x; j < d;
         j += (int64_t)gridDim.x * kThreads) {
        float s = 0.0f;
        for (int64_t p = 0; p < parts; ++p) s += work[p * d + j];
        out[j] = from_f32<T>(s);
    }
}

template <typename T, typename R>
cudaError_t launch_fwd(const RmsArgs& a, int32_t y_dtype, cudaStream_t stream) {
    const unsigned blocks = (unsigned)std::min<int64_t>(a.rows, 1 << 20);
    if (y_dtype == CHOL_E4M3)
        rms_norm_loop_kernel<T, R, OUT_E4M3><<<blocks, kThreads, 0, stream>>>(a);
    else if (y_dtype == CHOL_I8)
        rms_norm_loop_kernel<T, R, OUT_I8><<<blocks, kThreads, 0, stream>>>(a);
    else
        rms_norm_loop_kernel<T, R, OUT_MODEL><<<blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t launch_adj(const RmsAdjArgs& a, cudaStream_t stream) {
    const int64_t parts = adj_w_parts(a.rows);
    const unsigned blocks = (unsigned)parts;
    rms_norm_adj_loop_kernel<T, R><<<blocks, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.adj_w == nullptr) return e;
    const unsigned cols = (unsigned)((a.d + kThreads - 1) / kThreads);
    column_sum_kernel<T><<<cols, kThreads, 0, stream>>>(a.work, parts, a.d,
                                                        static_cast<T*>(a.adj_w));
    return cudaGetLastError();
}

}  // namespace

cudaError_t rms_norm(const RmsArgs& a, int32_t dtype, int32_t res_dtype, int32_t y_dtype,
                     cudaStream_t stream) {
    return model_dispatch(dtype, [&](auto t) {
        using T = typename decltype(t)::type;
        return res_dtype == dtype ? launch_fwd<T, T>(a, y_dtype, stream)
                                  : launch_fwd<T, float>(a, y_dtype, stream);
    });
}

size_t rms_norm_adj_workspace_bytes(int64_t rows, int64_t d) {
    return rows <= 0 ? 0 : (size_t)adj_w_parts(rows) * (size_t)d * sizeof(float);
}

cudaError_t rms_norm_adj(const RmsAdjArgs& a, int32_t dtype, int32_t r_dtype,
                         cudaStream_t stream) {
    return model_dispatch(dtype, [&](auto t) {
        using T = typename decltype(t)::type;
        return r_dtype == dtype ? launch_adj<T, T>(a, stream) : launch_adj<T, float>(a, stream);
    });
}

}  // namespace chol
