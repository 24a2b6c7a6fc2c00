// Gated linear recurrence h_t = a_t h_{t-1} + b_t for every channel, and its
// reverse mode.
//
// A run of steps maps the state before it to the state after it by
// h -> A h + H (A the product of its a, H what it gives from zero), and such
// maps compose: the time axis is cut into chunks, each chunk's (A, H) is
// found by itself, the states between chunks follow from them in order, and
// then every chunk is run from its own first state.  The adjoint is the same
// recurrence from the end: with carry_t = a_t lambda_t,
//     lambda_t = adj_h_t + carry_{t+1},   carry_t = a_t adj_h_t + a_t carry_{t+1}.
// Where a sequence begins (or, for the adjoint, ends) the state is replaced
// by the sequence's own, whatever the one before it was.

#include <algorithm>

#include "learn.cuh"
#include "learn.h"

namespace chol {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 64;  // steps

// a and 1 - a of a gate; 1 - a is computed from g, so that it keeps its
// precision where a is close to 1.
template <int GATE> __device__ __forceinline__ float gate_a(float g) {
    if constexpr (GATE == CHOL_GATE_LINEAR) return g;
    else if constexpr (GATE == CHOL_GATE_LOG) return expf(g);
    else return 1.0f / (1.0f + expf(-g));
}
template <int GATE> __device__ __forceinline__ float gate_c(float g) {
    if constexpr (GATE == CHOL_GATE_LINEAR) return 1.0f - g;
    else if constexpr (GATE == CHOL_GATE_LOG) return -expm1f(g);
    else return 1.0f / (1.0f + expf(g));
}

// The sequence that a step belongs to, and its bounds [lo, hi).  Every index
// it gives is below nseq, whatever the offsets hold.
struct Cursor {
    const int64_t* offsets;
    int64_t nseq, s, lo, hi;

    __device__ Cursor(const LinrecArgs& a, int64_t b, int64_t t) {
        offsets = a.offsets;
        nseq = a.nseq;
        if (offsets == nullptr) {
            s = b, lo = 0, hi = a.time;
            return;
        }
        // the last s with offsets[s] <= t
        int64_t x = 0, y = nseq - 1;
        while (x < y) {
            const int64_t m = (x + y + 1) / 2;
            if (offsets[m] <= t) x = m; else y = m - 1;
        }
        s = x, lo = offsets[s], hi = offsets[s + 1];
    }
    __device__ void forward(int64_t t) {
        while (offsets != nullptr && hi <= t && s + 1 < nseq) {
            ++s;
            lo = hi, hi = offsets[s + 1];
        }
    }
    __device__ void backward(int64_t t) {
        while (offsets != nullptr && lo > t && s > 0) {
            --s;
            hi = lo, lo = offsets[s];
        }
    }
};

// (A, H) of chunk blockIdx.y: work[((b * chunks + chunk) * 2 + {0, 1}) * d + c].
// Where the chunk begins a sequence, what came before does not matter: A is
// NaN then, which no product of decays has to be (a decay that is NaN gives
// NaN states either way).
template <typename T, int GATE, bool COMP, bool ADJ>
__global__ void __launch_bounds__(kThreads) linrec_chunk_kernel(LinrecArgs a, float* work) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, chunks = gridDim.y;
    if (c >= a.d) return;
    for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
        const T* g = static_cast<const T*>(a.g) + b * a.g_bs + c;
        const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c;
        const T* dh = static_cast<const T*>(a.adj_h) + b * a.dh_bs + c;
        const int64_t t0 = blockIdx.y * (int64_t)kChunk, t1 = min(t0 + kChunk, a.time);
        float A = 1.0f, H = 0.0f;
        bool cut = false;
        Cursor q(a, b, ADJ ? t1 - 1 : t0);
        for (int64_t i = t0; i < t1; ++i) {
            const int64_t t = ADJ ? t1 - 1 - (i - t0) : i;
            const float gv = to_f32(g[t * a.g_ts]), av = gate_a<GATE>(gv);
            if constexpr (!ADJ) {
                q.forward(t);
                if (t == q.lo) {
                    cut = true;
                    H = a.state0 != nullptr ? a.state0[q.s * a.d + c] : 0.0f;
                }
                const float xv = to_f32(x[t * a.x_ts]);
                H = fmaf(av, H, COMP ? gate_c<GATE>(gv) * xv : xv);
            } else {
                q.backward(t);
                if (t == q.hi - 1) {
                    cut = true;
                    H = a.adj_s1 != nullptr ? a.adj_s1[q.s * a.d + c] : 0.0f;
                }
                H = av * (to_f32(dh[t * a.dh_ts]) + H);
            }
            A *= av;
        }
        float* w = work + ((b * chunks + blockIdx.y) * 2) * a.d + c;
        w[0] = cut ? __int_as_float(0x7fffffff) : A;
        w[a.d] = H;
    }
}

// The state before each chunk (behind it for the adjoint), in place of A.
template <bool ADJ>
__global__ void __launch_bounds__(kThreads)
linrec_carry_kernel(int64_t batch, int64_t chunks, int64_t d, float* work) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= d) return;
    for (int64_t b = blockIdx.y; b < batch; b += gridDim.y) {
        float s = 0.0f;
        for (int64_t i = 0; i < chunks; ++i) {
            float* w = work + ((b * chunks + (ADJ ? chunks - 1 - i : i)) * 2) * d + c;
            const float A = w[0], H = w[d];
            w[0] = s;
            s = isnan(A) ? H : fmaf(A, s, H);
        }
    }
}

// Every step of a chunk, from the state before it.
template <typename T, int GATE, bool COMP, bool ADJ>
__global__ void __launch_bounds__(kThreads) linrec_apply_kernel(LinrecArgs a, const float* work) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, chunks = gridDim.y;
    if (c >= a.d) return;
    for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
        const T* g = static_cast<const T*>(a.g) + b * a.g_bs + c;
        const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c;
        const T* dh = static_cast<const T*>(a.adj_h) + b * a.dh_bs + c;
        T* h = static_cast<T*>(a.h) + b * a.time * a.d + c;
        const int64_t t0 = blockIdx.y * (int64_t)kChunk, t1 = min(t0 + kChunk, a.time);
        float s = work != nullptr ? work[((b * chunks + blockIdx.y) * 2) * a.d + c] : 0.0f;
        Cursor q(a, b, ADJ ? t1 - 1 : t0);
        for (int64_t i = t0; i < t1; ++i) {
            const int64_t t = ADJ ? t1 - 1 - (i - t0) : i;
            const float gv = to_f32(g[t * a.g_ts]), av = gate_a<GATE>(gv);
            if constexpr (!ADJ) {
                q.forward(t);
                if (t == q.lo) s = a.state0 != nullptr ? a.state0[q.s * a.d + c] : 0.0f;
                const float xv = to_f32(x[t * a.x_ts]);
                s = fmaf(av, s, COMP ? gate_c<GATE>(gv) * xv : xv);
                h[t * a.d] = from_f32<T>(s);
                if (t == q.hi - 1 && a.state1 != nullptr) a.state1[q.s * a.d + c] = s;
            } else {
                q.backward(t);
                if (t == q.hi - 1) s = a.adj_s1 != nullptr ? a.adj_s1[q.s * a.d + c] : 0.0f;
                const float lam = to_f32(dh[t * a.dh_ts]) + s;
                float before = 0.0f;
                if (t > q.lo) before = to_f32(h[(t - 1) * a.d]);
                else if (a.state0 != nullptr) before = a.state0[q.s * a.d + c];
                const float cv = gate_c<GATE>(gv);
                const float da = COMP ? lam * (before - to_f32(x[t * a.x_ts])) : lam * before;
                float dg = da;
                if constexpr (GATE == CHOL_GATE_LOG) dg *= av;
                if constexpr (GATE == CHOL_GATE_LOGIT) dg *= av * cv;
                const int64_t o = (b * a.time + t) * a.d + c;
                static_cast<T*>(a.adj_g)[o] = from_f32<T>(dg);
                static_cast<T*>(a.adj_x)[o] = from_f32<T>(COMP ? lam * cv : lam);
                s = av * lam;
                if (t == q.lo && a.adj_s0 != nullptr) a.adj_s0[q.s * a.d + c] = s;
            }
        }
        // empty sequences pass their states through
        if (a.offsets == nullptr || blockIdx.y != 0) continue;
        const float* from = ADJ ? a.adj_s1 : a.state0;
        float* to = ADJ ? a.adj_s0 : a.state1;
        if (to == nullptr) continue;
        for (int64_t k = 0; k < a.nseq; ++k)
            if (a.offsets[k] >= a.offsets[k + 1])
                to[k * a.d + c] = from != nullptr ? from[k * a.d + c] : 0.0f;
    }
}

inline int64_t chunks_of(int64_t time) { return (time + kChunk - 1) / kChunk; }

template <typename T, int GATE, bool COMP, bool ADJ>
cudaError_t launch(const LinrecArgs& a, cudaStream_t stream) {
    const int64_t chunks = chunks_of(a.time);
    const unsigned cb = (unsigned)((a.d + kThreads - 1) / kThreads);
    const unsigned zb = (unsigned)std::min<int64_t>(a.batch, 65535);
    if (chunks > 65535) return cudaErrorInvalidValue;
    float* work = static_cast<float*>(a.work);
    if (a.status != nullptr) {
        const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    if (chunks > 1) {
        linrec_chunk_kernel<T, GATE, COMP, ADJ>
            <<<dim3(cb, (unsigned)chunks, zb), kThreads, 0, stream>>>(a, work);
        linrec_carry_kernel<ADJ>
            <<<dim3(cb, zb), kThreads, 0, stream>>>(a.batch, chunks, a.d, work);
    }
    linrec_apply_kernel<T, GATE, COMP, ADJ>
        <<<dim3(cb, (unsigned)chunks, zb), kThreads, 0, stream>>>(a, chunks > 1 ? work : nullptr);
    return cudaGetLastError();
}

template <typename T, bool COMP, bool ADJ>
cudaError_t by_gate(const LinrecArgs& a, int32_t gate, cudaStream_t stream) {
    switch (gate) {
        case CHOL_GATE_LINEAR: return launch<T, CHOL_GATE_LINEAR, COMP, ADJ>(a, stream);
        case CHOL_GATE_LOG: return launch<T, CHOL_GATE_LOG, COMP, ADJ>(a, stream);
        default: return launch<T, CHOL_GATE_LOGIT, COMP, ADJ>(a, stream);
    }
}

}  // namespace

size_t linrec_workspace_bytes(int64_t batch, int64_t time, int64_t d, int32_t) {
    const int64_t chunks = chunks_of(time);
    return chunks > 1 ? (size_t)batch * chunks * 2 * d * sizeof(float) : 0;
}

cudaError_t linrec(const LinrecArgs& a, int32_t dtype, int32_t gate, bool complement, bool adjoint,
                   cudaStream_t stream) {
    return model_dispatch(dtype, [&](auto t) {
        using T = typename decltype(t)::type;
        if (adjoint)
            return complement ? by_gate<T, true, true>(a, gate, stream)
                              : by_gate<T, false, true>(a, gate, stream);
        return complement ? by_gate<T, true, false>(a, gate, stream)
                          : by_gate<T, false, false>(a, gate, stream);
    });
}

}  // namespace chol
