// Kernels of the gated linear recurrence (linrec.cu has the formulas and the
// choice between them).
//
// A run of steps takes the state before it to the state after it by
// s -> A s + H (A the product of the steps' a, H what they give from zero),
// and such maps compose.  linrec_tile_kernel walks a block of channels along
// the whole time axis, a tile of steps at a time:
//   - a thread holds LS consecutive steps of V channels (one 16-byte vector
//     per step) and reduces them to a map; the threads of a warp that hold the
//     same channels scan their maps with shuffles, and the warps' maps meet in
//     shared memory;
//   - a cluster of up to 8 thread blocks takes as many tiles at once: every
//     block sends its tile's map to the others' shared memory, and after one
//     cluster barrier each applies the maps before its own to the state that
//     it carries from tile to tile.  No block waits on global memory, and no
//     other cluster's work is waited for;
//   - the threads run their steps again from the state before them, which is
//     known now, and write.
// So every input is read once, and the next tile's inputs are on their way
// while this one's maps are combined.
//
// Where a packed sequence begins, the state is the sequence's own: a map that
// holds such a step is marked as cut, and what came before it is not used at
// all (not multiplied by zero, which would let a NaN through).
//
// The adjoint is the same recurrence walked from the end, on the carry
// a_t lambda_t:  lambda_t = adj_h_t + carry_{t+1}.
#pragma once

#include "learn.cuh"
#include "learn.h"

namespace chol {
namespace linrec_detail {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// a and c = 1 - a of a gate.  c keeps its relative precision where a is
// close to 1: from the exponential itself for the logistic gate, from a
// polynomial of expm1 (Taylor to g^7, 2^-26 relative at 0.35) for the
// logarithmic one.
template <int GATE> __device__ __forceinline__ void gate(float g, float& a, float& c) {
    if constexpr (GATE == CHOL_GATE_LINEAR) {
        a = g;
        c = 1.0f - g;
    } else if constexpr (GATE == CHOL_GATE_LOG) {
        a = __expf(g);
        float p = 1.0f / 5040.0f;
        p = fmaf(p, g, 1.0f / 720.0f);
        p = fmaf(p, g, 1.0f / 120.0f);
        p = fmaf(p, g, 1.0f / 24.0f);
        p = fmaf(p, g, 1.0f / 6.0f);
        p = fmaf(p, g, 0.5f);
        p = fmaf(p, g, 1.0f);
        c = fabsf(g) < 0.35f ? -p * g : 1.0f - a;
    } else {
        const float e = __expf(-g);  // infinity gives a = 0, c = 1
        a = __frcp_rn(1.0f + e);
        c = e > 1.0f ? 1.0f - a : e * a;
    }
}

// V elements of a row as they lie in memory.
template <typename T, int V> struct Raw {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, bool ok) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (ok) q = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    }
    __device__ __forceinline__ float get(int v) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
        else return to_f32(reinterpret_cast<const T*>(w)[v]);
    }
};
template <typename T> struct Raw<T, 1> {
    T x;
    __device__ __forceinline__ void load(const T* p, bool ok) {
        x = from_f32<T>(0.0f);
        if (ok) x = *p;
    }
    __device__ __forceinline__ float get(int) const { return to_f32(x); }
};

template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        alignas(16) T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = from_f32<T>(v[i]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
    }
}

// V float32 states of channels c .. c + V (rows of d floats, 4-byte aligned).
template <int V> __device__ __forceinline__ void load_state(const float* s, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = s != nullptr ? s[i] : 0.0f;
}
template <int V> __device__ __forceinline__ void store_state(float* s, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = v[i];
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores into the shared memory of block `rank` of the cluster, at the
// address that `p` has here.
__device__ __forceinline__ void put(float2* p, uint32_t rank, float2 v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void put(int* p, uint32_t rank, int v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Steps of a tile that begin or end a sequence, as the tile is walked: the
// sequence's number, else -1.
struct Marks {
    int* enter;
    int* leave;
};

// Marks of the steps [lo, hi) of the time axis, by every thread of the block;
// row_of gives a step's place in the tile.  Any offsets give marks in the tile
// and sequences below nseq.
template <bool ADJ, typename F>
__device__ __forceinline__ void mark(const LinrecArgs& a, int64_t lo, int64_t hi, Marks m, F row_of) {
    // the first j with offsets[j] >= lo
    int64_t x = 0, y = a.nseq + 1;
    while (x < y) {
        const int64_t mid = (x + y) / 2;
        if (a.offsets[mid] < lo) x = mid + 1; else y = mid;
    }
    for (int64_t j = x + threadIdx.x; j <= a.nseq; j += kThreads) {
        const int64_t o = a.offsets[j];
        if (o > hi) break;
        int* first = ADJ ? m.leave : m.enter;
        int* last = ADJ ? m.enter : m.leave;
        if (j < a.nseq && o >= lo && o < hi && a.offsets[j + 1] > o) first[row_of(o)] = (int)j;
        if (j > 0 && o - 1 >= lo && o - 1 < hi && a.offsets[j - 1] < o) last[row_of(o - 1)] = (int)j - 1;
    }
}

// One block of CX * V channels of one row of the batch per cluster; `tiles`
// is the number of tiles that the cluster's blocks share out, `blocks` the
// number of channel blocks of a row.  All blocks of a cluster go through the
// same number of barriers.
template <typename T, int V, int CX, int LS, int GATE, bool ADJ, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2)
linrec_tile_kernel(const LinrecArgs a, const bool comp, const int64_t blocks, const int cs) {
    constexpr int C = CX * V;         // channels
    constexpr int TW = 32 / CX;       // threads of a warp along time
    constexpr int L = kWarps * TW * LS;  // steps of a tile
    __shared__ float2 warp_map[kWarps][C];
    __shared__ float2 tile_map[2][kMaxCluster][C];
    __shared__ __align__(16) float warp_state[kWarps][C];
    __shared__ int warp_cut[kWarps], tile_cut[2][kMaxCluster];
    __shared__ int marks[PACKED ? 2 : 1][2][PACKED ? L : 1];

    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int cx = lane % CX, tw = lane / CX;
    const int row0 = (warp * TW + tw) * LS;
    const uint32_t rank = cs > 1 ? cluster_rank() : 0;
    const int64_t U = a.time;
    const int64_t tiles = (U + L - 1) / L, rounds = (tiles + cs - 1) / cs;
    const int64_t total = a.batch * blocks;
    auto t_of = [&](int64_t u) { return ADJ ? U - 1 - u : u; };
    const float* state_in = ADJ ? a.adj_s1 : a.state0;
    float* state_out = ADJ ? a.adj_s0 : a.state1;

    if (cs > 1) cluster_arrive();  // every block of the cluster has started ...
    if constexpr (PACKED) {
        for (int i = threadIdx.x; i < 2 * L; i += kThreads) (&marks[0][0][0])[i] = -1;
        __syncthreads();
    }
    if (cs > 1) cluster_wait();    // ... before one writes to another
    int buf = 0;
    for (int64_t job = blockIdx.x / cs; job < total; job += gridDim.x / cs) {
        const int64_t b = job / blocks;
        const int64_t c = (job % blocks) * C + cx * V;
        const bool here = c < a.d;
        const T* g = static_cast<const T*>(a.g) + b * a.g_bs + c;
        const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c;
        const T* h_in = static_cast<const T*>(a.h) + b * U * a.d + c;
        const T* dh = static_cast<const T*>(a.adj_h) + b * a.dh_bs + c;
        const bool want_x = !ADJ || comp;

        // the state before the tiles of a round, of one channel per thread
        const int64_t own = (job % blocks) * C + threadIdx.x;
        float running = 0.0f;
        if (!PACKED && threadIdx.x < C && own < a.d && state_in != nullptr)
            running = state_in[b * a.d + own];

        Raw<T, V> rg[LS], rx[LS], rd[ADJ ? LS : 1], rh[ADJ ? LS : 1];
        auto fetch = [&](int64_t tile) {
            const int64_t u0 = tile * L + row0;
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                const int64_t u = u0 + i, t = t_of(u);
                const bool ok = here && u < U;
                rg[i].load(g + t * a.g_ts, ok);
                if constexpr (ADJ) {
                    rd[i].load(dh + t * a.dh_ts, ok);
                    rh[i].load(h_in + (t - 1) * a.d, ok && t > 0);
                }
                rx[i].load(x + t * a.x_ts, ok && want_x);
            }
        };
        fetch(rank);
        for (int64_t round = 0; round < rounds; ++round) {
            const int64_t tile = round * cs + rank;
            const int64_t u0 = tile * L + row0;
            int *enter = nullptr, *leave = nullptr;
            if constexpr (PACKED) {
                enter = marks[buf][0], leave = marks[buf][1];
                const int64_t first = tile * L, last = min(first + L, U);
                if (first < U) {
                    const int64_t lo = ADJ ? t_of(last - 1) : first, hi = ADJ ? t_of(first) + 1 : last;
                    mark<ADJ>(a, lo, hi, {enter, leave}, [&](int64_t t) { return (int)(t_of(t) - first); });
                }
                __syncthreads();
                // the other buffer is for the next tile; its readers are all past it
                for (int i = threadIdx.x; i < 2 * L; i += kThreads) marks[buf ^ 1][i / L][i % L] = -1;
            }
            // a thread's steps to one map; a and what the steps add are kept
            float av[LS][V], bv[LS][V], A[V], H[V];
            bool cut = false;
#pragma unroll
            for (int v = 0; v < V; ++v) A[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                const bool in = u0 + i < U;
                if constexpr (PACKED) {
                    const int s = enter[row0 + i];
                    if (s >= 0) {
                        cut = true;
                        load_state<V>(state_in != nullptr && here ? state_in + s * a.d + c : nullptr, H);
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float cv;
                    gate<GATE>(rg[i].get(v), av[i][v], cv);
                    if constexpr (!ADJ) {
                        const float xv = rx[i].get(v);
                        bv[i][v] = comp ? cv * xv : xv;
                    } else {
                        bv[i][v] = rd[i].get(v);
                    }
                    if (!in) av[i][v] = 1.0f, bv[i][v] = 0.0f;
                    H[v] = ADJ ? av[i][v] * (bv[i][v] + H[v]) : fmaf(av[i][v], H[v], bv[i][v]);
                    A[v] *= av[i][v];
                }
            }
            // what the adjoint's second pass needs beside a and adj_h
            Raw<T, V> kg[ADJ ? LS : 1], kx[ADJ ? LS : 1], kh[ADJ ? LS : 1];
            if constexpr (ADJ) {
#pragma unroll
                for (int i = 0; i < LS; ++i) kg[i] = rg[i], kx[i] = rx[i], kh[i] = rh[i];
            }
            if (round + 1 < rounds) fetch(tile + cs);

            // maps of all steps of the warp up to and with this thread's
            int cuts = cut;
#pragma unroll
            for (int o = 1; o < TW; o *= 2) {
                const int pc = PACKED ? __shfl_up_sync(0xffffffffu, cuts, o * CX) : 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float pa = __shfl_up_sync(0xffffffffu, A[v], o * CX);
                    const float ph = __shfl_up_sync(0xffffffffu, H[v], o * CX);
                    if (tw >= o && !(PACKED && cuts)) {
                        H[v] = fmaf(A[v], ph, H[v]);
                        A[v] *= pa;
                    }
                }
                if (PACKED && tw >= o) cuts |= pc;
            }
            if (tw == TW - 1) {
#pragma unroll
                for (int v = 0; v < V; ++v) warp_map[warp][cx * V + v] = make_float2(A[v], H[v]);
                if (PACKED && cx == 0) warp_cut[warp] = cuts;
            }
            // of the steps before this thread's
            if constexpr (TW > 1) {
                const int pc = PACKED ? __shfl_up_sync(0xffffffffu, cuts, CX) : 0;
                cuts = tw > 0 ? pc : 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float pa = __shfl_up_sync(0xffffffffu, A[v], CX);
                    const float ph = __shfl_up_sync(0xffffffffu, H[v], CX);
                    A[v] = tw > 0 ? pa : 1.0f;
                    H[v] = tw > 0 ? ph : 0.0f;
                }
            } else {
                cuts = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) A[v] = 1.0f, H[v] = 0.0f;
            }
            __syncthreads();
            float s = running;
            if (cs > 1) {
                if (threadIdx.x < C) {
                    float ma = 1.0f, mh = 0.0f;
                    int mc = 0;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 m = warp_map[w][threadIdx.x];
                        if (PACKED && warp_cut[w]) {
                            ma = m.x, mh = m.y, mc = 1;
                        } else {
                            mh = fmaf(m.x, mh, m.y);
                            ma *= m.x;
                        }
                    }
                    for (int r = 0; r < cs; ++r) {
                        put(&tile_map[buf][rank][threadIdx.x], r, make_float2(ma, mh));
                        if (PACKED && threadIdx.x == 0) put(&tile_cut[buf][rank], r, mc);
                    }
                }
                cluster_arrive();
                cluster_wait();
                if (threadIdx.x < C) {
                    for (int r = 0; r < cs; ++r) {
                        if (r == (int)rank) s = running;
                        const float2 m = tile_map[buf][r][threadIdx.x];
                        running = PACKED && tile_cut[buf][r] ? m.y : fmaf(m.x, running, m.y);
                    }
                }
            }
            if (threadIdx.x < C) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    warp_state[w][threadIdx.x] = s;
                    const float2 m = warp_map[w][threadIdx.x];
                    s = PACKED && warp_cut[w] ? m.y : fmaf(m.x, s, m.y);
                }
                if (cs == 1) running = s;
            }
            __syncthreads();
            // the steps again, from the state before them
            float st[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                st[v] = warp_state[warp][cx * V + v];
                st[v] = PACKED && cuts ? H[v] : fmaf(A[v], st[v], H[v]);
            }
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                const int64_t u = u0 + i, t = t_of(u);
                if (!here || u >= U) break;
                int64_t leaving = -1;
                if constexpr (PACKED) {
                    const int e = enter[row0 + i];
                    if (e >= 0) load_state<V>(state_in != nullptr ? state_in + e * a.d + c : nullptr, st);
                    leaving = leave[row0 + i];
                } else {
                    if (u == U - 1) leaving = b;
                }
                const int64_t o = (b * U + t) * a.d + c;
                if constexpr (!ADJ) {
#pragma unroll
                    for (int v = 0; v < V; ++v) st[v] = fmaf(av[i][v], st[v], bv[i][v]);
                    store<T, V>(static_cast<T*>(a.h) + o, st);
                } else {
                    float before[V], dg[V], dx[V];
                    if (leaving >= 0) {
                        load_state<V>(a.state0 != nullptr ? a.state0 + leaving * a.d + c : nullptr, before);
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v) before[v] = kh[i].get(v);
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float a2, cv;
                        gate<GATE>(kg[i].get(v), a2, cv);
                        const float lam = bv[i][v] + st[v];
                        dx[v] = comp ? lam * cv : lam;
                        float da = lam * (comp ? before[v] - kx[i].get(v) : before[v]);
                        if constexpr (GATE == CHOL_GATE_LOG) da *= a2;
                        if constexpr (GATE == CHOL_GATE_LOGIT) da *= a2 * cv;
                        dg[v] = da;
                        st[v] = av[i][v] * lam;
                    }
                    store<T, V>(static_cast<T*>(a.adj_g) + o, dg);
                    store<T, V>(static_cast<T*>(a.adj_x) + o, dx);
                }
                if (leaving >= 0 && state_out != nullptr) store_state<V>(state_out + leaving * a.d + c, st);
            }
            buf ^= 1;
        }
        if constexpr (PACKED) {
            // empty sequences pass their states through
            if (rank == 0 && here && state_out != nullptr)
                for (int64_t s = warp * TW + tw; s < a.nseq; s += kWarps * TW) {
                    if (a.offsets[s] < a.offsets[s + 1]) continue;
                    float st[V];
                    load_state<V>(state_in != nullptr ? state_in + s * a.d + c : nullptr, st);
                    store_state<V>(state_out + s * a.d + c, st);
                }
        }
    }
}

// A few steps (one, in serving): a thread walks V channels by itself.
template <typename T, int V, int GATE, bool ADJ>
__global__ void __launch_bounds__(128)
linrec_step_kernel(const LinrecArgs a, const bool comp) {
    const int64_t vecs = (a.d + V - 1) / V, total = a.batch * vecs;
    for (int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 128) {
        const int64_t b = i / vecs, c = (i % vecs) * V, U = a.time;
        const T* g = static_cast<const T*>(a.g) + b * a.g_bs + c;
        const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c;
        float st[V];
        const float* from = ADJ ? a.adj_s1 : a.state0;
        float* to = ADJ ? a.adj_s0 : a.state1;
        load_state<V>(from != nullptr ? from + b * a.d + c : nullptr, st);
        for (int64_t u = 0; u < U; ++u) {
            const int64_t t = ADJ ? U - 1 - u : u, o = (b * U + t) * a.d + c;
            Raw<T, V> rg, rx;
            rg.load(g + t * a.g_ts, true);
            rx.load(x + t * a.x_ts, !ADJ || comp);
            if constexpr (!ADJ) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float av, cv;
                    gate<GATE>(rg.get(v), av, cv);
                    st[v] = fmaf(av, st[v], comp ? cv * rx.get(v) : rx.get(v));
                }
                store<T, V>(static_cast<T*>(a.h) + o, st);
            } else {
                Raw<T, V> rd, rh;
                rd.load(static_cast<const T*>(a.adj_h) + b * a.dh_bs + t * a.dh_ts + c, true);
                rh.load(static_cast<const T*>(a.h) + o - a.d, t > 0);
                float before[V], dg[V], dx[V];
                if (t > 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v) before[v] = rh.get(v);
                } else {
                    load_state<V>(a.state0 != nullptr ? a.state0 + b * a.d + c : nullptr, before);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float av, cv;
                    gate<GATE>(rg.get(v), av, cv);
                    const float lam = rd.get(v) + st[v];
                    dx[v] = comp ? lam * cv : lam;
                    float da = lam * (comp ? before[v] - rx.get(v) : before[v]);
                    if constexpr (GATE == CHOL_GATE_LOG) da *= av;
                    if constexpr (GATE == CHOL_GATE_LOGIT) da *= av * cv;
                    dg[v] = da;
                    st[v] = av * lam;
                }
                store<T, V>(static_cast<T*>(a.adj_g) + o, dg);
                store<T, V>(static_cast<T*>(a.adj_x) + o, dx);
            }
        }
        if (to != nullptr) store_state<V>(to + b * a.d + c, st);
    }
}

// Channel blocks of `C` channels, and the cluster that shares out their tiles
// of `L` steps: doubled while the thread blocks would still all run at once
// (two on each SM) and there are tiles for them.
struct Grid {
    int64_t blocks;
    int cs;
    unsigned grid;
};
inline Grid grid_of(const LinrecArgs& a, int C, int L) {
    Grid q;
    q.blocks = (a.d + C - 1) / C;
    const int64_t total = a.batch * q.blocks, slots = 2 * (int64_t)device_sm_count();
    const int64_t tiles = (a.time + L - 1) / L;
    q.cs = 1;
    while (q.cs < kMaxCluster && total * q.cs * 2 <= slots && q.cs < tiles) q.cs *= 2;
    q.grid = (unsigned)(std::min<int64_t>(total, 1 << 24) * q.cs);
    return q;
}

template <typename T, int V, int CX, int LS, int GATE, bool ADJ, bool PACKED>
cudaError_t launch_tile(const LinrecArgs& a, bool comp, cudaStream_t stream) {
    const Grid q = grid_of(a, CX * V, kThreads / CX * LS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(q.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = q.cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = q.cs > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linrec_tile_kernel<T, V, CX, LS, GATE, ADJ, PACKED>, a, comp,
                              q.blocks, q.cs);
}

template <typename T, int V, int CX, int LS, int GATE, bool ADJ>
cudaError_t launch_any(const LinrecArgs& a, bool comp, cudaStream_t stream) {
    return a.offsets != nullptr ? launch_tile<T, V, CX, LS, GATE, ADJ, true>(a, comp, stream)
                                : launch_tile<T, V, CX, LS, GATE, ADJ, false>(a, comp, stream);
}

// Steps that a thread walks by itself: up to here the chain of dependent
// steps is shorter than a tile's synchronisation.
constexpr int64_t kFewSteps = 8;

template <typename T, int GATE, bool ADJ>
cudaError_t launch(const LinrecArgs& a, bool comp, bool vec, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T), LS = ADJ ? 2 : 4;
    if (a.time <= kFewSteps && a.offsets == nullptr) {
        const int64_t total = a.batch * ((a.d + (vec ? V : 1) - 1) / (vec ? V : 1));
        const unsigned grid = (unsigned)std::min<int64_t>((total + 127) / 128, 1 << 24);
        if (vec) linrec_step_kernel<T, V, GATE, ADJ><<<grid, 128, 0, stream>>>(a, comp);
        else linrec_step_kernel<T, 1, GATE, ADJ><<<grid, 128, 0, stream>>>(a, comp);
        return cudaGetLastError();
    }
    if (!vec) return launch_any<T, 1, 32, LS * 2, GATE, ADJ>(a, comp, stream);
    // 128-byte rows of a channel block; 32-byte ones, and longer tiles, where
    // the wider blocks would leave most SMs idle
    if (a.batch * ((a.d + 8 * V - 1) / (8 * V)) * kMaxCluster < device_sm_count() &&
        a.time > kThreads / 8 * LS * kMaxCluster)
        return launch_any<T, V, 2, LS, GATE, ADJ>(a, comp, stream);
    return launch_any<T, V, 8, LS, GATE, ADJ>(a, comp, stream);
}

}  // namespace linrec_detail

// One element type and direction (linrec_<type>_<direction>.cu).
template <typename T, bool ADJ>
cudaError_t linrec_typed(const LinrecArgs& a, int32_t gate, bool comp, bool vec, cudaStream_t stream);

#define CHOL_LINREC(T, ADJ)                                                                       \
    template <>                                                                                   \
    cudaError_t linrec_typed<T, ADJ>(const LinrecArgs& a, int32_t gate, bool comp, bool vec,      \
                                     cudaStream_t stream) {                                       \
        switch (gate) {                                                                           \
            case CHOL_GATE_LINEAR:                                                                \
                return linrec_detail::launch<T, CHOL_GATE_LINEAR, ADJ>(a, comp, vec, stream);     \
            case CHOL_GATE_LOG:                                                                   \
                return linrec_detail::launch<T, CHOL_GATE_LOG, ADJ>(a, comp, vec, stream);        \
            default:                                                                              \
                return linrec_detail::launch<T, CHOL_GATE_LOGIT, ADJ>(a, comp, vec, stream);      \
        }                                                                                         \
    }

}  // namespace chol
