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
//     block sends its tile's map to the others' shared memory, where an
//     mbarrier counts the bytes, and each applies the maps before its own to
//     the state that it carries from round to round.  No block waits on global
//     memory, nor on another cluster (the wait has a limit all the same; past
//     it the states become NaN);
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
#ifndef CHOL_LR_V
#define CHOL_LR_V V
#define CHOL_LR_CX 8
#define CHOL_LR_LSF 4
#define CHOL_LR_LSA 2
#define CHOL_LR_OCC 2
#endif

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
        a = exp2_fast(g * 1.44269504f);
        float p = 1.0f / 5040.0f;
        p = fmaf(p, g, 1.0f / 720.0f);
        p = fmaf(p, g, 1.0f / 120.0f);
        p = fmaf(p, g, 1.0f / 24.0f);
        p = fmaf(p, g, 1.0f / 6.0f);
        p = fmaf(p, g, 0.5f);
        p = fmaf(p, g, 1.0f);
        c = fabsf(g) < 0.35f ? -p * g : 1.0f - a;
    } else {
        const float e = exp2_fast(g * -1.44269504f);  // infinity gives a = 0, c = 1
        a = rcp_fast(1.0f + e);
        c = e > 1.0f ? 1.0f - a : e * a;
    }
}

// V elements of a row as they lie in memory: 8 or 16 bytes.
template <typename T, int V> struct Raw {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, bool ok) {
        if constexpr (kWords == 4) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (ok) q = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            uint2 q = make_uint2(0, 0);
            if (ok) q = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = q.x, w[1] = q.y;
        }
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
            else unpack2<T>(w[i], f[2 * i], f[2 * i + 1]);
        }
    }
};
template <typename T> struct Raw<T, 1> {
    T x;
    __device__ __forceinline__ void load(const T* p, bool ok) {
        x = from_f32<T>(0.0f);
        if (ok) x = __ldg(p);
    }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(x); }
};

template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        uint32_t w[V * sizeof(T) / 4];
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(T) / 4); ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
            else w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        }
        if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
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
// All blocks of the cluster have come here (memory is not ordered by it).
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Stores into the shared memory of block `rank` of the cluster, at the
// addresses that `p` and `bar` have here: the bytes are counted on `bar` when
// they are there.  No fence is needed, so the tile before may still be on
// its way to memory.
__device__ __forceinline__ void send(float2* p, uint64_t* bar, uint32_t rank, float2 v) {
    uint32_t at, on;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(on) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::
                     "r"(at), "f"(v.x), "f"(v.y), "r"(on)
                 : "memory");
}
__device__ __forceinline__ void send(int* p, uint64_t* bar, uint32_t rank, int v) {
    uint32_t at, on;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(on) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::
                     "r"(at), "r"(v), "r"(on)
                 : "memory");
}

// Waits for a phase of `bar` and for what was sent with it; gives up (false)
// after a number of polls.
__device__ __forceinline__ bool wait_maps(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 18); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
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
__global__ void __launch_bounds__(kThreads, CHOL_LR_OCC)
linrec_tile_kernel(const LinrecArgs a, const bool comp, const int64_t blocks, const int cs) {
    constexpr int C = CX * V;         // channels
    constexpr int TW = 32 / CX;       // threads of a warp along time
    constexpr int L = kWarps * TW * LS;  // steps of a tile
    __shared__ float2 warp_map[kWarps][C];
    __shared__ float2 tile_map[2][kMaxCluster][C];
    __shared__ __align__(16) float warp_state[kWarps][C];
    __shared__ int warp_cut[kWarps], tile_cut[2][kMaxCluster];
    __shared__ int marks[PACKED ? 2 : 1][2][PACKED ? L : 1];
    __shared__ uint64_t arrived[2];  // the maps of a round, by its parity

    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int cx = lane % CX, tw = lane / CX;
    const int row0 = (warp * TW + tw) * LS;
    const uint32_t rank = cs > 1 ? cluster_rank() : 0;
    const int64_t U = a.time;
    const int64_t tiles = (U + L - 1) / L, rounds = (tiles + cs - 1) / cs;
    const int64_t total = a.batch * blocks;
    const int64_t round_steps = (int64_t)cs * L;
    const float* state_in = ADJ ? a.adj_s1 : a.state0;
    float* state_out = ADJ ? a.adj_s0 : a.state1;
    // a step later, as the axis is walked, in elements of each array
    const int64_t sg = ADJ ? -a.g_ts : a.g_ts, sx = ADJ ? -a.x_ts : a.x_ts, sd = -a.dh_ts;
    const int64_t so = ADJ ? -a.d : a.d;

    if constexpr (PACKED) {
        for (int i = threadIdx.x; i < 2 * L; i += kThreads) (&marks[0][0][0])[i] = -1;
    }
    if (threadIdx.x == 0) {
        mbar_init(&arrived[0], 1);
        mbar_init(&arrived[1], 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (cs > 1) cluster_meet();  // before one block writes to another
    const uint32_t round_bytes = (uint32_t)cs * (C * (uint32_t)sizeof(float2) + (PACKED ? 4u : 0u));
    int buf = 0;
    uint32_t parity = 0;   // of the round's wait: changes every second round
    bool lost = false;     // a wait ran out: the states are NaN from there on
    for (int64_t job = blockIdx.x / cs; job < total; job += gridDim.x / cs) {
        const int64_t b = job / blocks;
        const int64_t c = (job % blocks) * C + cx * V;
        const bool here = c < a.d;
        // this thread's first step of the tile that is fetched next
        int64_t u0 = (int64_t)rank * L + row0;
        const int64_t t0 = ADJ ? U - 1 - u0 : u0;
        const T* g = static_cast<const T*>(a.g) + b * a.g_bs + c + t0 * a.g_ts;
        const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c + t0 * a.x_ts;
        const T* dh = ADJ ? static_cast<const T*>(a.adj_h) + b * a.dh_bs + c + t0 * a.dh_ts : nullptr;
        int64_t o = (b * U + t0) * a.d + c;  // of the contiguous arrays
        const T* h_before = ADJ ? static_cast<const T*>(a.h) + o - a.d : nullptr;
        const bool want_x = !ADJ || comp;

        // the state before the tiles of a round, of one channel per thread
        const int64_t own = (job % blocks) * C + threadIdx.x;
        float running = 0.0f;
        if (!PACKED && threadIdx.x < C && own < a.d && state_in != nullptr)
            running = state_in[b * a.d + own];

        // Steps of this thread that there are, of a tile whose first is u.
        // The others, all behind the last, are fetched as zeros and give
        // states that nothing reads.
        auto steps_at = [&](int64_t u) {
            return here ? (int)max((int64_t)0, min((int64_t)LS, U - u)) : 0;
        };
        Raw<T, V> rg[LS], rx[LS], rd[ADJ ? LS : 1], rh[ADJ ? LS : 1];
        auto fetch = [&](int64_t u) {
            const int n = steps_at(u);
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                rg[i].load(g + i * sg, i < n);
                if constexpr (ADJ) {
                    rd[i].load(dh + i * sd, i < n);
                    rh[i].load(h_before + i * so, i < n && u + i < U - 1);
                }
                rx[i].load(x + i * sx, i < n && want_x);
            }
            g += round_steps * sg;
            x += round_steps * sx;
            if constexpr (ADJ) dh += round_steps * sd, h_before += round_steps * so;
        };
        fetch(u0);
        for (int64_t round = 0; round < rounds; ++round, u0 += round_steps, o += round_steps * so) {
            int *enter = nullptr, *leave = nullptr;
            if constexpr (PACKED) {
                enter = marks[buf][0], leave = marks[buf][1];
                const int64_t first = u0 - row0, last = min(first + L, U);
                if (first < U) {
                    const int64_t lo = ADJ ? U - last : first, hi = ADJ ? U - first : last;
                    mark<ADJ>(a, lo, hi, {enter, leave},
                              [&](int64_t t) { return (int)((ADJ ? U - 1 - t : t) - first); });
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
                if constexpr (PACKED) {
                    const int s = enter[row0 + i];
                    if (s >= 0) {
                        cut = true;
                        load_state<V>(state_in != nullptr && here ? state_in + s * a.d + c : nullptr, H);
                    }
                }
                float gv[V];
                rg[i].get(gv);
                if constexpr (ADJ) rd[i].get(bv[i]); else rx[i].get(bv[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float cv;
                    gate<GATE>(gv[v], av[i][v], cv);
                    if (!ADJ && comp) bv[i][v] *= cv;
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
            if (round + 1 < rounds) fetch(u0 + round_steps);

            // maps of all steps of the warp up to and with this thread's
            int cuts = cut;
#pragma unroll
            for (int k = 1; k < TW; k *= 2) {
                const int pc = PACKED ? __shfl_up_sync(0xffffffffu, cuts, k * CX) : 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float pa = __shfl_up_sync(0xffffffffu, A[v], k * CX);
                    const float ph = __shfl_up_sync(0xffffffffu, H[v], k * CX);
                    if (tw >= k && !(PACKED && cuts)) {
                        H[v] = fmaf(A[v], ph, H[v]);
                        A[v] *= pa;
                    }
                }
                if (PACKED && tw >= k) cuts |= pc;
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
                    if (threadIdx.x == 0) mbar_arrive_expect_tx(&arrived[buf], round_bytes);
                    for (int r = 0; r < cs; ++r) {
                        send(&tile_map[buf][rank][threadIdx.x], &arrived[buf], r, make_float2(ma, mh));
                        if (PACKED && threadIdx.x == 0) send(&tile_cut[buf][rank], &arrived[buf], r, mc);
                    }
                    // A block sends the maps of the round after next only when it
                    // has this block's of the next, so a buffer is never
                    // overwritten while it is read.
                    lost = lost || !wait_maps(&arrived[buf], parity);
                    for (int r = 0; r < cs; ++r) {
                        if (r == (int)rank) s = running;
                        const float2 m = tile_map[buf][r][threadIdx.x];
                        running = PACKED && tile_cut[buf][r] ? m.y : fmaf(m.x, running, m.y);
                    }
                    if (lost) s = running = __int_as_float(0x7fffffff);
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
            const int n = steps_at(u0);
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                if (i >= n) break;
                int64_t leaving = -1;
                if constexpr (PACKED) {
                    const int e = enter[row0 + i];
                    if (e >= 0) load_state<V>(state_in != nullptr ? state_in + e * a.d + c : nullptr, st);
                    leaving = leave[row0 + i];
                } else {
                    if (u0 + i == U - 1) leaving = b;
                }
                const int64_t at = o + i * so;
                if constexpr (!ADJ) {
#pragma unroll
                    for (int v = 0; v < V; ++v) st[v] = fmaf(av[i][v], st[v], bv[i][v]);
                    store<T, V>(static_cast<T*>(a.h) + at, st);
                } else {
                    float before[V], gv[V], xv[V], dg[V], dx[V];
                    kg[i].get(gv);
                    kx[i].get(xv);
                    kh[i].get(before);
                    if (leaving >= 0)
                        load_state<V>(a.state0 != nullptr ? a.state0 + leaving * a.d + c : nullptr, before);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float a2, cv;
                        gate<GATE>(gv[v], a2, cv);
                        const float lam = bv[i][v] + st[v];
                        dx[v] = comp ? lam * cv : lam;
                        float da = lam * (comp ? before[v] - xv[v] : before[v]);
                        if constexpr (GATE == CHOL_GATE_LOG) da *= a2;
                        if constexpr (GATE == CHOL_GATE_LOGIT) da *= a2 * cv;
                        dg[v] = da;
                        st[v] = av[i][v] * lam;
                    }
                    store<T, V>(static_cast<T*>(a.adj_g) + at, dg);
                    store<T, V>(static_cast<T*>(a.adj_x) + at, dx);
                }
                if (leaving >= 0 && state_out != nullptr) store_state<V>(state_out + leaving * a.d + c, st);
            }
            parity ^= (uint32_t)buf;
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
    if (cs > 1) cluster_meet();  // no block leaves while another may write to it
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
            float gv[V], xv[V], av[V], cv[V];
            rg.get(gv);
            rx.get(xv);
#pragma unroll
            for (int v = 0; v < V; ++v) gate<GATE>(gv[v], av[v], cv[v]);
            if constexpr (!ADJ) {
#pragma unroll
                for (int v = 0; v < V; ++v) st[v] = fmaf(av[v], st[v], comp ? cv[v] * xv[v] : xv[v]);
                store<T, V>(static_cast<T*>(a.h) + o, st);
            } else {
                Raw<T, V> rd, rh;
                rd.load(static_cast<const T*>(a.adj_h) + b * a.dh_bs + t * a.dh_ts + c, true);
                rh.load(static_cast<const T*>(a.h) + o - a.d, t > 0);
                float before[V], dhv[V], dg[V], dx[V];
                rd.get(dhv);
                rh.get(before);
                if (t == 0) load_state<V>(a.state0 != nullptr ? a.state0 + b * a.d + c : nullptr, before);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float lam = dhv[v] + st[v];
                    dx[v] = comp ? lam * cv[v] : lam;
                    float da = lam * (comp ? before[v] - xv[v] : before[v]);
                    if constexpr (GATE == CHOL_GATE_LOG) da *= av[v];
                    if constexpr (GATE == CHOL_GATE_LOGIT) da *= av[v] * cv[v];
                    dg[v] = da;
                    st[v] = av[v] * lam;
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
    const int64_t total = a.batch * q.blocks, slots = CHOL_LR_OCC * (int64_t)device_sm_count();
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
    return launch_any<T, CHOL_LR_V, CHOL_LR_CX, ADJ ? CHOL_LR_LSA : CHOL_LR_LSF, GATE, ADJ>(a, comp, stream);
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
