// The gated linear recurrence: the scan with its decays and inputs made from
// gates in the same pass.  Per lane, with k = c softplus(lam):
//
//   rg = sigmoid(r), ig = sigmoid(i), G = k rg, a = exp(-G), s = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + s_t ig_t x_t           (first token of a segment:
//                                               a = 0, hence s = 1)
//
// 1 - a is taken from the exponential's Taylor series where G <= 1/4, so that
// decays near one keep their distance from one, and 1 - a^2 = (1 - a)(1 + a).
//
// A tile is TC = NW * L tokens of 64 lanes: warp w of the NW consumer warps
// holds L tokens of them, two lanes a thread.  Each thread reduces its tokens
// to the map h -> P h + Q, the warps' maps meet in shared memory, and the
// tile's map is published in global memory.  The state that enters the tile
// is folded from the maps of the tiles before it, always in the same order,
// so that two calls agree bit for bit: maps of tiles and of groups of 16
// tiles, and the state after every 256 tiles.  A fixed grid of CTAs takes the
// tiles by ticket, all lanes' earliest tiles first, so a tile waits for
// running CTAs alone; one warp copies tiles in ahead (bulk tensor copies into
// S stages), one folds entering states ahead, and the consumers keep a and
// the input of their tokens in registers between the two walks, so that HBM
// carries each element once.
#pragma once

#include "gates_args.h"
#include "packed_f32x2.cuh"
#include "scan_common.cuh"

namespace lrscan {

enum GatesSite : int { kSiteGatesFold = 20, kSiteGatesRow = 21 };

// ----------------------------------------------------------------------------
// Gates of two lanes
// ----------------------------------------------------------------------------
__device__ __forceinline__ float ex2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(x) = 1 / (1 + 2^(-x log2 e))
__device__ __forceinline__ void sigmoid2(float (&g)[2], const float (&x)[2]) {
    float t[2];
    mul_x2(t[0], t[1], x[0], x[1], -kLog2e, -kLog2e);
    t[0] = ex2_fast(t[0]);
    t[1] = ex2_fast(t[1]);
    add_x2(t[0], t[1], t[0], t[1], 1.0f, 1.0f);
    g[0] = rcp_fast(t[0]);
    g[1] = rcp_fast(t[1]);
}

// k = c softplus(lam)
__device__ __forceinline__ float gate_rate(float lam, float c) {
    return c * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam))));
}

// rg and k to G = k rg, a = exp(-G), s = sqrt(1 - a^2) and 1/s (large where s
// is 0).  far: some lane's k is over 1/4, so the series alone does not do.
__device__ __forceinline__ void decay2(const float (&k)[2], const float (&rg)[2], bool far, float (&G)[2],
                                       float (&a)[2], float (&s)[2], float (&rs)[2]) {
    float n[2], q[2], m[2], y[2];
    mul_x2(G[0], G[1], k[0], k[1], rg[0], rg[1]);
    mul_x2(n[0], n[1], G[0], G[1], -1.0f, -1.0f);
    // 1 - exp(n) = G (1 + n/2 + n^2/6 + ...) to the sixth power: 5e-8 of it at G = 1/4
    fma_x2(q[0], q[1], n[0], n[1], 1.0f / 720, 1.0f / 720, 1.0f / 120, 1.0f / 120);
    fma_x2(q[0], q[1], n[0], n[1], q[0], q[1], 1.0f / 24, 1.0f / 24);
    fma_x2(q[0], q[1], n[0], n[1], q[0], q[1], 1.0f / 6, 1.0f / 6);
    fma_x2(q[0], q[1], n[0], n[1], q[0], q[1], 0.5f, 0.5f);
    fma_x2(q[0], q[1], n[0], n[1], q[0], q[1], 1.0f, 1.0f);
    mul_x2(m[0], m[1], G[0], G[1], q[0], q[1]);
    if (far) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float e = 1.0f - ex2_fast(kLog2e * n[v]);
            m[v] = G[v] > 0.25f ? e : m[v];
        }
    }
    fma_x2(a[0], a[1], m[0], m[1], -1.0f, -1.0f, 1.0f, 1.0f);
    fma_x2(y[0], y[1], m[0], m[1], a[0], a[1], m[0], m[1]);  // m (1 + a)
#pragma unroll
    for (int v = 0; v < 2; ++v) rs[v] = rsqrt_fast(fmaxf(y[v], 1e-37f));
    mul_x2(s[0], s[1], y[0], y[1], rs[0], rs[1]);
}

// ----------------------------------------------------------------------------
// Maps h -> P h + Q.  A map with P = 0 (a segment starts inside) takes nothing
// of what came before, not even an infinity.
// ----------------------------------------------------------------------------
template <bool SEG> __device__ __forceinline__ float apply_map(float P, float Q, float h) {
    const float y = __fmaf_rn(P, h, Q);
    return SEG && P == 0.0f ? Q : y;
}
template <bool SEG> __device__ __forceinline__ float join_rate(float P, float Pin) {
    return SEG && P == 0.0f ? 0.0f : P * Pin;
}
// (P, Q) := (P2, Q2) o (P, Q), two lanes; m = P2, P2', Q2, Q2'
template <bool SEG> __device__ __forceinline__ void join2(float (&P)[2], float (&Q)[2], const float4 &m) {
    if constexpr (SEG) {
        Q[0] = apply_map<SEG>(m.x, m.z, Q[0]);
        Q[1] = apply_map<SEG>(m.y, m.w, Q[1]);
        P[0] = join_rate<SEG>(m.x, P[0]);
        P[1] = join_rate<SEG>(m.y, P[1]);
    } else {
        fma_x2(Q[0], Q[1], m.x, m.y, Q[0], Q[1], m.z, m.w);
        mul_x2(P[0], P[1], m.x, m.y, P[0], P[1]);
    }
}

// Publication: a lane's map is one 64-bit word (P low, Q high), stored whole;
// all-ones words mean nothing is out yet (a NaN with those bits is published
// as another NaN).
constexpr uint32_t kNotOut = 0xffffffffu;
__device__ __forceinline__ uint64_t map_word(float P, float Q) {
    uint32_t p = __float_as_uint(P), q = __float_as_uint(Q);
    p = p == kNotOut ? 0x7fffffffu : p;
    q = q == kNotOut ? 0x7fffffffu : q;
    return (static_cast<uint64_t>(q) << 32) | p;
}
__device__ __forceinline__ void publish2(uint64_t *at, const float (&P)[2], const float (&Q)[2]) {
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(at), "l"(map_word(P[0], Q[0])),
                 "l"(map_word(P[1], Q[1]))
                 : "memory");
}
__device__ __forceinline__ void peek2(const uint64_t *at, uint64_t (&w)[2]) {
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[1]) : "l"(at) : "memory");
}
__device__ __forceinline__ bool is_out(const uint64_t (&w)[2]) {
    return static_cast<uint32_t>(w[0]) != kNotOut && static_cast<uint32_t>(w[1]) != kNotOut;
}
__device__ __forceinline__ float4 map_of(const uint64_t (&w)[2]) {
    return make_float4(__uint_as_float(static_cast<uint32_t>(w[0])), __uint_as_float(static_cast<uint32_t>(w[1])),
                       __uint_as_float(static_cast<uint32_t>(w[0] >> 32)),
                       __uint_as_float(static_cast<uint32_t>(w[1] >> 32)));
}

// Folds the n published maps at `at` (64 words apart), earliest first, into
// (P, Q), one warp, its lanes two tile lanes each.  False when the wait
// expired or the CTA is aborting.
template <bool SEG>
__device__ __forceinline__ bool fold_maps(const uint64_t *at, int n, float (&P)[2], float (&Q)[2], const WaitCtx &wc) {
    constexpr int kBatch = 8;
    for (int e0 = 0; e0 < n; e0 += kBatch) {
        uint64_t w[kBatch][2];
        uint64_t start = 0;
        for (uint32_t spin = 0;; ++spin) {
            bool all = true;
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (e0 + e < n) peek2(at + static_cast<size_t>(e0 + e) * kGatesLanes, w[e]);
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (e0 + e < n) all = all && is_out(w[e]);
            if (__all_sync(0xffffffffu, all)) break;
            if ((spin & 15u) == 15u) {
                const uint64_t now = global_timer_ns();
                if (start == 0) start = now;
                bool stop = *wc.abort_flag != 0;
                if (now - start > wc.timeout_ns) {
                    record_error(wc, kErrTimeout, kSiteGatesFold);
                    stop = true;
                }
                if (__any_sync(0xffffffffu, stop)) return false;
            }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (e0 + e < n) join2<SEG>(P, Q, map_of(w[e]));
    }
    return true;
}

// ----------------------------------------------------------------------------
// Shared-memory plan, the same for both directions
// ----------------------------------------------------------------------------
struct GatesTile {
    int n, c, b, d0;  // n < 0: no more tiles
};

template <class St, int NW, int L, int S, int PLANES, bool BULK> struct GatesGeo {
    static constexpr int TC = NW * L;
    static constexpr int kConsumers = NW * 32;
    static constexpr int kThreads = kConsumers + 64;  // and the copy warp and the fold warp
    static constexpr int kPlane = TC * kGatesLanes * static_cast<int>(sizeof(St));
    static constexpr int kStage = BULK ? PLANES * kPlane : 0;
    static constexpr int kWords = (TC + 31) / 32;
    static constexpr int off_sum = S * kStage;                                     // float [2][NW][32][6]
    static constexpr int off_lam = off_sum + 2 * NW * 32 * 6 * 4;                  // float [2][NW][64]
    static constexpr int off_rate = off_lam + (PLANES == 4 ? 2 * NW * 64 * 4 : 0); // float [S][64]
    static constexpr int off_in = off_rate + S * 64 * 4;                           // float [S][64]
    static constexpr int off_tile = off_in + S * 64 * 4;                           // GatesTile [S]
    static constexpr int off_seg = off_tile + S * 16;                              // u32 [S][kWords]
    static constexpr int off_bar = (off_seg + S * kWords * 4 + 7) / 8 * 8;         // u64 [4][S]
    static constexpr int off_flag = off_bar + 4 * S * 8;
    static constexpr int kBytes = off_flag + 16 + 128;                             // and the base's alignment
};

template <bool BULK> __device__ __forceinline__ int lane_at(int lane, int v) { return BULK ? 2 * lane + v : lane + 32 * v; }

__device__ __forceinline__ void consumers_sync(int threads) {
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// The copy warp, both directions: takes tickets, names the stage's tile, its
// lanes' rates and the tokens that start a segment, and copies its planes in.
template <class Geo, bool BULK, bool SEG, bool BWD, int PLANES, int S>
__device__ __forceinline__ void gates_copy_warp(const GatesArgs &g, const CUtensorMap *const (&maps)[4], char *smem,
                                                uint32_t full, uint32_t empty, const WaitCtx &wc) {
    const int lane = threadIdx.x & 31;
    const unsigned total = static_cast<unsigned>(g.nl) * g.nc;
    float *rate = reinterpret_cast<float *>(smem + Geo::off_rate);
    GatesTile *tile = reinterpret_cast<GatesTile *>(smem + Geo::off_tile);
    uint32_t *segw = reinterpret_cast<uint32_t *>(smem + Geo::off_seg);
    const bool one = g.nc == 1;  // no tile waits for another: no tickets
    unsigned tk = blockIdx.x;
    if (!one) {
        if (lane == 0) tk = atomicAdd(g.ticket, 1u) + 1u;  // the word starts as all ones
        tk = __shfl_sync(0xffffffffu, tk, 0);
    }
    int issued = 0;
    bool ok = true;
    for (int it = 0;; ++it) {
        const int s = it % S;
        ok = mbar_wait(empty + 8 * s, ((it / S) & 1) ^ 1, wc, kSiteProducerEmpty);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        GatesTile t;
        const bool end = tk >= total;
        t.c = static_cast<int>(tk / static_cast<unsigned>(g.nl));
        t.n = static_cast<int>(tk % static_cast<unsigned>(g.nl));
        t.b = t.n / g.ndt;
        t.d0 = (t.n % g.ndt) * kGatesLanes;
        if (end) t.n = -1;
        const long long t0 = static_cast<long long>(BWD ? g.nc - 1 - t.c : t.c) * Geo::TC;
        if (lane == 0) {
            tile[s] = t;
            if (end) {
                mbar_arrive(full + 8 * s);
            } else if (BULK) {
                mbar_arrive_expect_tx(full + 8 * s, Geo::kStage);
                const uint32_t dst = smem_addr(smem) + s * Geo::kStage;
#pragma unroll
                for (int p = 0; p < PLANES; ++p)
                    tma_load_3d(dst + p * Geo::kPlane, maps[p], t.d0, static_cast<int>(t0), t.b, full + 8 * s);
            } else {
                mbar_arrive(full + 8 * s);
            }
        }
        if (end) {
            __syncwarp();
            if (lane == 0) mbar_arrive(full + 8 * s);
            break;
        }
        issued = it + 1;
        if (one)
            tk += gridDim.x;
        else if (lane == 0)
            tk = atomicAdd(g.ticket, 1u) + 1u;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int d = t.d0 + lane_at<BULK>(lane, v);
            rate[s * 64 + lane_at<BULK>(lane, v)] = gate_rate(d < g.D ? __ldg(g.lam + d) : 0.0f, g.c);
        }
        if constexpr (SEG) {
            const int32_t *seg = g.seg + static_cast<long long>(t.b) * g.T + t0;
#pragma unroll
            for (int k = 0; k < Geo::kWords; ++k) {
                const int row = 32 * k + lane;
                const bool first = row < Geo::TC && t0 + row < g.T && __ldg(seg + row) == 0;
                const uint32_t bits = __ballot_sync(0xffffffffu, first);
                if (lane == 0) segw[s * Geo::kWords + k] = bits;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full + 8 * s);
        if (!one) tk = __shfl_sync(0xffffffffu, tk, 0);
    }
    if (BULK && !ok && lane == 0) {
        // leaving early: no copy of this CTA may still be on its way
        for (int it = issued > S ? issued - S : 0; it < issued; ++it) {
            const uint64_t start = global_timer_ns();
            while (!mbar_try_wait(full + 8 * (it % S), (it / S) & 1))
                if (global_timer_ns() - start > wc.timeout_ns) {
                    record_error(wc, kErrTimeout, kSiteDrain);
                    break;
                }
        }
    }
}

// The fold warp, both directions: the state (or adjoint) that enters each of
// the CTA's tiles, and the maps of groups of tiles.  `start` [B, D]: what
// enters the first tile, or null for zeros.
template <class Geo, bool BULK, bool SEG, int S>
__device__ __forceinline__ void gates_fold_warp(const GatesArgs &g, const float *start, char *smem, uint32_t full,
                                                uint32_t empty, uint32_t hfull, uint32_t hempty, const WaitCtx &wc) {
    constexpr int R = kGatesRadix;
    const int lane = threadIdx.x & 31;
    const GatesTile *tile = reinterpret_cast<const GatesTile *>(smem + Geo::off_tile);
    float *hin = reinterpret_cast<float *>(smem + Geo::off_in);
    for (int it = 0;; ++it) {
        const int s = it % S;
        const uint32_t ph = (it / S) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * s, ph, wc, kSiteConsumerFull))) return;
        const GatesTile t = tile[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        if (t.n < 0) return;
        const int c = t.c, g1 = c / R, g2 = g1 / R;
        const int n1 = (g.nc + R - 1) / R, n2 = (n1 + R - 1) / R;
        const size_t word = static_cast<size_t>(lane) * 2;
        uint64_t *agg1 = g.agg1 + static_cast<size_t>(t.n) * g.nc * kGatesLanes + word;
        uint64_t *agg2 = g.agg2 + static_cast<size_t>(t.n) * n1 * kGatesLanes + word;
        uint64_t *agg3 = g.agg3 + static_cast<size_t>(t.n) * n2 * kGatesLanes + word;
        // the tiles of this tile's own group before it
        float P[2] = {1.0f, 1.0f}, Q[2] = {0.0f, 0.0f};
        if (!fold_maps<SEG>(agg1 + static_cast<size_t>(g1) * R * kGatesLanes, c - g1 * R, P, Q, wc)) return;
        float PG[2] = {P[0], P[1]}, QG[2] = {Q[0], Q[1]};
        const bool closes = c % R == R - 1 && c + 1 < g.nc;
        if (closes) {  // the group's map is out before anything of earlier groups is waited for
            if (!fold_maps<SEG>(agg1 + static_cast<size_t>(c) * kGatesLanes, 1, PG, QG, wc)) return;
            publish2(agg2 + static_cast<size_t>(g1) * kGatesLanes, PG, QG);
        }
        // what enters the group
        float h[2] = {0.0f, 0.0f}, none[2] = {1.0f, 1.0f};
        if (g2 > 0) {
            if (!fold_maps<SEG>(agg3 + static_cast<size_t>(g2 - 1) * kGatesLanes, 1, none, h, wc)) return;
        } else if (start != nullptr) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int d = t.d0 + lane_at<BULK>(lane, v);
                if (d < g.D) h[v] = __ldg(start + static_cast<long long>(t.b) * g.D + d);
            }
        }
        if (!fold_maps<SEG>(agg2 + static_cast<size_t>(g2) * R * kGatesLanes, g1 - g2 * R, none, h, wc)) return;
        if (!__all_sync(0xffffffffu, mbar_wait(hempty + 8 * s, ph ^ 1, wc, kSiteProducerEmpty))) return;
#pragma unroll
        for (int v = 0; v < 2; ++v) hin[s * 64 + lane_at<BULK>(lane, v)] = apply_map<SEG>(P[v], Q[v], h[v]);
        __syncwarp();
        if (lane == 0) mbar_arrive(hfull + 8 * s);
        if (closes && c % (R * R) == R * R - 1) {  // the state after these R * R tiles
            float zero[2] = {0.0f, 0.0f}, S2[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) S2[v] = apply_map<SEG>(PG[v], QG[v], h[v]);
            publish2(agg3 + static_cast<size_t>(g2) * kGatesLanes, zero, S2);
        }
    }
}

// Two lanes of one token from the stage (bulk) or from memory.
template <class St, bool BULK>
__device__ __forceinline__ void stage_pair(const char *plane, int row, int lane, float (&x)[2]) {
    unpack_lanes<St, 2>(reinterpret_cast<const St *>(plane) + row * kGatesLanes + 2 * lane, x);
}
template <class St>
__device__ __forceinline__ float load_one(const St *p, bool in) {
    if (!in) return 0.0f;
    float x[1];
    load_lanes_global<St, 1>(p, x);
    return x[0];
}
template <class St, bool BULK>
__device__ __forceinline__ void store_pair(St *row, int lane, const bool (&in)[2], float y0, float y1) {
    if constexpr (BULK) {
        float y[2] = {y0, y1};
        if (in[0]) store_lanes<St, 2>(row + 2 * lane, y);
    } else {
        float u[1] = {y0}, w[1] = {y1};
        if (in[0]) store_lanes<St, 1>(row + lane, u);
        if (in[1]) store_lanes<St, 1>(row + lane + 32, w);
    }
}

// ----------------------------------------------------------------------------
// Forward
// ----------------------------------------------------------------------------
template <class St, int NW, int L, int S, bool BULK, bool SEG, int CTAS>
__global__ void __launch_bounds__(NW * 32 + 64, CTAS)
gates_fwd_kernel(const GatesArgs g, const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mi,
                 const __grid_constant__ CUtensorMap mx) {
    using Geo = GatesGeo<St, NW, L, S, 3, BULK>;
    extern __shared__ char smem_base[];
    char *smem = smem_base + ((128u - (smem_addr(smem_base) & 127u)) & 127u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *flag = reinterpret_cast<volatile int *>(smem + Geo::off_flag);
    const uint32_t bars = smem_addr(smem) + Geo::off_bar;
    const uint32_t full = bars, empty = bars + 8 * S, hfull = bars + 16 * S, hempty = bars + 24 * S;
    const WaitCtx wc{g.status, flag, g.timeout_ns};
    if (threadIdx.x == 0) {
        *flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 2);
            mbar_init(empty + 8 * s, NW + 1);
            mbar_init(hfull + 8 * s, 1);
            mbar_init(hempty + 8 * s, NW);
        }
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == NW) {
        const CUtensorMap *const maps[4] = {&mr, &mi, &mx, nullptr};
        gates_copy_warp<Geo, BULK, SEG, false, 3, S>(g, maps, smem, full, empty, wc);
        return;
    }
    if (warp == NW + 1) {
        gates_fold_warp<Geo, BULK, SEG, S>(g, g.h0, smem, full, empty, hfull, hempty, wc);
        return;
    }
    const GatesTile *tile = reinterpret_cast<const GatesTile *>(smem + Geo::off_tile);
    const float *rate = reinterpret_cast<const float *>(smem + Geo::off_rate);
    const float *hin = reinterpret_cast<const float *>(smem + Geo::off_in);
    const uint32_t *segw = reinterpret_cast<const uint32_t *>(smem + Geo::off_seg);
    float4 *sums = reinterpret_cast<float4 *>(smem + Geo::off_sum);
    const long long ns = (g.T + kGatesSave - 1) / kGatesSave;
    for (int it = 0;; ++it) {
        const int s = it % S;
        const uint32_t ph = (it / S) & 1;
        bool ok = mbar_wait(full + 8 * s, ph, wc, kSiteConsumerFull);
        const GatesTile t = tile[s];
        if (bar_sync_or(2, NW * 32, !ok)) return;  // one warp's failed wait stops them all
        if (t.n < 0) return;
        const long long t0 = static_cast<long long>(t.c) * Geo::TC + warp * L;  // this warp's first token
        bool in[2];
        float k[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            in[v] = t.d0 + lane_at<BULK>(lane, v) < g.D;
            k[v] = rate[s * 64 + lane_at<BULK>(lane, v)];
        }
        const bool far = __any_sync(0xffffffffu, k[0] > 0.25f || k[1] > 0.25f || k[0] != k[0] || k[1] != k[1]);
        uint32_t first = 0;
        if constexpr (SEG) first = segw[s * Geo::kWords + (warp * L) / 32] >> ((warp * L) & 31);
        float a[L][2], b[L][2];
        float P[2] = {1.0f, 1.0f}, Q[2] = {0.0f, 0.0f};
        const char *stage = smem + s * Geo::kStage;
        [[maybe_unused]] float raw[BULK ? 1 : L][3][2];
        if constexpr (!BULK) {
#pragma unroll
            for (int l = 0; l < L; ++l)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const bool ld = in[v] && t0 + l < g.T;
                    const long long d = t.d0 + lane_at<BULK>(lane, v);
                    raw[l][0][v] = load_one(static_cast<const St *>(g.r.p) + t.b * g.r.sb + (t0 + l) * g.r.st + d, ld);
                    raw[l][1][v] = load_one(static_cast<const St *>(g.i.p) + t.b * g.i.sb + (t0 + l) * g.i.st + d, ld);
                    raw[l][2][v] = load_one(static_cast<const St *>(g.x.p) + t.b * g.x.sb + (t0 + l) * g.x.st + d, ld);
                }
        }
        const bool ragged = t0 + L > g.T;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float r[2], i[2], x[2], rg[2], ig[2], G[2], sq[2], rs[2];
            if constexpr (BULK) {
                stage_pair<St, BULK>(stage, warp * L + l, lane, r);
                stage_pair<St, BULK>(stage + Geo::kPlane, warp * L + l, lane, i);
                stage_pair<St, BULK>(stage + 2 * Geo::kPlane, warp * L + l, lane, x);
            } else {
#pragma unroll
                for (int v = 0; v < 2; ++v) { r[v] = raw[l][0][v]; i[v] = raw[l][1][v]; x[v] = raw[l][2][v]; }
            }
            sigmoid2(rg, r);
            sigmoid2(ig, i);
            decay2(k, rg, far, G, a[l], sq, rs);
            mul_x2(b[l][0], b[l][1], ig[0], ig[1], x[0], x[1]);
            const bool start = SEG && ((first >> l) & 1u);
            if (start) {  // the token's own input alone
#pragma unroll
                for (int v = 0; v < 2; ++v) { a[l][v] = 0.0f; sq[v] = 1.0f; }
            }
            mul_x2(b[l][0], b[l][1], b[l][0], b[l][1], sq[0], sq[1]);
            if (ragged && t0 + l >= g.T) {
#pragma unroll
                for (int v = 0; v < 2; ++v) { a[l][v] = 1.0f; b[l][v] = 0.0f; }
            }
            if (start) {
#pragma unroll
                for (int v = 0; v < 2; ++v) { P[v] = 0.0f; Q[v] = b[l][v]; }
            } else {
                fma_x2(Q[0], Q[1], a[l][0], a[l][1], Q[0], Q[1], b[l][0], b[l][1]);
                mul_x2(P[0], P[1], P[0], P[1], a[l][0], a[l][1]);
            }
        }
        float4 *sum = sums + (it & 1) * NW * 32;
        sum[warp * 32 + lane] = make_float4(P[0], P[1], Q[0], Q[1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        consumers_sync(NW * 32);
        float Pe[2] = {1.0f, 1.0f}, Qe[2] = {0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW - 1; ++w)
            if (w < warp) join2<SEG>(Pe, Qe, sum[w * 32 + lane]);
        if (warp == NW - 1 && t.c + 1 < g.nc) {
            float Pt[2] = {Pe[0], Pe[1]}, Qt[2] = {Qe[0], Qe[1]};
            join2<SEG>(Pt, Qt, make_float4(P[0], P[1], Q[0], Q[1]));
            publish2(g.agg1 + (static_cast<size_t>(t.n) * g.nc + t.c) * kGatesLanes + 2 * lane, Pt, Qt);
        }
        ok = mbar_wait(hfull + 8 * s, ph, wc, kSiteGatesRow);
        float h[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = apply_map<SEG>(Pe[v], Qe[v], hin[s * 64 + lane_at<BULK>(lane, v)]);
        __syncwarp();
        if (lane == 0) mbar_arrive(hempty + 8 * s);
        if (!ok) continue;  // the next barrier stops the consumers
        if (g.saved != nullptr && (warp * L) % kGatesSave == 0 && t0 < g.T) {
            float *to = g.saved + (t.b * ns + t0 / kGatesSave) * g.D + t.d0;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (in[v]) to[lane_at<BULK>(lane, v)] = h[v];
        }
        St *out = static_cast<St *>(g.o0.p) + t.b * g.o0.sb + t0 * g.o0.st + t.d0;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            if (SEG && ((first >> l) & 1u)) {
                h[0] = b[l][0];
                h[1] = b[l][1];
            } else {
                fma_x2(h[0], h[1], a[l][0], a[l][1], h[0], h[1], b[l][0], b[l][1]);
            }
            if (!ragged || t0 + l < g.T) store_pair<St, BULK>(out, lane, in, h[0], h[1]);
            out += g.o0.st;
        }
        if (warp == NW - 1 && t.c + 1 == g.nc && g.edge != nullptr) {
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (in[v]) g.edge[t.b * g.D + t.d0 + lane_at<BULK>(lane, v)] = h[v];
        }
    }
}

// ----------------------------------------------------------------------------
// Backward.  With g_t = grad_out_t + a_{t+1} g_{t+1}, token t hands
// c_t = a_t g_t = a_t grad_out_t + a_t c_{t+1} to the token before it: maps
// over the tile's own decays, folded from the last tile to the first, with
// the same P as the forward's.  The states of the tile's tokens are made
// again in fp32 from the state saved before it, so that neither the rounded
// output is read nor its rounding enters the gradients.  Per token
//   q  = dL/d(log a) log a = -G a g (h_{t-1} - ig x a / s)
//   grad_r = q (1 - rg)     grad_x = g s ig     grad_i = grad_x x (1 - ig)
//   grad_lam = sigmoid(lam) / softplus(lam) sum q
// (first token of a segment: a = 0 and s = 1 are constants, so q = 0).
// ----------------------------------------------------------------------------
template <class St, int NW, int L, int S, bool BULK, bool SEG, int CTAS>
__global__ void __launch_bounds__(NW * 32 + 64, CTAS)
gates_bwd_kernel(const GatesArgs g, const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mi,
                 const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg) {
    using Geo = GatesGeo<St, NW, L, S, 4, BULK>;
    static_assert(Geo::TC == kGatesSave, "a tile starts at a saved state");
    extern __shared__ char smem_base[];
    char *smem = smem_base + ((128u - (smem_addr(smem_base) & 127u)) & 127u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *flag = reinterpret_cast<volatile int *>(smem + Geo::off_flag);
    const uint32_t bars = smem_addr(smem) + Geo::off_bar;
    const uint32_t full = bars, empty = bars + 8 * S, hfull = bars + 16 * S, hempty = bars + 24 * S;
    const WaitCtx wc{g.status, flag, g.timeout_ns};
    if (threadIdx.x == 0) {
        *flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 2);
            mbar_init(empty + 8 * s, NW + 1);
            mbar_init(hfull + 8 * s, 1);
            mbar_init(hempty + 8 * s, NW);
        }
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == NW) {
        const CUtensorMap *const maps[4] = {&mr, &mi, &mx, &mg};
        gates_copy_warp<Geo, BULK, SEG, true, 4, S>(g, maps, smem, full, empty, wc);
        return;
    }
    if (warp == NW + 1) {
        gates_fold_warp<Geo, BULK, SEG, S>(g, g.grad_last, smem, full, empty, hfull, hempty, wc);
        return;
    }
    const GatesTile *tile = reinterpret_cast<const GatesTile *>(smem + Geo::off_tile);
    const float *rate = reinterpret_cast<const float *>(smem + Geo::off_rate);
    const float *cin = reinterpret_cast<const float *>(smem + Geo::off_in);
    const uint32_t *segw = reinterpret_cast<const uint32_t *>(smem + Geo::off_seg);
    float2 *sums = reinterpret_cast<float2 *>(smem + Geo::off_sum);   // [2][NW][3][32]: P, Q forward, Q backward
    float *lams = reinterpret_cast<float *>(smem + Geo::off_lam);     // [2][NW][64]
    long long part_row = -1;                                          // of the tile before this one
    int part_d0 = 0;
    for (int it = 0;; ++it) {
        const int s = it % S;
        const uint32_t ph = (it / S) & 1;
        bool ok = mbar_wait(full + 8 * s, ph, wc, kSiteConsumerFull);
        const GatesTile t = tile[s];
        if (bar_sync_or(2, NW * 32, !ok)) return;
        // the tile before this one: its warps' sums of q, in warp order
        if (part_row >= 0 && warp < 2) {
            const float *from = lams + ((it & 1) ^ 1) * NW * 64;
            const int j = threadIdx.x;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) sum += from[w * 64 + j];
            if (part_d0 + j < g.D) g.part[part_row * g.D + part_d0 + j] = sum;
        }
        if (t.n < 0) return;
        const int ct = g.nc - 1 - t.c;  // the tile's place in time
        part_row = static_cast<long long>(ct) * g.B + t.b;
        part_d0 = t.d0;
        const long long t0 = static_cast<long long>(ct) * Geo::TC + warp * L;
        bool in[2];
        float k[2], hs[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int d = t.d0 + lane_at<BULK>(lane, v);
            in[v] = d < g.D;
            k[v] = rate[s * 64 + lane_at<BULK>(lane, v)];
            hs[v] = in[v] ? __ldg(g.saved + (static_cast<long long>(t.b) * g.nc + ct) * g.D + d) : 0.0f;
        }
        const bool far = __any_sync(0xffffffffu, k[0] > 0.25f || k[1] > 0.25f || k[0] != k[0] || k[1] != k[1]);
        uint32_t first = 0;
        if constexpr (SEG) first = segw[s * Geo::kWords + (warp * L) / 32] >> ((warp * L) & 31);
        const bool ragged = t0 + L > g.T;
        // a: decays; u = s ig; b = u x; v1 = x (1 - ig); w1 = G a; w2 = ig x a / s; z = 1 - rg; go
        float a[L][2], u[L][2], b[L][2], v1[L][2], w1[L][2], w2[L][2], z[L][2], go[L][2];
        float P[2] = {1.0f, 1.0f}, Q[2] = {0.0f, 0.0f};
        const char *stage = smem + s * Geo::kStage;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float r[2], i[2], x[2], rg[2], ig[2], G[2], sq[2], rs[2];
            if constexpr (BULK) {
                stage_pair<St, BULK>(stage, warp * L + l, lane, r);
                stage_pair<St, BULK>(stage + Geo::kPlane, warp * L + l, lane, i);
                stage_pair<St, BULK>(stage + 2 * Geo::kPlane, warp * L + l, lane, x);
                stage_pair<St, BULK>(stage + 3 * Geo::kPlane, warp * L + l, lane, go[l]);
            } else {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const bool ld = in[v] && t0 + l < g.T;
                    const long long d = t.d0 + lane_at<BULK>(lane, v);
                    r[v] = load_one(static_cast<const St *>(g.r.p) + t.b * g.r.sb + (t0 + l) * g.r.st + d, ld);
                    i[v] = load_one(static_cast<const St *>(g.i.p) + t.b * g.i.sb + (t0 + l) * g.i.st + d, ld);
                    x[v] = load_one(static_cast<const St *>(g.x.p) + t.b * g.x.sb + (t0 + l) * g.x.st + d, ld);
                    go[l][v] = load_one(static_cast<const St *>(g.go.p) + t.b * g.go.sb + (t0 + l) * g.go.st + d, ld);
                }
            }
            sigmoid2(rg, r);
            sigmoid2(ig, i);
            decay2(k, rg, far, G, a[l], sq, rs);
            const bool start = SEG && ((first >> l) & 1u);
            if (start) {
#pragma unroll
                for (int v = 0; v < 2; ++v) { a[l][v] = 0.0f; sq[v] = 1.0f; rs[v] = 1.0f; }
            }
            if (ragged && t0 + l >= g.T) {
#pragma unroll
                for (int v = 0; v < 2; ++v) { a[l][v] = 1.0f; sq[v] = 0.0f; rs[v] = 0.0f; G[v] = 0.0f; }
            }
            float ixa[2], nig[2];
            mul_x2(u[l][0], u[l][1], sq[0], sq[1], ig[0], ig[1]);
            mul_x2(b[l][0], b[l][1], u[l][0], u[l][1], x[0], x[1]);
            fma_x2(nig[0], nig[1], ig[0], ig[1], -1.0f, -1.0f, 1.0f, 1.0f);
            mul_x2(v1[l][0], v1[l][1], x[0], x[1], nig[0], nig[1]);
            fma_x2(z[l][0], z[l][1], rg[0], rg[1], -1.0f, -1.0f, 1.0f, 1.0f);
            mul_x2(w1[l][0], w1[l][1], G[0], G[1], a[l][0], a[l][1]);
            mul_x2(ixa[0], ixa[1], ig[0], ig[1], x[0], x[1]);
            mul_x2(ixa[0], ixa[1], ixa[0], ixa[1], a[l][0], a[l][1]);
            mul_x2(w2[l][0], w2[l][1], ixa[0], ixa[1], rs[0], rs[1]);
            if (start) {
#pragma unroll
                for (int v = 0; v < 2; ++v) { P[v] = 0.0f; Q[v] = b[l][v]; }
            } else {
                fma_x2(Q[0], Q[1], a[l][0], a[l][1], Q[0], Q[1], b[l][0], b[l][1]);
                mul_x2(P[0], P[1], P[0], P[1], a[l][0], a[l][1]);
            }
        }
        // the adjoint's map over these tokens, last to first
        float QB[2] = {0.0f, 0.0f};
#pragma unroll
        for (int l = L - 1; l >= 0; --l) {
            if (SEG && ((first >> l) & 1u)) {
                QB[0] = QB[1] = 0.0f;
            } else {
                add_x2(QB[0], QB[1], QB[0], QB[1], go[l][0], go[l][1]);
                mul_x2(QB[0], QB[1], QB[0], QB[1], a[l][0], a[l][1]);
            }
        }
        float2 *sum = sums + (it & 1) * NW * 96;
        sum[warp * 96 + lane] = make_float2(P[0], P[1]);
        sum[warp * 96 + 32 + lane] = make_float2(Q[0], Q[1]);
        sum[warp * 96 + 64 + lane] = make_float2(QB[0], QB[1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        consumers_sync(NW * 32);
        float h[2] = {hs[0], hs[1]}, Pe[2] = {1.0f, 1.0f}, Qe[2] = {0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) {
                const float2 p = sum[w * 96 + lane], q = sum[w * 96 + 32 + lane];
                h[0] = apply_map<SEG>(p.x, q.x, h[0]);
                h[1] = apply_map<SEG>(p.y, q.y, h[1]);
            }
            const int y = NW - 1 - w;
            if (y > warp) {
                const float2 p = sum[y * 96 + lane], q = sum[y * 96 + 64 + lane];
                join2<SEG>(Pe, Qe, make_float4(p.x, p.y, q.x, q.y));
            }
        }
        if (warp == 0 && t.c + 1 < g.nc) {
            float Pt[2] = {Pe[0], Pe[1]}, Qt[2] = {Qe[0], Qe[1]};
            join2<SEG>(Pt, Qt, make_float4(P[0], P[1], QB[0], QB[1]));
            publish2(g.agg1 + (static_cast<size_t>(t.n) * g.nc + t.c) * kGatesLanes + 2 * lane, Pt, Qt);
        }
        // the states again: w1 becomes dL/d(log a) log a for a unit adjoint
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float e[2];
            if (SEG && ((first >> l) & 1u)) {
                w1[l][0] = w1[l][1] = 0.0f;
                h[0] = b[l][0];
                h[1] = b[l][1];
            } else {
                fma_x2(e[0], e[1], h[0], h[1], -1.0f, -1.0f, w2[l][0], w2[l][1]);
                mul_x2(w1[l][0], w1[l][1], w1[l][0], w1[l][1], e[0], e[1]);
                fma_x2(h[0], h[1], a[l][0], a[l][1], h[0], h[1], b[l][0], b[l][1]);
            }
        }
        ok = mbar_wait(hfull + 8 * s, ph, wc, kSiteGatesRow);
        float cc[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) cc[v] = apply_map<SEG>(Pe[v], Qe[v], cin[s * 64 + lane_at<BULK>(lane, v)]);
        __syncwarp();
        if (lane == 0) mbar_arrive(hempty + 8 * s);
        if (!ok) continue;
        St *gr = static_cast<St *>(g.o0.p) + t.b * g.o0.sb + (t0 + L - 1) * g.o0.st + t.d0;
        St *gi = static_cast<St *>(g.o1.p) + t.b * g.o1.sb + (t0 + L - 1) * g.o1.st + t.d0;
        St *gx = static_cast<St *>(g.o2.p) + t.b * g.o2.sb + (t0 + L - 1) * g.o2.st + t.d0;
        float ql[2] = {0.0f, 0.0f};
#pragma unroll
        for (int l = L - 1; l >= 0; --l) {
            float gt[2], q[2], yr[2], yi[2], yx[2];
            add_x2(gt[0], gt[1], go[l][0], go[l][1], cc[0], cc[1]);
            mul_x2(q[0], q[1], gt[0], gt[1], w1[l][0], w1[l][1]);
            add_x2(ql[0], ql[1], ql[0], ql[1], q[0], q[1]);
            mul_x2(yr[0], yr[1], q[0], q[1], z[l][0], z[l][1]);
            mul_x2(yx[0], yx[1], gt[0], gt[1], u[l][0], u[l][1]);
            mul_x2(yi[0], yi[1], yx[0], yx[1], v1[l][0], v1[l][1]);
            if (SEG && ((first >> l) & 1u))
                cc[0] = cc[1] = 0.0f;
            else
                mul_x2(cc[0], cc[1], gt[0], gt[1], a[l][0], a[l][1]);
            if (!ragged || t0 + l < g.T) {
                store_pair<St, BULK>(gr, lane, in, yr[0], yr[1]);
                store_pair<St, BULK>(gi, lane, in, yi[0], yi[1]);
                store_pair<St, BULK>(gx, lane, in, yx[0], yx[1]);
            }
            gr -= g.o0.st;
            gi -= g.o1.st;
            gx -= g.o2.st;
        }
        float *lam = lams + (it & 1) * NW * 64 + warp * 64;
        lam[lane_at<BULK>(lane, 0)] = ql[0];
        lam[lane_at<BULK>(lane, 1)] = ql[1];
        if (warp == 0 && ct == 0 && g.edge != nullptr) {
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (in[v]) g.edge[t.b * g.D + t.d0 + lane_at<BULK>(lane, v)] = cc[v];
        }
    }
}

}  // namespace lrscan
