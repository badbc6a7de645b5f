// Token embedding: out[n] = scale weight[ids[n]], and the gradient of the
// table, grad_weight[v] = scale times the sum of grad_out[n] over the tokens
// with ids[n] = v, in the order of the tokens (two calls agree bit for bit).
// A negative id is no token: a row of zeros, and no gradient.
//
// Backward in three kernels.  One cluster sorts the tokens by id, stably, by
// digits of up to 9 bits: each warp counts the digits of its own stretch of
// tokens, the counts become every warp's first places, and the warp moves its
// tokens there.  Then CTAs sum the rows of equal stretches of the sorted
// tokens, whatever ids they hold, so that a frequent id takes many CTAs and a
// rare one shares its CTA; other CTAs of the same launch write the zeros of
// the rows that have no token.  A stretch's first and last ids may go on
// outside it: those sums are left in fp32, and the third kernel adds them up.
#pragma once

#include "embed_args.h"
#include "scan_common.cuh"

namespace lrscan {

__device__ __forceinline__ long long token_id(const EmbedArgs &a, long long n) {
    return a.wide ? __ldg(static_cast<const long long *>(a.ids) + n)
                  : static_cast<long long>(__ldg(static_cast<const int *>(a.ids) + n));
}
__device__ __forceinline__ void report_id(const EmbedArgs &a, long long n) {
    if (atomicCAS(&a.status->code, 0, kErrRange) == 0) {
        a.status->where = kSiteEmbedId;
        a.status->block = static_cast<unsigned>(n);
    }
}

// Eight (or one) lanes.
template <class St, int V> __device__ __forceinline__ void row_load(const St *p, float (&x)[V]) {
    if constexpr (V == 8 && std::is_same<St, float>::value) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        load_lanes_global<St, V>(p, x);
    }
}

constexpr int kRowsPerThread = 4;

template <class W, class O, int V, int R> __global__ void __launch_bounds__(256) embed_fwd_kernel(const EmbedArgs a) {
    const unsigned nd = static_cast<unsigned>((a.D + 32 * V - 1) / (32 * V));
    const long long d = (static_cast<long long>(blockIdx.x % nd) * 32 + threadIdx.x) * V;
    const long long n0 = static_cast<long long>(blockIdx.x / nd) * (8 * R) + threadIdx.y;
    if (d >= a.D) return;
    float x[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long n = n0 + 8 * r;
        const long long id = n < a.N ? token_id(a, n) : -1;
        if (id >= a.V && d == 0) report_id(a, n);
        if (id >= 0 && id < a.V) {
            row_load<W, V>(static_cast<const W *>(a.in) + id * a.D + d, x[r]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[r][v] = 0.0f;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long n = n0 + 8 * r;
        if (n >= a.N) break;
#pragma unroll
        for (int v = 0; v < V; ++v) x[r][v] *= a.scale;
        store_lanes<O, V>(static_cast<O *>(a.out) + n * a.D + d, x[r]);
    }
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Lanes of the warp that hold the same digit, `bits` bits long.
__device__ __forceinline__ unsigned same_digit(unsigned digit, int bits) {
    unsigned peers = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool one = (digit >> b) & 1u;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        peers &= one ? ones : ~ones;
    }
    return peers;
}

// Sorts (id, token number) by id, stably; marks the ids that occur.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortWarps * 32, 1)
embed_sort_kernel(const EmbedArgs a) {
    extern __shared__ uint32_t count[];  // [kSortWarps][bins + 1]: a warp's counts, then its next places
    __shared__ uint32_t base[kSortBins];
    __shared__ uint32_t sums[kSortBins / 32];
    const int bins = 1 << a.bits, row = bins + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned rank = cluster_rank();
    const long long stretch = ((a.N + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
    const long long first = (static_cast<long long>(rank) * kSortWarps + warp) * stretch;
    const long long last = first + stretch < a.N ? first + stretch : a.N;
    for (long long v = rank * blockDim.x + threadIdx.x; v < a.V; v += kSortCtas * blockDim.x) a.present[v] = 0;
    uint32_t *mine = count + warp * row;
    for (int p = 0; p < a.passes; ++p) {
        const uint32_t *kin = p & 1 ? a.keys[1] : a.keys[0], *vin = p & 1 ? a.vals[1] : a.vals[0];
        uint32_t *kout = p & 1 ? a.keys[0] : a.keys[1], *vout = p & 1 ? a.vals[0] : a.vals[1];
        const int shift = p * a.bits;
        auto key_of = [&](long long n) -> uint32_t {
            if (p > 0) return kin[n];
            const long long id = token_id(a, n);
            if (id >= a.V) report_id(a, n);
            return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
        };
        for (int j = threadIdx.x; j < kSortWarps * row; j += blockDim.x) count[j] = 0;
        __syncthreads();
        for (long long n0 = first; n0 < last; n0 += 32) {
            const bool there = n0 + lane < last;
            // lanes past the end hold the last digit, and do not count
            const unsigned digit = there ? (key_of(n0 + lane) >> shift) & (bins - 1) : bins - 1;
            const unsigned live = __ballot_sync(0xffffffffu, there);
            const unsigned peers = same_digit(digit, a.bits) & live;
            if (there && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        uint32_t *totals = a.totals + (static_cast<size_t>(p) * kSortCtas) * kSortBins;
        for (int j = threadIdx.x; j < bins; j += blockDim.x) {  // a digit's count, and each warp's share before it
            uint32_t t = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = count[w * row + j];
                count[w * row + j] = t;
                t += c;
            }
            totals[rank * kSortBins + j] = t;
        }
        cluster_barrier();
        if (threadIdx.x < bins) {  // whole warps: bins is 32 at least
            uint32_t all = 0, before = 0;
            for (unsigned r = 0; r < kSortCtas; ++r) {
                const uint32_t t = __ldcg(totals + r * kSortBins + threadIdx.x);
                before += r < rank ? t : 0;
                all += t;
            }
            uint32_t incl = all;
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl += o;
            }
            if (lane == 31) sums[warp] = incl;
            base[threadIdx.x] = incl - all + before;
        }
        __syncthreads();
        if (threadIdx.x < bins) {
            uint32_t add = 0;
            for (int w = 0; w < warp; ++w) add += sums[w];
            base[threadIdx.x] += add;
        }
        __syncthreads();
        for (long long n0 = first; n0 < last; n0 += 32) {
            const bool there = n0 + lane < last;
            const uint32_t key = there ? key_of(n0 + lane) : 0;
            const unsigned digit = there ? (key >> shift) & (bins - 1) : bins - 1;
            const unsigned live = __ballot_sync(0xffffffffu, there);
            const unsigned peers = same_digit(digit, a.bits) & live;
            if (there) {
                const uint32_t at = base[digit] + mine[digit] + __popc(peers & ((1u << lane) - 1u));
                kout[at] = key;
                vout[at] = p > 0 ? vin[n0 + lane] : static_cast<uint32_t>(n0 + lane);
                if (p + 1 == a.passes && key < a.V) a.present[key] = 1;
            }
            __syncwarp();
            if (there && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
            __syncwarp();
        }
        cluster_barrier();  // the tokens are where the next pass reads them
    }
}

template <class O, int V>
__device__ __forceinline__ void put_row(const EmbedArgs &a, long long id, long long d, float (&x)[V]) {
    O *to = static_cast<O *>(a.out) + id * a.D + d;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] *= a.scale;
    if (a.add) {
        float y[V];
        if constexpr (V == 8 && std::is_same<O, float>::value) {
            float u[4], w[4];
            unpack_lanes<O, 4>(to, u);
            unpack_lanes<O, 4>(to + 4, w);
#pragma unroll
            for (int v = 0; v < 4; ++v) { y[v] = u[v]; y[v + 4] = w[v]; }
        } else {
            unpack_lanes<O, V>(to, y);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] += y[v];
    }
    store_lanes<O, V>(to, x);
}

constexpr int kSumAhead = 8;     // rows in flight a thread
constexpr int kMostPer = 32;     // most sorted tokens a CTA sums
constexpr int kZeroRows = 32;    // rows of the table a zeroing CTA looks at

template <class G, class O, int V> __global__ void __launch_bounds__(512) embed_sum_kernel(const EmbedArgs a, int blocks) {
    const long long d = (static_cast<long long>(blockIdx.y) * blockDim.x + threadIdx.x) * V;
    if (blockIdx.x >= blocks) {  // rows without a token
        if (d >= a.D) return;
        const long long v0 = static_cast<long long>(blockIdx.x - blocks) * kZeroRows;
        float zero[V];
#pragma unroll
        for (int v = 0; v < V; ++v) zero[v] = 0.0f;
        for (int r = 0; r < kZeroRows && v0 + r < a.V; ++r)
            if (!a.present[v0 + r]) store_lanes<O, V>(static_cast<O *>(a.out) + (v0 + r) * a.D + d, zero);
        return;
    }
    __shared__ uint32_t key[kMostPer + 2], val[kMostPer];
    const uint32_t *keys = a.passes & 1 ? a.keys[1] : a.keys[0], *vals = a.passes & 1 ? a.vals[1] : a.vals[0];
    const uint32_t none = static_cast<uint32_t>(a.V);
    const long long j0 = static_cast<long long>(blockIdx.x) * a.per;
    const int n = static_cast<int>(a.N - j0 < a.per ? a.N - j0 : a.per);
    for (int j = threadIdx.x; j < n + 2; j += blockDim.x) {  // and the ids on both sides
        const long long at = j0 + j - 1;
        key[j] = at >= 0 && at < a.N ? keys[at] : none;
        if (j < n) val[j] = vals[j0 + j];
    }
    __syncthreads();
    if (d >= a.D) return;
    const G *rows = static_cast<const G *>(a.in) + d;
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;
    bool opened = key[0] != key[1];  // the current id starts in this stretch
    for (int i0 = 0; i0 < n; i0 += kSumAhead) {
        typename RawOf<G, std::is_same<G, float>::value && V == 8 ? 4 : V>::T raw[kSumAhead][std::is_same<G, float>::value && V == 8 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) {
            if (i0 + i < n && key[i0 + i + 1] != none) {
                const G *p = rows + static_cast<long long>(val[i0 + i]) * a.D;
                if constexpr (std::is_same<G, float>::value && V == 8) {
                    raw[i][0] = load_raw<G, 4>(p);
                    raw[i][1] = load_raw<G, 4>(p + 4);
                } else {
                    raw[i][0] = load_raw<G, V>(p);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) {
            if (i0 + i >= n) break;
            const uint32_t id = key[i0 + i + 1];
            if (id == none) return;  // the tokens that are none come last
            float x[V];
            if constexpr (std::is_same<G, float>::value && V == 8) {
                float u[4], w[4];
                widen_raw(raw[i][0], u);
                widen_raw(raw[i][1], w);
#pragma unroll
                for (int v = 0; v < 4; ++v) { x[v] = u[v]; x[v + 4] = w[v]; }
            } else {
                widen_raw(raw[i][0], x);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] += x[v];
            const bool ends = key[i0 + i + 2] != id;
            if (!ends && i0 + i + 1 < n) continue;
            if (ends && opened) {
                put_row<O, V>(a, id, d, sum);
            } else {  // goes on before (slot 0) or only after (slot 1) this stretch
                float *to = a.part + (static_cast<long long>(blockIdx.x) * 2 + (opened ? 1 : 0)) * a.D + d;
#pragma unroll
                for (int v = 0; v < V; ++v) to[v] = sum[v];
            }
            opened = true;
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] = 0.0f;
        }
    }
}

// An id that starts in stretch `blockIdx.x` and goes on in others: 32 columns a
// CTA, whose eight warps take every eighth stretch.
template <class O> __global__ void __launch_bounds__(256) embed_join_kernel(const EmbedArgs a) {
    __shared__ float sums[8][33];
    const uint32_t *keys = a.passes & 1 ? a.keys[1] : a.keys[0];
    const long long j1 = (static_cast<long long>(blockIdx.x) + 1) * a.per;  // the next stretch
    if (j1 >= a.N) return;
    const uint32_t id = keys[j1];
    if (id >= a.V || keys[j1 - 1] != id) return;
    const long long j0 = j1 - a.per;
    if (keys[j0] == id && j0 > 0 && keys[j0 - 1] == id) return;  // starts earlier
    // the last stretch that holds the id, by bisection of the stretches' first ids
    long long lo = blockIdx.x + 1, hi = (a.N + a.per - 1) / a.per;  // keys[lo * per] is the id, keys[hi * per] is not
    while (hi - lo > 1) {
        const long long mid = (lo + hi) / 2;
        if (keys[mid * a.per] == id)
            lo = mid;
        else
            hi = mid;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long d = static_cast<long long>(blockIdx.y) * 32 + lane;
    float sum = 0.0f;
    if (d < a.D) {
        if (warp == 0) sum = a.part[(static_cast<long long>(blockIdx.x) * 2 + 1) * a.D + d];
#pragma unroll 8
        for (long long j = blockIdx.x + 1 + warp; j <= lo; j += 8) sum += a.part[j * 2 * a.D + d];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && d < a.D) {
        float x[1] = {0.0f};
#pragma unroll
        for (int w = 0; w < 8; ++w) x[0] += sums[w][lane];
        put_row<O, 1>(a, id, d, x);
    }
}

}  // namespace lrscan
