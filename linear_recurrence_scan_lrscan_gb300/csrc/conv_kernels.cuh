// The short causal convolution of each channel:
//
//   y_t = bias + sum_{k < K} w[K-1-k] x_{t-k}
//
// a tap counting only where no segment starts in t-k+1 .. t (tokens before
// token 0 are x0, or zeros).  Backward: grad_x_t = sum_k w[K-1-k] grad_out_{t+k}
// over the same pairs of tokens, grad_w[K-1-k] = sum grad_out_t x_{t-k},
// grad_bias = sum grad_out_t.
//
// A thread walks kConvSteps tokens of V lanes with the last K - 1 tokens in
// registers, so that HBM carries each element once (the tokens that two walks
// share come from L2); a warp covers 32 V neighbouring lanes, a CTA
// kConvSplit walks one after another in time.  `run` counts the tokens before
// t that are in t's segment.
#pragma once

#include "conv_args.h"
#include "scan_common.cuh"

namespace lrscan {

// Tokens read ahead by a walk.
constexpr int kConvAhead = 8;

template <class St, int V> __device__ __forceinline__ void conv_load(const St *p, bool in, float (&x)[V]) {
    if (in) {
        load_lanes_global<St, V>(p, x);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = 0.0f;
    }
}

template <class St, int V>
__device__ __forceinline__ typename RawOf<St, V>::T conv_raw(const St *p, bool in) {
    typename RawOf<St, V>::T r{};
    if (in) r = load_raw<St, V>(p);
    return r;
}

// x at token t, which may be before token 0.
template <class St, int V, int K>
__device__ __forceinline__ void conv_token(const ConvArgs &a, long long b, long long t, long long d, bool in,
                                           float (&x)[V]) {
    if (t >= 0)
        conv_load<St, V>(static_cast<const St *>(a.x.p) + b * a.x.sb + t * a.x.st + d, in, x);
    else
        conv_load<St, V>(static_cast<const St *>(a.x0) + (b * (K - 1) + t + (K - 1)) * a.D + d, in && a.x0 != nullptr, x);
}

template <class St, int V, int K> __global__ void __launch_bounds__(32 * kConvSplit) conv_fwd_kernel(const ConvArgs a) {
    const unsigned lanes = blockIdx.x % a.ndt, chunk = blockIdx.x / a.ndt;
    const long long b = blockIdx.y;
    const long long d = (static_cast<long long>(lanes) * 32 + threadIdx.x) * V;
    const long long t0 = (static_cast<long long>(chunk) * kConvSplit + threadIdx.y) * kConvSteps;
    if (d >= a.D || t0 >= a.T) return;
    const int n = static_cast<int>(a.T - t0 < kConvSteps ? a.T - t0 : kConvSteps);
    float w[K][V], bias[V], hist[K - 1][V];  // hist[k]: x_{t-1-k}; w[k]: the tap of x_{t-k}
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][v] = __ldg(a.w + (d + v) * K + (K - 1 - k));
        bias[v] = a.bias ? __ldg(a.bias + d + v) : 0.0f;
    }
    const int32_t *seg = a.seg ? a.seg + b * a.T : nullptr;
    int run = K - 1;
#pragma unroll
    for (int k = K - 2; k >= 0; --k) {
        const long long t = t0 - 1 - k;
        conv_token<St, V, K>(a, b, t, d, true, hist[k]);
        run = seg && t >= 0 && __ldg(seg + t) == 0 ? 0 : (run < K - 1 ? run + 1 : K - 1);
    }
    const St *xp = static_cast<const St *>(a.x.p) + b * a.x.sb + t0 * a.x.st + d;
    St *op = static_cast<St *>(a.o.p) + b * a.o.sb + t0 * a.o.st + d;
    for (int j0 = 0; j0 < n; j0 += kConvAhead) {
        typename RawOf<St, V>::T xr[kConvAhead];
        int first[kConvAhead];
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
            xr[j] = conv_raw<St, V>(xp + (j0 + j) * a.x.st, j0 + j < n);
            first[j] = seg && j0 + j < n ? __ldg(seg + t0 + j0 + j) : 1;
        }
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
            if (j0 + j >= n) break;
            run = first[j] == 0 ? 0 : (run < K - 1 ? run + 1 : K - 1);
            float x[V], y[V];
            widen_raw(xr[j], x);
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = __fmaf_rn(w[0][v], x[v], bias[v]);
#pragma unroll
            for (int k = 1; k < K; ++k)
                if (k <= run)
#pragma unroll
                    for (int v = 0; v < V; ++v) y[v] = __fmaf_rn(w[k][v], hist[k - 1][v], y[v]);
            store_lanes<St, V>(op + (j0 + j) * a.o.st, y);
#pragma unroll
            for (int k = K - 2; k > 0; --k)
#pragma unroll
                for (int v = 0; v < V; ++v) hist[k][v] = hist[k - 1][v];
#pragma unroll
            for (int v = 0; v < V; ++v) hist[0][v] = x[v];
        }
    }
    if (a.last != nullptr && t0 + n == a.T) {
        St *to = static_cast<St *>(a.last) + b * (K - 1) * a.D + d;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) store_lanes<St, V>(to + (K - 2 - k) * a.D, hist[k]);
    }
}

// A walk adds grad_out_t's part to the gradients of tokens t .. t-K+1, which it
// holds until they are complete; it reads K - 1 tokens of grad_out past its
// own for them.  The walk at token 0 holds the tokens of x0 too.
template <class St, int V, int K> __global__ void __launch_bounds__(32 * kConvSplit, 2) conv_bwd_kernel(const ConvArgs a) {
    __shared__ float sums[kConvSplit][K + 1][32 * V];
    const unsigned lanes = blockIdx.x % a.ndt, chunk = blockIdx.x / a.ndt;
    const long long b = blockIdx.y;
    const long long d = (static_cast<long long>(lanes) * 32 + threadIdx.x) * V;
    const long long t0 = (static_cast<long long>(chunk) * kConvSplit + threadIdx.y) * kConvSteps;
    const bool in = d < a.D;
    float gw[K][V], gb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        gb[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) gw[k][v] = 0.0f;
    }
    if (in && t0 < a.T) {
        const int n = static_cast<int>(a.T - t0 < kConvSteps ? a.T - t0 : kConvSteps);
        float w[K][V], hist[K - 1][V], held[K][V];  // held[k]: gradient of token t-k so far
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][v] = __ldg(a.w + (d + v) * K + (K - 1 - k));
        const int32_t *seg = a.seg ? a.seg + b * a.T : nullptr;
        const St *gl = static_cast<const St *>(a.grad_last) + b * (K - 1) * a.D + d;
        const long long tail = a.T - (K - 1);  // the first token of `last`
        int run = K - 1;
#pragma unroll
        for (int k = K - 2; k >= 0; --k) {
            const long long t = t0 - 1 - k;
            conv_token<St, V, K>(a, b, t, d, true, hist[k]);
            run = seg && t >= 0 && __ldg(seg + t) == 0 ? 0 : (run < K - 1 ? run + 1 : K - 1);
            // tokens before token 0 that are still among the last ones
            conv_load<St, V>(gl + (t - tail) * a.D, a.grad_last != nullptr && t < 0 && t >= tail, held[k]);
        }
        const St *xp = static_cast<const St *>(a.x.p) + b * a.x.sb + t0 * a.x.st + d;
        const St *gp = static_cast<const St *>(a.go.p) + b * a.go.sb + t0 * a.go.st + d;
        St *op = static_cast<St *>(a.o.p) + b * a.o.sb + d;
        St *o0 = static_cast<St *>(a.grad_x0) + b * (K - 1) * a.D + d;
        const long long left = a.T - t0;
        for (int j0 = 0; j0 < n + K - 1; j0 += kConvAhead) {
            typename RawOf<St, V>::T xr[kConvAhead], gr[kConvAhead];
            int first[kConvAhead];
#pragma unroll
            for (int j = 0; j < kConvAhead; ++j) {
                const bool there = j0 + j < n + K - 1 && j0 + j < left;
                xr[j] = conv_raw<St, V>(xp + (j0 + j) * a.x.st, j0 + j < n);
                gr[j] = conv_raw<St, V>(gp + (j0 + j) * a.go.st, there);
                first[j] = seg && there ? __ldg(seg + t0 + j0 + j) : 1;
            }
#pragma unroll
            for (int j = 0; j < kConvAhead; ++j) {
                if (j0 + j >= n + K - 1) break;
                const long long t = t0 + j0 + j;
                float x[V], g[V];
                widen_raw(xr[j], x);
                widen_raw(gr[j], g);
                run = first[j] == 0 ? 0 : (run < K - 1 ? run + 1 : K - 1);
#pragma unroll
                for (int k = K - 1; k > 0; --k)
#pragma unroll
                    for (int v = 0; v < V; ++v) held[k][v] = held[k - 1][v];
                conv_load<St, V>(gl + (t - tail) * a.D, a.grad_last != nullptr && t < a.T && t >= tail, held[0]);
                if (t < a.T) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (k == 0 || k <= run)
#pragma unroll
                            for (int v = 0; v < V; ++v) held[k][v] = __fmaf_rn(w[k][v], g[v], held[k][v]);
                    if (j0 + j < n) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            gb[v] += g[v];
                            gw[0][v] = __fmaf_rn(g[v], x[v], gw[0][v]);
                        }
#pragma unroll
                        for (int k = 1; k < K; ++k)
                            if (k <= run)
#pragma unroll
                                for (int v = 0; v < V; ++v) gw[k][v] = __fmaf_rn(g[v], hist[k - 1][v], gw[k][v]);
#pragma unroll
                        for (int k = K - 2; k > 0; --k)
#pragma unroll
                            for (int v = 0; v < V; ++v) hist[k][v] = hist[k - 1][v];
#pragma unroll
                        for (int v = 0; v < V; ++v) hist[0][v] = x[v];
                    }
                }
                const long long done = t - (K - 1);  // complete now
                if (done >= t0)
                    store_lanes<St, V>(op + done * a.o.st, held[K - 1]);
                else if (done < 0 && a.grad_x0 != nullptr && done >= -(K - 1))
                    store_lanes<St, V>(o0 + (done + (K - 1)) * a.D, held[K - 1]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) sums[threadIdx.y][K - 1 - k][threadIdx.x + 32 * v] = gw[k][v];
        sums[threadIdx.y][K][threadIdx.x + 32 * v] = gb[v];
    }
    __syncthreads();
    float *part = a.part + (b * a.chunks + chunk) * (K + 1) * a.D;
    const int me = threadIdx.y * 32 + threadIdx.x;
    for (int j = me; j < (K + 1) * 32 * V; j += 32 * kConvSplit) {
        const int row = j / (32 * V), lane = j % (32 * V);  // lane: in the order of the channels
        float sum = 0.0f;
#pragma unroll
        for (int y = 0; y < kConvSplit; ++y) sum += sums[y][row][lane / V + 32 * (lane % V)];
        const long long at = static_cast<long long>(lanes) * 32 * V + lane;
        if (at < a.D) part[row * a.D + at] = sum;
    }
}

template <class St, int K> __global__ void __launch_bounds__(256) conv_step_kernel(const ConvStep g) {
    const long long d = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (d >= g.D) return;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = __ldg(g.w + d * K + k);
    const float bias = g.bias ? __ldg(g.bias + d) : 0.0f;
    for (long long b = blockIdx.y; b < g.B; b += gridDim.y) {
        const long long slot = g.slots ? __ldg(g.slots + b) : b;
        float y[1] = {0.0f};
        if (slot >= 0 && slot < g.S) {
            St *win = static_cast<St *>(g.state) + slot * (K - 1) * g.D + d;
            St before[K - 1], now = static_cast<const St *>(g.x)[b * g.sx + d];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) before[k] = win[k * g.D];
            float x[1];
            unpack_lanes<St, 1>(&now, x);
            y[0] = __fmaf_rn(w[K - 1], x[0], bias);
#pragma unroll
            for (int k = K - 2; k >= 0; --k) {
                unpack_lanes<St, 1>(&before[k], x);
                y[0] = __fmaf_rn(w[k], x[0], y[0]);
            }
#pragma unroll
            for (int k = 0; k + 1 < K - 1; ++k) win[k * g.D] = before[k + 1];
            win[(K - 2) * g.D] = now;
        } else if (slot >= g.S && threadIdx.x == 0 && blockIdx.x == 0) {
            if (atomicCAS(&g.status->code, 0, kErrRange) == 0) {
                g.status->where = kSiteConvSlot;
                g.status->block = static_cast<unsigned>(b);
            }
        }
        store_lanes<St, 1>(static_cast<St *>(g.out) + b * g.so + d, y);
    }
}

}  // namespace lrscan
