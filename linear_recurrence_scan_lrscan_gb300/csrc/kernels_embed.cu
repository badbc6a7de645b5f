// Launchers of the token-embedding kernels.
#include "embed_args.h"
#include "embed_kernels.cuh"
#include "launch.h"

namespace lrscan {
namespace {

template <class W, class O, int V> int fwd(const EmbedArgs &a) {
    const long long nd = (a.D + 32 * V - 1) / (32 * V);
    const dim3 block(32, 8);
    // several rows a thread once the rows alone keep the SMs busy
    const long long few = (a.N + 7) / 8 * nd, many = (a.N + 8 * kRowsPerThread - 1) / (8 * kRowsPerThread) * nd;
    if (many >= 4LL * a.sm_count) {
        if (many > 0x7fffffffLL) return 1;
        embed_fwd_kernel<W, O, V, kRowsPerThread><<<static_cast<unsigned>(many), block, 0, a.stream>>>(a);
    } else {
        embed_fwd_kernel<W, O, V, 1><<<static_cast<unsigned>(few), block, 0, a.stream>>>(a);
    }
    return cudaGetLastError() != cudaSuccess;
}

template <class G, class O, int V> int sums(const EmbedArgs &a) {
    const long long lanes = (a.D + V - 1) / V;
    const int threads = static_cast<int>(lanes >= 512 ? 512 : (lanes + 31) / 32 * 32);
    const long long blocks = (a.N + a.per - 1) / a.per, zero = a.add ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
    const long long ny = (lanes + threads - 1) / threads;
    if (blocks + zero > 0x7fffffffLL || ny > 65535) return 1;
    embed_sum_kernel<G, O, V><<<dim3(static_cast<unsigned>(blocks + zero), static_cast<unsigned>(ny)), threads, 0,
                                a.stream>>>(a, static_cast<int>(blocks));
    if (cudaGetLastError() != cudaSuccess) return 1;
    if (blocks < 2) return 0;
    embed_join_kernel<O><<<dim3(static_cast<unsigned>(blocks - 1), static_cast<unsigned>((a.D + 31) / 32)), 256, 0,
                           a.stream>>>(a);
    return cudaGetLastError() != cudaSuccess;
}

template <class G, class O> int bwd(const EmbedArgs &a) {
    const int smem = kSortWarps * ((1 << a.bits) + 1) * 4;
    static bool allowed[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    if (!allowed[dev]) {
        if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSortWarps * (kSortBins + 1) * 4) != cudaSuccess)
            return 1;
        allowed[dev] = true;
    }
    embed_sort_kernel<<<kSortCtas, kSortWarps * 32, smem, a.stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return 1;
    return a.vec ? sums<G, O, 8>(a) : sums<G, O, 1>(a);
}

}  // namespace

int embed_fwd_launch(const EmbedArgs &a, int wdtype, int odtype) {
    if (wdtype == 0 && odtype == 0) return a.vec ? fwd<float, float, 8>(a) : fwd<float, float, 1>(a);
    if (wdtype == 0) return a.vec ? fwd<float, bf16_t, 8>(a) : fwd<float, bf16_t, 1>(a);
    if (odtype == 0) return a.vec ? fwd<bf16_t, float, 8>(a) : fwd<bf16_t, float, 1>(a);
    return a.vec ? fwd<bf16_t, bf16_t, 8>(a) : fwd<bf16_t, bf16_t, 1>(a);
}

int embed_bwd_launch(const EmbedArgs &a, int gdtype, int wdtype) {
    if (gdtype == 0 && wdtype == 0) return bwd<float, float>(a);
    if (gdtype == 0) return bwd<float, bf16_t>(a);
    if (wdtype == 0) return bwd<bf16_t, float>(a);
    return bwd<bf16_t, bf16_t>(a);
}

}  // namespace lrscan
