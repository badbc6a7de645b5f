// Launchers of the token-embedding kernels.
#include "embed_args.h"
#include "embed_kernels.cuh"
#include "launch.h"

namespace lrscan {
namespace {

// Lanes of a thread where rows fit wide accesses: 16 bytes of the wider type, so
// that a warp's accesses have no gaps on either side.
template <class A, class B> constexpr int kWide = 16 / (sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B));

template <class W, class O, int V> int fwd(const EmbedArgs &a) {
    const long long nd = (a.D + 32 * V - 1) / (32 * V);
    const dim3 block(32, 8);
    // several rows a thread once the rows alone keep the SMs busy
    const long long few = (a.N + 7) / 8 * nd, many = (a.N + 8 * kRowsPerThread - 1) / (8 * kRowsPerThread) * nd;
    if (many > 0x7fffffffLL) return 1;
    const cudaError_t e =
        many >= 4LL * a.sm_count
            ? launch_pdl(embed_fwd_kernel<W, O, V, kRowsPerThread>, dim3(static_cast<unsigned>(many)), block, 0, a.stream, a)
            : launch_pdl(embed_fwd_kernel<W, O, V, 1>, dim3(static_cast<unsigned>(few)), block, 0, a.stream, a);
    return e != cudaSuccess;
}

template <class G, class O, int V> int bwd_vec(EmbedArgs a) {
    constexpr int kMost = 212 * 1024;  // beside 8 KB that are static
    int smem = kSortWarps * ((1 << a.bits) + 1) * 4;
    const long long stretch = ((a.N + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
    const long long held = stretch * kSortWarps;  // tokens of a CTA
    a.held = 0;
    if (a.passes > 1 && smem + held * 16 <= kMost) {
        a.held = static_cast<int>(held);
        smem += static_cast<int>(held * 16);
    }
    if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) return 1;
    if (launch_pdl(embed_sort_kernel, dim3(kSortCtas), dim3(kSortWarps * 32), smem, a.stream, a) != cudaSuccess) return 1;
    const long long lanes = (a.D + V - 1) / V;
    constexpr int U = V == 1 ? 4 : 1;
    const long long ny = (lanes + 512 * U - 1) / (512 * U);  // a row's lanes in equal parts
    const int threads = static_cast<int>(((lanes + U * ny - 1) / (U * ny) + 31) / 32 * 32);
    a.zeros = a.add ? 0 : 2 * a.sm_count;
    const long long blocks = a.zeros + (a.N + a.per - 1) / a.per;
    if (blocks > 0x7fffffffLL || ny > 65535) return 1;
    if (launch_pdl(embed_sum_kernel<G, O, V, U>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(ny)), dim3(threads), 0,
                   a.stream, a) != cudaSuccess)
        return 1;
    if (a.N <= kLongRun) return 0;
    return launch_pdl(embed_join_kernel<O, (V > 1 ? 4 : 1)>, dim3(8 * a.sm_count), dim3(256), 0, a.stream, a) != cudaSuccess;
}

template <class G, class O> int bwd(const EmbedArgs &a) { return a.vec ? bwd_vec<G, O, kWide<G, O>>(a) : bwd_vec<G, O, 1>(a); }

}  // namespace

int embed_fwd_launch(const EmbedArgs &a, int wdtype, int odtype) {
    if (wdtype == 0 && odtype == 0) return a.vec ? fwd<float, float, 16 / sizeof(float)>(a) : fwd<float, float, 1>(a);
    if (wdtype == 0) return a.vec ? fwd<float, bf16_t, 16 / sizeof(bf16_t)>(a) : fwd<float, bf16_t, 1>(a);
    if (odtype == 0) return a.vec ? fwd<bf16_t, float, 16 / sizeof(float)>(a) : fwd<bf16_t, float, 1>(a);
    return a.vec ? fwd<bf16_t, bf16_t, 16 / sizeof(bf16_t)>(a) : fwd<bf16_t, bf16_t, 1>(a);
}

int embed_bwd_launch(const EmbedArgs &a, int gdtype, int wdtype) {
    if (gdtype == 0 && wdtype == 0) return bwd<float, float>(a);
    if (gdtype == 0) return bwd<float, bf16_t>(a);
    if (wdtype == 0) return bwd<bf16_t, float>(a);
    return bwd<bf16_t, bf16_t>(a);
}

}  // namespace lrscan
