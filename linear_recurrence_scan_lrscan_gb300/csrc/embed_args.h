// Arguments of the token-embedding kernels (embed_kernels.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gates_args.h"

namespace lrscan {

struct EmbedArgs {
    const void *ids;      // [N] int32 or int64
    bool wide;            // int64
    const void *in;       // forward: weight [V, D]; backward: grad_out [N, D]
    void *out;            // forward: [N, D]; backward: grad_weight [V, D]
    float scale;
    bool add;             // backward: add to grad_weight
    bool vec;             // rows fit accesses of eight lanes
    long long N, V, D;
    DevStatus *status;
    cudaStream_t stream;
    int sm_count;
    // backward scratch
    uint32_t *keys[2], *vals[2];  // [N]: token ids (V: none) and token numbers
    int *runs;                    // long runs, and where each starts [N / kLongRun]
    uint32_t *run_at;
    float *part;                  // [blocks][2][D]
    int bits;                     // of a digit
    int passes;
    int per;                      // sorted tokens of a stretch
    int zeros;                    // CTAs of the second kernel that write zeros
    int held;                     // tokens of a CTA that the sort keeps on chip, or 0
};

constexpr int kSortCtas = 8;      // one cluster
constexpr int kSortWarps = 32;
constexpr int kSortBits = 9;      // most bits of a digit
constexpr int kSortBins = 1 << kSortBits;
constexpr int kLongRun = 32;      // a run of more tokens than this is shared

int embed_fwd_launch(const EmbedArgs &a, int wdtype, int odtype);
int embed_bwd_launch(const EmbedArgs &a, int gdtype, int wdtype);

}  // namespace lrscan
