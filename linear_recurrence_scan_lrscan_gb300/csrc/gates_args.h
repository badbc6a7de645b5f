// Arguments of the gated-recurrence kernels (gates_kernels.cuh) that the host
// side fills in (layer_abi.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lrscan {

struct DevStatus;

constexpr int kErrRange = -1;          // == LRSCAN_EINVAL: a slot or an id out of range, found on the device
enum RangeSite : int { kSiteGatesSlot = 30, kSiteConvSlot = 31, kSiteEmbedId = 32 };

// A [B, T, D] tensor whose D elements of one token are contiguous: strides of
// a batch row and of a token, in elements.
struct RowsArg {
    void *p;
    long long sb, st;
};

constexpr int kGatesSave = 16;    // tokens between saved states
constexpr int kGatesRadix = 16;   // tiles a level of the tree of maps joins
constexpr int kGatesLanes = 64;   // lanes of a tile

struct GatesArgs {
    RowsArg r, i, x;              // gates before their sigmoid, input
    RowsArg go;                   // backward: grad_out
    RowsArg o0, o1, o2;           // forward: out; backward: grad_r, grad_i, grad_x
    const float *lam;             // [D]
    float c;
    const float *rate;            // [D] c softplus(lam), or null: computed where it is used
    const float *h0;              // forward: [B, D] or null
    const float *grad_last;       // backward: [B, D] or null
    float *edge;                  // [B, D] or null: forward `last`, backward `grad_h0`
    float *saved;                 // [B, ceil(T / kGatesSave), D]; forward output or null, backward input
    const int32_t *seg;           // [B, T] or null
    float *part;                  // backward: [NC * B][D] partial sums of the lam gradient
    long long B, T, D;
    int ndt;                      // lane tiles of a batch row
    int nl;                       // B * ndt
    int nc;                       // time tiles
    unsigned int *ticket;         // all-ones before the launch (nc > 1)
    uint64_t *agg1, *agg2, *agg3; // maps of a tile, of kGatesRadix tiles; states after kGatesRadix^2 tiles
    DevStatus *status;
    uint64_t timeout_ns;
};

struct GatesLaunch {
    GatesArgs a;
    CUtensorMap maps[4];          // r, i, x, grad_out (bulk-copied form only)
    bool bulk;                    // rows fit bulk copies
    cudaStream_t stream;
};

constexpr int kGatesTileRows = 64;  // tokens of a tile
int gates_launch(const GatesLaunch &L, int dtype, int dir, int sm_count);
// Sets the bytes (of a multiple of 16) at `words` to all ones and the rates.
int gates_begin_launch(void *words, size_t bytes, const float *lam, float c, long long D, float *rate, int sm_count,
                       cudaStream_t stream);
// grad_lam from the partial sums part [rows][D], in a fixed order; `part` has
// gates_finish_slices(rows) more rows after them.
int gates_finish_slices(long long rows);
int gates_finish_launch(float *part, long long rows, long long D, const float *lam, float *grad_lam,
                        cudaStream_t stream);
// One token a row: state [S, D] in place; slots may be null.
struct GatesStep {
    const void *r, *i, *x;
    long long sr, si, sx, so;     // row strides in elements
    void *out;
    const float *lam;
    float c;
    float *state;
    const int32_t *slots;
    long long S, B, D;
    DevStatus *status;
    cudaStream_t stream;
};
int gates_step_launch(const GatesStep &L, int dtype);

}  // namespace lrscan
