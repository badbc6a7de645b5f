// Column sums of an fp32 matrix part [rows][cols] in a fixed order, for the
// kernels that leave one row of partial sums a tile: a CTA takes 32 columns,
// its 32 warps every 32nd row of the CTA's slice of rows, and their sums are
// added in warp order.  Many rows are cut in slices, whose sums take the rows
// after the matrix and are then summed alike.  Eight loads in flight a thread, and a
// slice for every 256 rows; latency bounds it, and each of its one or two launches
// begins while the kernel before ends.
#pragma once

#include <cuda_runtime.h>

#include "launch.h"
#include "scan_common.cuh"

namespace lrscan {

template <class Put>
__global__ void __launch_bounds__(1024) column_sums_kernel(const float *part, long long rows, long long cols, Put put) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long d = static_cast<long long>(blockIdx.x) * 32 + lane;
    const long long per = (rows + gridDim.y - 1) / gridDim.y;
    const long long r0 = per * blockIdx.y, r1 = r0 + per < rows ? r0 + per : rows;
    float sum = 0.0f;
    pdl_wait();
    pdl_trigger();
    if (d < cols) {
#pragma unroll 8
        for (long long r = r0 + warp; r < r1; r += 32) sum += __ldg(part + r * cols + d);
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && d < cols) {
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) sum += sums[w][lane];
        put(blockIdx.y, d, sum);
    }
}

struct PutSlice {
    float *to;
    long long cols;
    __device__ void operator()(long long slice, long long d, float sum) const { to[slice * cols + d] = sum; }
};

// Rows past the matrix that `part` has to have room for.
inline int column_slices(long long rows) {
    const long long s = rows / 256;
    return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <class Put> int column_sums(float *part, long long rows, long long cols, const Put &put, cudaStream_t st) {
    const int slices = column_slices(rows);
    const unsigned x = static_cast<unsigned>((cols + 31) / 32);
    cudaError_t e = cudaSuccess;
    if (slices > 1) {
        float *second = part + rows * cols;
        e = launch_pdl(column_sums_kernel<PutSlice>, dim3(x, slices), dim3(1024), 0, st, part, rows, cols,
                       PutSlice{second, cols});
        part = second;
        rows = slices;
    }
    if (e == cudaSuccess) e = launch_pdl(column_sums_kernel<Put>, dim3(x, 1), dim3(1024), 0, st, part, rows, cols, put);
    return e != cudaSuccess;
}

}  // namespace lrscan
