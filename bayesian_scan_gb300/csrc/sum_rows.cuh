// sum_rows.cuh -- column sums of an fp32 matrix in a fixed order: the last
// step of the gradients that every block of a backward pass has a share of.
#pragma once
#include <cuda_runtime.h>

namespace kdn {
namespace {

constexpr int SUM_COLS = 32, SUM_GROUPS = 32;

// A block adds 32 columns: a warp takes every 32nd row, four loads at a time,
// then the warps' sums are added in order.  Columns below `split` go to
// `low`, the others to `high` (either may be null: not wanted).
__global__ void __launch_bounds__(SUM_COLS * SUM_GROUPS)
sum_rows_kernel(const float* __restrict__ m, long long rows, long long cols, float* __restrict__ low,
                float* __restrict__ high, long long split) {
    __shared__ float share[SUM_GROUPS][SUM_COLS + 1];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const long long c = static_cast<long long>(blockIdx.x) * SUM_COLS + lane;
    float s = 0.f;
    if (c < cols) {
        long long r = g;
        for (; r + 3 * SUM_GROUPS < rows; r += 4 * SUM_GROUPS) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = m[(r + i * SUM_GROUPS) * cols + c];
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += SUM_GROUPS) s += m[r * cols + c];
    }
    share[g][lane] = s;
    __syncthreads();
    // transposed: warp g adds column g, one warp's sum per lane
    s = share[lane][g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const long long k = static_cast<long long>(blockIdx.x) * SUM_COLS + g;
    if (lane == 0 && k < cols) {
        if (k < split) {
            if (low) low[k] = s;
        } else if (high) {
            high[k - split] = s;
        }
    }
}

inline cudaError_t sum_rows(const float* m, long long rows, long long cols, float* low, float* high, long long split,
                            cudaStream_t stream) {
    const long long blocks = (cols + SUM_COLS - 1) / SUM_COLS;
    sum_rows_kernel<<<static_cast<unsigned>(blocks), SUM_COLS * SUM_GROUPS, 0, stream>>>(m, rows, cols, low, high, split);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kdn
