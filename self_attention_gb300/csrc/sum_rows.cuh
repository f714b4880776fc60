// Sums of the rows of an fp32 matrix, for the joins of partial sums: out[c] = sum over r of part[r][c], in a
// fixed order.
#pragma once

namespace attn {

constexpr int kSumCols = 4;   // columns a block of 256 threads

// Columns c..c+3 by a block: 64 lanes of rows take every 64th row, five at a time in flight, then a warp adds
// a column's 64 sums up.  Bound by latency: with 32 columns a block and 8 lanes the join of 304 rows of 768
// columns beside dw's took 8.4 us, so 4.0.
__device__ __forceinline__ void sum_columns(const float *part, float *out, int rows, int cols, int c)
{
    __shared__ float sums[64 * 5];
    const int in = threadIdx.x & 3, from = threadIdx.x >> 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s = 0.f;
    for (int r = from; r < rows; r += 5 * 64) {
        float v[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) v[k] = r + k * 64 < rows ? part[(size_t)(r + k * 64) * cols + c + in] : 0.f;
#pragma unroll
        for (int k = 0; k < 5; ++k) s += v[k];
    }
    sums[from * 5 + in] = s;
    __syncthreads();
    if (warp >= kSumCols) return;
    s = sums[lane * 5 + warp] + sums[(lane + 32) * 5 + warp];   // column `warp`, its 64 sums over the lanes
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) out[c + warp] = s;
}

}  // namespace attn
