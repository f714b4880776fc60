// Linear layers with their epilogue, forward and backward: tiles of 32 x 32 outputs in shared
// memory, one fp32 multiply-add a product.
#include "act.cuh"
#include "common.cuh"
#include "kernels.h"

#include <cuda_fp8.h>

namespace attn {
namespace {

constexpr int TILE = 32;

__device__ __forceinline__ float bf(const void *p, size_t i)
{
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float e4m3(const void *p, size_t i)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t *>(p)[i], __NV_E4M3);
    return __half2float(__half(h));
}

// Element (m, c) of the [G, H, T, dk] view.
struct View {
    int H, T, dk;
    __device__ size_t at(long long m, int c) const
    {
        return (((size_t)(m / T) * H + c / dk) * T + m % T) * dk + c % dk;
    }
};

// C[r, c] = sum_k A(r, k) B(k, c), then store(r, c, sum).
template <class LA, class LB, class ST>
__device__ void gemm_tile(long long R, int C, long long KK, LA la, LB lb, ST store)
{
    __shared__ float sa[TILE][TILE + 1], sb[TILE][TILE + 1];
    const int tx = threadIdx.x % TILE, ty = threadIdx.x / TILE;   // 32 x 8 threads
    const long long ct = (C + TILE - 1) / TILE, r0 = blockIdx.x / ct * TILE;
    const int c0 = (int)(blockIdx.x % ct) * TILE;
    float acc[4] = {};
    for (long long k0 = 0; k0 < KK; k0 += TILE) {
        for (int j = 0; j < 4; ++j) {
            const int q = ty + 8 * j;
            sa[q][tx] = (r0 + q < R && k0 + tx < KK) ? la(r0 + q, k0 + tx) : 0.f;
            sb[q][tx] = (k0 + q < KK && c0 + tx < C) ? lb(k0 + q, c0 + tx) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < TILE; ++k)
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(sa[ty + 8 * j][k], sb[k][tx], acc[j]);
        __syncthreads();
    }
    for (int j = 0; j < 4; ++j)
        if (r0 + ty + 8 * j < R && c0 + tx < C) store(r0 + ty + 8 * j, c0 + tx, acc[j]);
}

__global__ void __launch_bounds__(256) linear_kernel(const LinArgs a)
{
    const View v{a.H, a.T, a.dk};
    gemm_tile(
        a.M, a.N, a.K,
        [&](long long m, long long k) { return a.q8 ? e4m3(a.x, m * a.K + k) : bf(a.x, v.at(m, (int)k)); },
        [&](long long k, int n) { return a.q8 ? e4m3(a.w, (size_t)n * a.K + k) : bf(a.w, (size_t)k * a.N + n); },
        [&](long long m, int n, float z) {
            const size_t i = (size_t)m * a.N + n;
            if (a.q8) z *= a.x_scale[m] * a.w_scale[n];
            if (a.bias) z += a.bias[n];
            if (a.z) static_cast<__nv_bfloat16 *>(a.z)[i] = __float2bfloat16(z);
            float y = activate(z, a.act);
            if (a.residual) y += bf(a.residual, i);
            static_cast<__nv_bfloat16 *>(a.y)[i] = __float2bfloat16(y);
        });
}

__global__ void __launch_bounds__(256) linear_dx_kernel(const LinBwdArgs a, const void *dz)
{
    const View v{a.H, a.T, a.dk};
    gemm_tile(
        a.M, a.K, a.N, [&](long long m, long long n) { return bf(dz, (size_t)m * a.N + n); },
        [&](long long n, int k) { return bf(a.w, (size_t)k * a.N + n); },
        [&](long long m, int k, float s) { static_cast<__nv_bfloat16 *>(a.dx)[v.at(m, k)] = __float2bfloat16(s); });
}

__global__ void __launch_bounds__(256) linear_dw_kernel(const LinBwdArgs a, const void *dz)
{
    const View v{a.H, a.T, a.dk};
    gemm_tile(
        a.K, a.N, a.M, [&](long long k, long long m) { return bf(a.x, v.at(m, (int)k)); },
        [&](long long m, int n) { return bf(dz, (size_t)m * a.N + n); },
        [&](long long k, int n, float s) {
            static_cast<__nv_bfloat16 *>(a.dw)[(size_t)k * a.N + n] = __float2bfloat16(s);
        });
}

// dz = dy act'(z) and its column sums over a block of rows, one thread a column.
__global__ void linear_dz_kernel(const LinBwdArgs a, int blocks)
{
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= a.N) return;
    float s = 0.f;
    for (long long m = blockIdx.y; m < a.M; m += blocks) {
        const size_t i = (size_t)m * a.N + n;
        float d = bf(a.dy, i);
        if (a.z) {
            d *= act_slope(bf(a.z, i), a.act);
            static_cast<__nv_bfloat16 *>(a.dz)[i] = __float2bfloat16(d);
        }
        s += d;
    }
    a.col_part[(size_t)blockIdx.y * a.N + n] = s;
}

__global__ void col_sum_kernel(const float *part, float *out, int blocks, int N)
{
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[(size_t)b * N + n];
    out[n] = s;
}

unsigned tiles(long long R, long long C) { return (unsigned)((R + TILE - 1) / TILE * ((C + TILE - 1) / TILE)); }

}  // namespace

cudaError_t launch_linear(const LinArgs &a, cudaStream_t stream)
{
    linear_kernel<<<tiles(a.M, a.N), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

int lin_bwd_row_blocks(int M, int) { return M < 128 ? (M > 0 ? M : 1) : 128; }
int lin_dw_splits(int, int, int, int) { return 1; }

cudaError_t launch_linear_bwd(const LinBwdArgs &a, cudaStream_t stream)
{
    const int blocks = lin_bwd_row_blocks(a.M, a.N);
    if (a.z || a.dbias) linear_dz_kernel<<<dim3((a.N + 127) / 128, blocks), 128, 0, stream>>>(a, blocks);
    if (a.dbias) col_sum_kernel<<<(a.N + 127) / 128, 128, 0, stream>>>(a.col_part, a.dbias, blocks, a.N);
    const void *dz = a.z ? a.dz : a.dy;
    if (a.dx) linear_dx_kernel<<<tiles(a.M, a.K), 256, 0, stream>>>(a, dz);
    if (a.dw) linear_dw_kernel<<<tiles(a.K, a.N), 256, 0, stream>>>(a, dz);
    return cudaGetLastError();
}

}  // namespace attn
