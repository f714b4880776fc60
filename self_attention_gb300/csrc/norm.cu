// Root-mean-square norm with the residual's addition, its 8-bit form and its backward.
#include "common.cuh"
#include "kernels.h"

#include <cuda_fp8.h>

namespace attn {
namespace {

constexpr float kQ8Max = 448.f;      // largest e4m3
constexpr float kAmaxFloor = 1e-30f;

__device__ __forceinline__ float bf(const void *p, size_t i)
{
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <bool MAX>
__device__ __forceinline__ float block_reduce(float v)
{
    __shared__ float part[32], all;
    __syncthreads();
    auto op = [](float a, float b) {
        float r;
        if (MAX)
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
        else
            r = a + b;
        return r;
    };
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = part[0];
        for (unsigned i = 1; i < blockDim.x / 32; ++i) t = op(t, part[i]);
        all = t;
    }
    __syncthreads();
    return all;
}

// One block a row.
__global__ void __launch_bounds__(256) rms_norm_kernel(const NormArgs a)
{
    for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t row = (size_t)m * a.D;
        auto h = [&](int d) { return bf(a.x, row + d) + (a.residual ? bf(a.residual, row + d) : 0.f); };
        float s = 0.f;
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) s += h(d) * h(d);
        const float rstd = a.weight ? 1.f / sqrtf(block_reduce<false>(s) / a.D + a.eps) : 1.f;
        auto y = [&](int d) { return a.weight ? h(d) * rstd * a.weight[d] : h(d); };
        float inv = 1.f;
        if (a.q8) {
            float t = 0.f;
            for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
                const float v = fabsf(y(d));
                asm("max.NaN.f32 %0, %1, %0;" : "+f"(t) : "f"(v));
            }
            t = block_reduce<true>(t);
            t = t < kAmaxFloor ? kAmaxFloor : t;
            if (!(t <= 3.4e38f)) t = __int_as_float(0x7fffffff);
            inv = kQ8Max / t;
            if (threadIdx.x == 0) a.scale[m] = t / kQ8Max;
        }
        if (a.rstd && threadIdx.x == 0) a.rstd[m] = rstd;
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
            const float hv = h(d), yv = y(d);
            if (a.h) static_cast<__nv_bfloat16 *>(a.h)[row + d] = __float2bfloat16(hv);
            if (a.q8)
                static_cast<__nv_fp8_storage_t *>(a.y)[row + d] =
                    __nv_cvt_float_to_fp8(yv * inv, __NV_SATFINITE, __NV_E4M3);
            else
                static_cast<__nv_bfloat16 *>(a.y)[row + d] = __float2bfloat16(yv);
        }
    }
}

__global__ void __launch_bounds__(256) rms_norm_dx_kernel(const NormBwdArgs a)
{
    for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t row = (size_t)m * a.D;
        const float r = a.rstd[m];
        float s = 0.f;
        for (int d = threadIdx.x; d < a.D; d += blockDim.x)
            s += bf(a.dy, row + d) * a.weight[d] * (bf(a.h, row + d) * r);
        s = block_reduce<false>(s) / a.D;
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
            float v = r * (bf(a.dy, row + d) * a.weight[d] - bf(a.h, row + d) * r * s);
            if (a.dh) v += bf(a.dh, row + d);
            static_cast<__nv_bfloat16 *>(a.dx)[row + d] = __float2bfloat16(v);
        }
    }
}

// Partial sums over a block of rows, one thread a column; then their sum.
__global__ void rms_norm_dw_kernel(const NormBwdArgs a, int blocks)
{
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    float s = 0.f;
    for (long long m = blockIdx.y; m < a.M; m += blocks)
        s += bf(a.dy, (size_t)m * a.D + d) * bf(a.h, (size_t)m * a.D + d) * a.rstd[m];
    a.part[(size_t)blockIdx.y * a.D + d] = s;
}

__global__ void sum_parts_kernel(const float *part, float *out, int blocks, int D)
{
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= D) return;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[(size_t)b * D + d];
    out[d] = s;
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs &a, cudaStream_t stream)
{
    rms_norm_kernel<<<a.M < 65536 ? a.M : 65536, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

int norm_bwd_blocks(int M, int) { return M < 128 ? (M > 0 ? M : 1) : 128; }

cudaError_t launch_rms_norm_bwd(const NormBwdArgs &a, cudaStream_t stream)
{
    const int blocks = norm_bwd_blocks(a.M, a.D);
    rms_norm_dw_kernel<<<dim3((a.D + 127) / 128, blocks), 128, 0, stream>>>(a, blocks);
    sum_parts_kernel<<<(a.D + 127) / 128, 128, 0, stream>>>(a.part, a.dweight, blocks, a.D);
    rms_norm_dx_kernel<<<a.M < 65536 ? a.M : 65536, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace attn
