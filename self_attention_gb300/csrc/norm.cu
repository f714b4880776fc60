// Root-mean-square norm with the residual's addition, its 8-bit form and its backward.
//
// All of it is bound by HBM: each row is read once into registers, reduced, and written once.  A row
// is taken by 8 or 16 lanes (up to 64 and 128 columns), a warp (to 2048; no barrier, only shuffles), by
// 256 threads (to 16384) or by 1024 threads (to 32768), each thread holding chunks of 8 neighbouring
// columns (16-byte loads); longer rows are read a second time from L2.  Measured on 128 to 470 MB in calls
// back to back: forward 32768 x 1024 with residual 40.9 us (6.6 TB/s, 0.97 of the measured copy), to 8 bits
// 32768 x 2048 70.0 us (6.7 TB/s); backward 32768 x 1024 47 us (5.7 TB/s), 18432 x 768 23.4 us with the join
// of dweight's partial sums: its rows are taken one after another by the same warps, for those sums.
#include "cluster.cuh"
#include "kernels.h"
#include "sum_rows.cuh"

namespace attn {
namespace {

constexpr float kQ8Max = 448.f;      // largest e4m3
constexpr float kAmaxFloor = 1e-30f;
constexpr int kPlanSms = 152;        // the plan of the backward is a function of the sizes alone

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

// Two bf16 -> a pair of fp32.
__device__ __forceinline__ uint64_t pair(uint32_t w)
{
    return ptx::f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                      ptx::pack_bf16x2(f[6], f[7]));
}

// Two fp32 values -> two e4m3 (round to nearest even, saturating); `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void load8(const float *p, float (&f)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Reduction over the TPR threads that hold a row (a part of a warp, a warp, or the whole block).
template <int TPR, class Op>
__device__ __forceinline__ float row_reduce(float v, Op op)
{
#pragma unroll
    for (int o = TPR < 32 ? TPR / 2 : 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
    if constexpr (TPR > 32) {
        __shared__ float part[TPR / 32];
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = part[0];
#pragma unroll 8
        for (int i = 1; i < TPR / 32; ++i) v = op(v, part[i]);
    }
    return v;
}

// Writes 8 columns of the normalised (or plain) row, in bf16 or in e4m3 times `inv`.
template <bool Q8>
__device__ __forceinline__ void store_y(void *y, size_t at, const float (&f)[8], float inv)
{
    if (Q8)
        static_cast<uint2 *>(y)[at] =
            make_uint2(pack_e4m3x2(f[0] * inv, f[1] * inv) | pack_e4m3x2(f[2] * inv, f[3] * inv) << 16,
                       pack_e4m3x2(f[4] * inv, f[5] * inv) | pack_e4m3x2(f[6] * inv, f[7] * inv) << 16);
    else
        static_cast<uint4 *>(y)[at] = pack8(f);
}

// 448 / max(amax, floor); NaN for a row with an infinity or a NaN.
__device__ __forceinline__ float q8_inverse(float amax, float &scale)
{
    float a = amax < kAmaxFloor ? kAmaxFloor : amax;
    if (!(a <= 3.402823466e38f)) a = __int_as_float(0x7fffffff);
    scale = a / kQ8Max;
    return kQ8Max / a;
}

__host__ __device__ constexpr int holders(int tpr) { return tpr <= 32 ? 128 / tpr : 1; }   // of a block

// Each holder (TPR threads) takes ROWS rows, all of them in flight at once.
template <int TPR, int CH, int ROWS, bool Q8>
__global__ void __launch_bounds__(TPR *holders(TPR)) rms_norm_kernel(const NormArgs a)
{
    const long long m0 = (long long)blockIdx.x * holders(TPR) * ROWS + threadIdx.x / TPR;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (TPR >= 32 && m0 >= a.M) return;   // whole warps (TPR = 32), or never
    const int t = threadIdx.x % TPR, nch = a.D / 8;
    uint4 xv[ROWS][CH], rv[ROWS][CH];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const long long m = m0 + k * holders(TPR);
        const size_t row = (size_t)m * nch;   // in chunks
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = t + c * TPR;
            if (i < nch && m < a.M) {
                xv[k][c] = static_cast<const uint4 *>(a.x)[row + i];
                if (a.residual) rv[k][c] = static_cast<const uint4 *>(a.residual)[row + i];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const long long m = m0 + k * holders(TPR);
        const size_t row = (size_t)m * nch;
        const int n = m < a.M ? nch : 0;   // (every lane takes part in the sums)
        float h[CH][8], s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = t + c * TPR;
            if (i >= n) continue;
            unpack8(xv[k][c], h[c]);
            if (a.residual) {
                float f[8];
                unpack8(rv[k][c], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] += f[e];
                if (a.h) static_cast<uint4 *>(a.h)[row + i] = pack8(h[c]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(h[c][e], h[c][e], s);
        }
        if (a.weight) {
            const float rstd = 1.f / sqrtf(row_reduce<TPR>(s, add) / (float)a.D + a.eps);
            if (a.rstd && t < n && t == 0) a.rstd[m] = rstd;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = t + c * TPR;
                if (i >= n) continue;
                float w[8];
                load8(a.weight + i * 8, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] = h[c][e] * rstd * w[e];
                if (!Q8) store_y<false>(a.y, row + i, h[c], 1.f);
            }
        }
        if (Q8) {
            float amax = 0.f, scale;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (t + c * TPR < n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(h[c][e]));
            const float inv = q8_inverse(row_reduce<TPR>(amax, max_nan), scale);
            if (t < n && t == 0) a.scale[m] = scale;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (t + c * TPR < n) store_y<true>(a.y, row + t + c * TPR, h[c], inv);
        }
    }
}

// Rows of more than 32768 columns: the row is read again for each pass over it.  h may be one of the
// inputs, so it is written in the last pass, by the thread that reads those elements.
template <bool Q8>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const NormArgs a)
{
    const size_t row = (size_t)blockIdx.x * (a.D / 8);
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    auto load_h = [&](int i, float (&h)[8]) {
        unpack8(static_cast<const uint4 *>(a.x)[row + i], h);
        if (a.residual) {
            float f[8];
            unpack8(static_cast<const uint4 *>(a.residual)[row + i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] += f[e];
        }
    };
    float s = 0.f, rstd = 1.f, amax = 0.f, inv = 1.f;
    float h[8], w[8];
    if (a.weight) {
        for (int i = threadIdx.x; i < a.D / 8; i += 1024) {
            load_h(i, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(h[e], h[e], s);
        }
        rstd = 1.f / sqrtf(row_reduce<1024>(s, add) / (float)a.D + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
    }
    auto load_y = [&](int i, float (&y)[8]) {
        if (!a.weight) return;
        load8(a.weight + i * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * rstd * w[e];
    };
    if (Q8) {
        for (int i = threadIdx.x; i < a.D / 8; i += 1024) {
            load_h(i, h);
            load_y(i, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(h[e]));
        }
        float scale;
        inv = q8_inverse(row_reduce<1024>(amax, max_nan), scale);
        if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
    }
    for (int i = threadIdx.x; i < a.D / 8; i += 1024) {
        load_h(i, h);
        if (a.h) static_cast<uint4 *>(a.h)[row + i] = pack8(h);
        load_y(i, h);
        store_y<Q8>(a.y, row + i, h, inv);
    }
}

// dx and the partial sums of dweight: each row-holder (a warp, or the block) walks its rows, keeping
// the sums of dy n for its columns in registers; the warps of a block then add theirs up in order.
// The rows a block takes, and so the order of the sums, follow from the sizes alone.
// The SM's own work shows beside the memory's (L1's data pipe was 64 % busy, the schedulers 48 %), so the
// weights lie in shared memory in two planes that are read without conflicts, and the arithmetic is on
// pairs: 18432 x 768 25.5 -> 23.5 us, 2048 x 16384 72 -> 63.  Measured and not kept: the next rows on their
// way to shared memory meanwhile (cp.async; 28.5 us, the data passes that pipe twice more), or to registers
// (26.1).  Threads and blocks an SM are the most whose registers hold a row, the sums and four columns of
// operands without spilling.
__host__ __device__ constexpr int bwd_blocks_per_sm(int ch) { return ch <= 1 ? 4 : ch <= 2 ? 3 : ch <= 4 ? 2 : 1; }
__host__ __device__ constexpr int bwd_threads(int tpr, int ch) { return tpr == 32 && ch == 3 ? 320 : 256; }
__host__ __device__ constexpr int bwd_tpr(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 2048 ? 32 : 256; }

template <int TPR, int CH>
__global__ void __launch_bounds__(bwd_threads(TPR, CH), bwd_blocks_per_sm(CH))
    rms_norm_bwd_kernel(const NormBwdArgs a, int blocks)
{
    constexpr int THREADS = bwd_threads(TPR, CH), RPB = THREADS / TPR;   // row-holders a block
    extern __shared__ __align__(16) float weights[];
    const int t = threadIdx.x % TPR, holder = threadIdx.x / TPR, nch = a.D / 8;
    const long long step = (long long)blocks * RPB;
    long long m = (long long)blockIdx.x * RPB + holder;
    uint64_t acc[CH][4] = {};
    uint4 dv[CH], hv[CH], gv[CH];
    float r = 0.f;
    auto load_row = [&] {   // everything the row needs is asked for at once
        if (m >= a.M) {   // (only beside another row of the warp)
            if (TPR < 32) {
                r = 0.f;
                dv[0] = hv[0] = gv[0] = make_uint4(0, 0, 0, 0);
            }
            return;
        }
        const size_t row = (size_t)m * nch;
        const uint4 *dy = static_cast<const uint4 *>(a.dy) + row, *h = static_cast<const uint4 *>(a.h) + row,
                    *dh = static_cast<const uint4 *>(a.dh) + row;
        r = a.rstd[m];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = t + c * TPR;
            if (i < nch) {
                dv[c] = dy[i];
                hv[c] = h[i];
                if (a.dh) gv[c] = dh[i];
            }
        }
    };
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    load_row();
    // a chunk's 8 weights as two planes of 16 bytes a thread: read side by side, without conflicts
    for (int i = threadIdx.x; i < a.D / 4; i += THREADS) {
        const int chunk = i >> 1;
        reinterpret_cast<float4 *>(weights)[(chunk / TPR * 2 + (i & 1)) * TPR + chunk % TPR] =
            *(reinterpret_cast<const float4 *>(a.weight) + i);
    }
    __syncthreads();
    const uint32_t wt = ptx::smem_u32(weights) + t * 16;
    const int in_warp = TPR < 32 ? holder % (32 / TPR) : 0;   // a warp's rows are neighbours, and end together
    for (; m - in_warp < a.M; m += step, load_row()) {
        uint64_t sum = 0;
        const uint64_t rr = ptx::f2_pack(r, r);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (t + c * TPR >= nch) continue;
            const uint32_t dw[4] = {dv[c].x, dv[c].y, dv[c].z, dv[c].w}, hw[4] = {hv[c].x, hv[c].y, hv[c].z, hv[c].w};
#pragma unroll
            for (int q = 0; q < 2; ++q) {   // four columns
                const ulonglong2 w4 = lds_f32x4(wt + (2 * c + q) * TPR * 16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint64_t p = ptx::mul_f32x2(pair(dw[2 * q + e]), ptx::mul_f32x2(pair(hw[2 * q + e]), rr));
                    acc[c][2 * q + e] = ptx::add_f32x2(acc[c][2 * q + e], p);
                    sum = ptx::fma_f32x2(p, e ? w4.y : w4.x, sum);
                }
            }
        }
        float lo, hi;
        ptx::f2_unpack(sum, lo, hi);
        const float s = -row_reduce<TPR>(lo + hi, add) / (float)a.D;
        const uint64_t ss = ptx::f2_pack(s, s);
        uint4 *dx = static_cast<uint4 *>(a.dx) + (size_t)m * nch;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (t + c * TPR >= nch) continue;
            const uint32_t dw[4] = {dv[c].x, dv[c].y, dv[c].z, dv[c].w}, hw[4] = {hv[c].x, hv[c].y, hv[c].z, hv[c].w},
                           gw[4] = {gv[c].x, gv[c].y, gv[c].z, gv[c].w};
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const ulonglong2 w4 = lds_f32x4(wt + (2 * c + q) * TPR * 16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 2 * q + e;
                    const uint64_t v = ptx::fma_f32x2(pair(dw[k]), e ? w4.y : w4.x,
                                                      ptx::mul_f32x2(ptx::mul_f32x2(pair(hw[k]), rr), ss));
                    ptx::f2_unpack(a.dh ? ptx::fma_f32x2(v, rr, pair(gw[k])) : ptx::mul_f32x2(v, rr), lo, hi);
                    o[k] = ptx::pack_bf16x2(lo, hi);
                }
            }
            if (TPR >= 32 || m < a.M) dx[t + c * TPR] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    float *part = a.part + (size_t)blockIdx.x * a.D;
    if constexpr (TPR > 32) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = t + c * TPR;
            if (i >= nch) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<uint64_t *>(part)[i * 4 + e] = acc[c][e];
        }
    } else {
        constexpr int COLS = 8 * TPR;   // at a time
        __shared__ __align__(16) float sums[RPB][COLS];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<uint64_t *>(sums[holder])[t * 4 + e] = acc[c][e];
            __syncthreads();
            const int col = c * COLS + threadIdx.x;
            if (threadIdx.x < COLS && col < a.D) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < RPB; ++w) v += sums[w][threadIdx.x];
                part[col] = v;
            }
        }
    }
}

// The same for rows of more than 16384 columns: two passes over each row, the sums of dy n in a
// block's own row of the workspace.
__global__ void __launch_bounds__(1024) rms_norm_bwd_long_kernel(const NormBwdArgs a, int blocks)
{
    float *part = a.part + (size_t)blockIdx.x * a.D;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    for (long long m = blockIdx.x; m < a.M; m += blocks) {
        const size_t row = (size_t)m * (a.D / 8);
        const float r = a.rstd[m];
        float d[8], n[8], w[8], s = 0.f;
        for (int i = threadIdx.x; i < a.D / 8; i += 1024) {
            unpack8(static_cast<const uint4 *>(a.dy)[row + i], d);
            unpack8(static_cast<const uint4 *>(a.h)[row + i], n);
            load8(a.weight + i * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = d[e] * (n[e] * r);
                part[i * 8 + e] = (m == blockIdx.x ? 0.f : part[i * 8 + e]) + p;
                s = fmaf(p, w[e], s);
            }
        }
        s = row_reduce<1024>(s, add) / (float)a.D;
        for (int i = threadIdx.x; i < a.D / 8; i += 1024) {
            unpack8(static_cast<const uint4 *>(a.dy)[row + i], d);
            unpack8(static_cast<const uint4 *>(a.h)[row + i], n);
            load8(a.weight + i * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = r * fmaf(d[e], w[e], -(n[e] * r) * s);
            if (a.dh) {
                unpack8(static_cast<const uint4 *>(a.dh)[row + i], n);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += n[e];
            }
            static_cast<uint4 *>(a.dx)[row + i] = pack8(d);
        }
    }
}

// The join of dweight's (and dbias's) partial sums.  Blocks this small find room beside the kernel before, and
// wait there for its end.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float *part, float *out, int rows, int cols)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    sum_columns(part, out, rows, cols, blockIdx.x * kSumCols);
}

template <int TPR, int CH, int ROWS = 1>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    constexpr int R = holders(TPR) * ROWS;
    const unsigned grid = (unsigned)(((long long)a.M + R - 1) / R);
    return a.q8 ? launch_overlapped(rms_norm_kernel<TPR, CH, ROWS, true>, grid, TPR * holders(TPR), 0, 1, stream, a)
                : launch_overlapped(rms_norm_kernel<TPR, CH, ROWS, false>, grid, TPR * holders(TPR), 0, 1, stream, a);
}

template <int TPR, int CH>
cudaError_t launch_norm_bwd(const NormBwdArgs &a, int blocks, cudaStream_t stream)
{
    constexpr int weights = CH * TPR * 32;
    if (weights > 32768) {
        static std::atomic<bool> set[64];
        const cudaError_t e = raise_smem((const void *)rms_norm_bwd_kernel<TPR, CH>, weights, set);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(rms_norm_bwd_kernel<TPR, CH>, blocks, bwd_threads(TPR, CH), weights, 1, stream, a, blocks);
}

}  // namespace

cudaError_t launch_sum_rows(const float *part, float *out, int rows, int cols, cudaStream_t stream)
{
    return launch_overlapped(sum_rows_kernel, cols / kSumCols, 256, 0, 1, stream, part, out, rows, cols);   // cols % 8 == 0
}

cudaError_t launch_rms_norm(const NormArgs &a, cudaStream_t stream)
{
    const int D = a.D;
    // a few rows (no more than two blocks an SM): 256 threads each hold one chunk of a row, which is read
    // and reduced sooner than by a warp (7 x 2048 to 8 bits: 4.8 against 6.1 us a call)
    if (D > 256 && D <= 2048 && a.M <= 2 * kPlanSms) return launch_norm<256, 1>(a, stream);
    // Short rows: as many threads a row as it has chunks, and of many rows (eight blocks an SM) four a holder,
    // since blocks of 2 KB start no faster than one a nanosecond (524288 x 64 with residual: 43 us, by whole
    // warps and one row 134; 131072 x 256 26 and 36, but with residual, twice the bytes a row, 42.5 and 41.4).
    const bool many = (long long)a.M * D >= 8LL * kPlanSms * 4096;
    if (D <= 64) return many ? launch_norm<8, 1, 4>(a, stream) : launch_norm<8, 1>(a, stream);
    if (D <= 128) return many ? launch_norm<16, 1, 4>(a, stream) : launch_norm<16, 1>(a, stream);
    if (D <= 256) return many && !a.residual ? launch_norm<32, 1, 4>(a, stream) : launch_norm<32, 1>(a, stream);
    if (D <= 512) return launch_norm<32, 2>(a, stream);
    if (D <= 1024) return launch_norm<32, 4>(a, stream);
    if (D <= 2048) return launch_norm<32, 8>(a, stream);
    if (D <= 4096) return launch_norm<256, 2>(a, stream);
    if (D <= 8192) return launch_norm<256, 4>(a, stream);
    if (D <= 16384) return launch_norm<256, 8>(a, stream);
    if (D <= 32768) return launch_norm<1024, 4>(a, stream);
    return launch_overlapped(a.q8 ? rms_norm_long_kernel<true> : rms_norm_long_kernel<false>, a.M, 1024, 0, 1, stream, a);
}

// As many blocks as fit the SMs at once (see bwd_blocks_per_sm); no more than there are rows for, and one
// for up to two rows a holder: its sums are dweight itself, which saves the join.
int norm_bwd_blocks(int M, int D)
{
    const int tpr = bwd_tpr(D), ch = D <= 16384 ? (D + 8 * tpr - 1) / (8 * tpr) : 8;
    const int rpb = bwd_threads(tpr, ch) / tpr, want = bwd_blocks_per_sm(ch) * kPlanSms;
    const int most = (int)(((long long)M + rpb - 1) / rpb);
    const int b = want < most ? want : most;
    return b > 2 ? b : 1;
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs &args, cudaStream_t stream)
{
    NormBwdArgs a = args;
    const int blocks = norm_bwd_blocks(a.M, a.D), D = a.D;
    if (blocks == 1) a.part = a.dweight;
    const cudaError_t e = D <= 64      ? launch_norm_bwd<8, 1>(a, blocks, stream)
                          : D <= 128   ? launch_norm_bwd<16, 1>(a, blocks, stream)
                          : D <= 256   ? launch_norm_bwd<32, 1>(a, blocks, stream)
                          : D <= 512   ? launch_norm_bwd<32, 2>(a, blocks, stream)
                          : D <= 768   ? launch_norm_bwd<32, 3>(a, blocks, stream)
                          : D <= 1024  ? launch_norm_bwd<32, 4>(a, blocks, stream)
                          : D <= 2048  ? launch_norm_bwd<32, 8>(a, blocks, stream)
                          : D <= 4096  ? launch_norm_bwd<256, 2>(a, blocks, stream)
                          : D <= 8192  ? launch_norm_bwd<256, 4>(a, blocks, stream)
                          : D <= 16384 ? launch_norm_bwd<256, 8>(a, blocks, stream)
                                       : launch_overlapped(rms_norm_bwd_long_kernel, blocks, 1024, 0, 1, stream, a, blocks);
    return e == cudaSuccess && blocks > 1 ? launch_sum_rows(a.part, a.dweight, blocks, D, stream) : e;
}

}  // namespace attn
