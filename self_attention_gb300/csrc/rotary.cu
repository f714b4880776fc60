// Rotary positions, and the append that brings new tokens into a cache.
//
// A pair of columns (a, b) at position p becomes a (cos t, sin t) + b (-sin t, cos t), t = p f, times an
// amplitude; the gradient is the same with -t.  The frequency f comes as whole turns a position in units of
// 2^-64, so that p f mod 1 is one 64-bit product whose overflow is the reduction: exact for any position,
// where an fp32 angle is off by a whole 2^-24 p f.  Its upper 32 bits, as a fraction of half a turn, go to
// sincospif(), the last of them set where a lower one is, so that the rounding to fp32 is that of all 64: the angle is
// off by at most 2^-25 of half a turn from the p-fold of f as it was given (cutting first would add 2^-31).
//
// Bound by HBM.  A thread takes eight pairs of one token (16 columns: two 16-byte chunks), computes their
// eight sines and cosines once and walks over heads with them, as many as still leave the GPU full of threads;
// four heads' loads are in flight at once.  Columns that are not turned, and values on their way into the
// cache, are copied by the same threads.
#include "cluster.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kThreads = 128;

struct Turn {
    float c[8], s[8];
};

// Sines and cosines of pairs 8 i ... 8 i + 7 at position p.
__device__ __forceinline__ void turn_of(Turn &t, const uint64_t *turns, int i, int p, float amplitude, float sign)
{
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(turns + 8 * i + e);
        const uint64_t a[2] = {f.x * (uint64_t)(int64_t)p, f.y * (uint64_t)(int64_t)p};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float s, c;
            const int32_t u = (int32_t)(a[k] >> 32) | ((uint32_t)a[k] != 0);
            sincospif((float)u * 0x1p-31f, &s, &c);
            t.c[e + k] = c * amplitude;
            t.s[e + k] = s * (amplitude * sign);
        }
    }
}

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The two chunks of one thread: columns j ... j + 7 and j + r / 2 ... (pairs across them), or 16 neighbours
// (pairs inside them).
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(uint4 &x, uint4 &y, const Turn &t)
{
    uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (INTERLEAVED) {
            const float a0 = lo(a[e]), a1 = hi(a[e]), b0 = lo(b[e]), b1 = hi(b[e]);
            a[e] = ptx::pack_bf16x2(a0 * t.c[e] - a1 * t.s[e], a0 * t.s[e] + a1 * t.c[e]);
            b[e] = ptx::pack_bf16x2(b0 * t.c[4 + e] - b1 * t.s[4 + e], b0 * t.s[4 + e] + b1 * t.c[4 + e]);
        } else {
            const float a0 = lo(a[e]), a1 = hi(a[e]), b0 = lo(b[e]), b1 = hi(b[e]);
            const float c0 = t.c[2 * e], s0 = t.s[2 * e], c1 = t.c[2 * e + 1], s1 = t.s[2 * e + 1];
            a[e] = ptx::pack_bf16x2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
            b[e] = ptx::pack_bf16x2(a0 * s0 + b0 * c0, a1 * s1 + b1 * c1);
        }
    }
    x = make_uint4(a[0], a[1], a[2], a[3]);
    y = make_uint4(b[0], b[1], b[2], b[3]);
}

// First columns of item i's two chunks (r columns are turned; items from r / 16 on are copied).
template <bool INTERLEAVED>
__device__ __forceinline__ void chunks(int i, int r, int &c0, int &c1)
{
    const bool across = !INTERLEAVED && i < r / 16;
    c0 = across ? 8 * i : 16 * i;
    c1 = across ? 8 * i + r / 2 : 16 * i + 8;
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void store16(__nv_bfloat16 *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a, int heads, float sign)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int items = a.d / 16;
    const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (at >= (long long)a.B * a.N * items) return;
    const int i = (int)(at % items);
    const long long bn = at / items;
    const int n = (int)(bn % a.N), b = (int)(bn / a.N);
    const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, a.H);
    int c0, c1;
    chunks<INTERLEAVED>(i, a.rotated, c0, c1);
    const bool turned = i < a.rotated / 16;
    const int p = a.positions ? a.positions[b * a.pos_stride + n] : n;
    const long long step = (long long)a.N * a.d;
    const long long base = ((long long)b * a.H + h0) * step + (long long)n * a.d;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + base;
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + base;
    Turn t;
    if (turned) turn_of(t, a.turns, i, p, a.amplitude, sign);
    for (int h = h0; h < h1; h += 4, x += 4 * step, y += 4 * step) {
        uint4 u[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (h + e < h1) {
                u[e] = load16(x + e * step + c0);
                v[e] = load16(x + e * step + c1);
            }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (h + e < h1) {
                if (turned) turn<INTERLEAVED>(u[e], v[e], t);
                store16(y + e * step + c0, u[e]);
                store16(y + e * step + c1, v[e]);
            }
    }
}

// Heads 0 ... H - 1 are the keys, H ... 2 H - 1 the values, the rest the queries, which stay where they are.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, int heads)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int items = a.d / 16;
    const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (at >= (long long)a.B * a.n * items) return;
    const int i = (int)(at % items);
    const long long bn = at / items;
    const int n = (int)(bn % a.n), b = (int)(bn / a.n);
    const int from = a.rows ? a.rows[bn] : n;
    const int length = max(a.lengths[b], 0);
    const bool fits = n < a.C - length;
    if (from < 0 || from >= a.T) return;
    const int slot = (int)((unsigned)length + (unsigned)n);
    const int p = a.positions ? a.positions[(long long)b * a.T + from] : slot;
    const bool turned = a.turns && i < a.rotated / 16;
    int c0, c1;
    chunks<INTERLEAVED>(i, a.turns ? a.rotated : 0, c0, c1);
    Turn t;
    if (turned) turn_of(t, a.turns, i, p, a.amplitude, 1.f);
    const int h0 = blockIdx.y * heads, all = 2 * a.H + (a.q ? a.Hq : 0), h1 = min(h0 + heads, all);
    for (int h = h0; h < h1; h += 4) {
        uint4 u[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int hh = h + e;
            if (hh >= h1) continue;
            const __nv_bfloat16 *x =
                hh < 2 * a.H ? static_cast<const __nv_bfloat16 *>(hh < a.H ? a.k : a.v) +
                                   (((long long)b * a.H + (hh < a.H ? hh : hh - a.H)) * a.T + from) * a.d
                             : static_cast<const __nv_bfloat16 *>(a.q) +
                                   (((long long)b * a.Hq + hh - 2 * a.H) * a.T + from) * a.d;
            u[e] = load16(x + c0);
            v[e] = load16(x + c1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int hh = h + e;
            if (hh >= h1) continue;
            if (turned && (hh < a.H || hh >= 2 * a.H)) turn<INTERLEAVED>(u[e], v[e], t);
            __nv_bfloat16 *y;
            if (hh < 2 * a.H) {
                if (!fits) continue;
                const long long row = ((long long)b * a.H + (hh < a.H ? hh : hh - a.H)) * a.C + slot;
                y = static_cast<__nv_bfloat16 *>(hh < a.H ? a.cache_k : a.cache_v) + row * a.d;
                if (i == 0 && hh < a.H) {
                    if (a.weights) a.weights[row] = 0.f;
                    if (a.slot_positions) a.slot_positions[row] = p;
                }
            } else {
                y = static_cast<__nv_bfloat16 *>(a.q_out) + (((long long)b * a.Hq + hh - 2 * a.H) * a.T + from) * a.d;
            }
            store16(y + c0, u[e]);
            store16(y + c1, v[e]);
        }
    }
}

// Heads a thread walks over: as many as leave 2048 threads an SM, in even shares.  (Measured with 1024, 2048 and 4096:
// 8 x 16 x 4096 x 64 22.1, 21.1 and 24.2 us, the gradient of 2 x 16 x 16384 x 128 45.7, 41.8 and 41.4, blocks of 256
// threads 1 us more; floors 19.8 and 39.6.)
int heads_a_thread(long long threads, int heads)
{
    const long long full = (long long)device_sm_count() * 2048, groups = (full + threads - 1) / threads;
    return groups >= heads ? 1 : (int)((heads + groups - 1) / groups);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, bool interleaved, bool backward, cudaStream_t stream)
{
    const long long threads = (long long)a.B * a.N * (a.d / 16);
    const int heads = heads_a_thread(threads, a.H);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)((a.H + heads - 1) / heads));
    const float sign = backward ? -1.f : 1.f;
    return interleaved ? launch_overlapped(rotary_kernel<true>, grid, dim3(kThreads), 0, 1, stream, a, heads, sign)
                       : launch_overlapped(rotary_kernel<false>, grid, dim3(kThreads), 0, 1, stream, a, heads, sign);
}

cudaError_t launch_append(const AppendArgs &a, bool interleaved, cudaStream_t stream)
{
    const long long threads = (long long)a.B * a.n * (a.d / 16);
    const int all = 2 * a.H + (a.q ? a.Hq : 0), heads = heads_a_thread(threads, all);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)((all + heads - 1) / heads));
    return interleaved ? launch_overlapped(append_kernel<true>, grid, dim3(kThreads), 0, 1, stream, a, heads)
                       : launch_overlapped(append_kernel<false>, grid, dim3(kThreads), 0, 1, stream, a, heads);
}

}  // namespace attn
