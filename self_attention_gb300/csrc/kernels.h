// Host-side launchers of the attention kernels (internal to the library; the public C ABI
// in include/attn.h validates arguments and calls these).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>

namespace attn {

struct FwdArgs {
    CUtensorMap tm_q, tm_k, tm_v;   // 3-D maps over [BH, N, d] bf16, 64 x rows boxes, 128-byte swizzle
    CUtensorMap tm_o;               // the same over O (128-row boxes), for tile stores
    void *o;                        // [BH, N, d] bf16
    float *lse;                     // [BH, N] fp32
    int bh, n, d;
    float scale;
    int v_f16;                      // 1: tm_v maps an fp16 copy of V (no rewrite in shared memory)
    float *o32;                     // null, or [BH, N, d] fp32: O before its bf16 rounding (diagnostic)
    int *status;                    // device status word
};

struct BwdArgs {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    CUtensorMap tm_dk, tm_dv;       // dK and dV with 128-row boxes (tile stores, d = 64)
    const void *o, *dout;           // [BH, N, d] bf16
    const float *lse;               // [BH, N]
    void *dq, *dk, *dv;             // [BH, N, d] bf16
    // [BH, n_pad / 2] x 4 fp32 workspace, per pair of rows (2k, 2k + 1):
    // {-lse log2 e of both rows, -rowsum(dO o O) of both rows}; -inf and 0 past N.
    float *stats;
    float *dq_acc;                  // [BH, N, d]  workspace: fp32 dQ accumulator
    int bh, n, n_pad, d;
    float scale;
    int *status;
};

// Streaming multiprocessors of the current device (cached per device, safe to call from several
// host threads).
int device_sm_count();

cudaError_t launch_fwd(const FwdArgs &a, cudaStream_t stream);
// v16[i] = v[i] rounded from bf16 to fp16, elems a multiple of 8, both 16-byte aligned.
cudaError_t launch_v_to_f16(const void *v, void *v16, long long elems, cudaStream_t stream);
// The three stream-ordered phases of the backward pass.
cudaError_t launch_bwd_preprocess(const BwdArgs &a, cudaStream_t stream);
cudaError_t launch_bwd_main(const BwdArgs &a, cudaStream_t stream);
cudaError_t launch_bwd_convert(const BwdArgs &a, cudaStream_t stream);
// Short sequences at d = 64 (N <= 256): the whole backward (statistics, dQ, dK, dV) in one
// kernel, one CTA per head, dQ accumulated on chip; used by attn_bwd and
// attn_bwd_deterministic where bwd_whole_heads(n, d, B*H) holds.
bool bwd_whole_heads(int n, int d, long long bh);
cudaError_t launch_bwd_heads(const BwdArgs &a, cudaStream_t stream);
// The deterministic backward: preprocess (no accumulator), the main kernel without its dQ part,
// then a query-stationary pass that computes dQ without atomics.
cudaError_t launch_bwd_deterministic(const BwdArgs &a, cudaStream_t stream);
// QKV projection (see proj.cu): tensor maps of the two operands (up to three each) and sizes.
struct ProjMaps {
    CUtensorMap a[3], b[3];
};
struct ProjArgs {
    int B, N, D, H, dk;
    __nv_bfloat16 *qkv[3];   // forward outputs Q, K, V [B,H,N,dk]
    __nv_bfloat16 *dx;       // [B,N,D]
    float *dw[3];            // [D,D] each
    int *status;
};
cudaError_t launch_proj_fwd(const ProjMaps &m, const ProjArgs &a, cudaStream_t stream);
cudaError_t launch_proj_dx(const ProjMaps &m, const ProjArgs &a, cudaStream_t stream);
cudaError_t launch_proj_dw(const ProjMaps &m, const ProjArgs &a, cudaStream_t stream);

// Standard attention (S and P through HBM; see unfused.cu): returns nullptr on success, else what
// failed (with *err set where a CUDA call failed).  s: [BH][N][N] fp32, p: [BH][N][N] bf16.
const char *launch_fwd_unfused(const FwdArgs &a, const void *q, const void *k, const void *v, float *s,
                               void *p, cudaStream_t stream, cudaError_t *err);

// Launches a kernel that may start while the one before it on the stream ends (it calls
// ptx::grid_dep_wait() before it touches global memory), in clusters of `cluster` blocks.
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, unsigned cluster,
                              cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raises the kernel's shared-memory limit, once per device.
inline cudaError_t raise_smem(const void *kernel, int bytes, std::atomic<bool> (&set)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) == cudaSuccess)
        set[dev].store(true, std::memory_order_relaxed);
    return e;
}

// 3-D tensor map (innermost first: d0, d1, d2 elements, dense) with boxes of box0 x box1 x 1 whose
// rows, 64 or 128 bytes, are swizzled over their length; elements outside read as zeros and are not
// written.
CUresult make_map_3d(CUtensorMap *m, const void *base, CUtensorMapDataType type, int elem_bytes, long long d0,
                     long long d1, long long d2, int box0, int box1);

// Linear layers (see linear.cu).  The x side is seen as [G, H, T, dk]: row m = g T + i, column
// c = h dk + e; a plain [M, K] matrix is G = H = 1, T = M, dk = K.
struct LinArgs {
    const void *x, *w;               // bf16 [G,H,T,dk], [K,N]; q8: e4m3 [M,K], [N,K]
    const float *x_scale, *w_scale;  // q8: [M], [N]
    const float *bias;               // null, or [N]
    const void *residual;            // null, or [M,N] bf16
    void *y, *z;                     // [M,N] bf16; z may be null
    int G, T, H, dk;
    int M, K, N;
    int act, q8;
    int *status;
};
// Whether the rows of G groups of T can be counted: padded to whole blocks and tiles they fit an int.
bool lin_rows_fit(int G, int T);
// The plans that launch_linear() and launch_linear_bwd() (asked for everything) follow, as attn_debug_linear_plan()
// gives them.
void lin_plan(int G, int T, int K, int N, int q8, int plan[5]);
void lin_bwd_plan(int G, int T, int K, int N, int has_act, int plan[5]);
cudaError_t launch_linear(const LinArgs &a, cudaStream_t stream);

struct LinBwdArgs {
    const void *x, *w, *dy, *z;      // z null: dz is dy
    void *dx, *dw;                   // bf16, each may be null
    float *dbias;                    // null, or [N]
    void *dz;                        // workspace: [M,N] bf16 (z given)
    float *col_part;                 // workspace: partial column sums, lin_bwd_col_rows() x [N]
    float *dw_part;                  // workspace: lin_dw_splits() x [K,N] where that is > 1
    int G, T, H, dk;
    int M, K, N;
    int act;
    int *status;
};
// The plan of the backward, a function of the sizes alone: how many partial column sums there are at
// most, and how many ways the rows of dw = x^T dz are split.
int lin_bwd_col_rows(int M, int N);
int lin_dw_splits(int G, int T, int K, int N);
cudaError_t launch_linear_bwd(const LinBwdArgs &a, cudaStream_t stream);

// Root-mean-square norm (see norm.cu).
struct NormArgs {
    const void *x, *residual;   // bf16 [M,D]
    const float *weight;        // [D]; null: no norm, the rows themselves are quantised (q8)
    void *y;                    // bf16 or e4m3
    float *scale;               // q8: [M]
    void *h;                    // null, or bf16 [M,D]
    float *rstd;                // null, or [M]
    int M, D, q8;
    float eps;
};
cudaError_t launch_rms_norm(const NormArgs &a, cudaStream_t stream);
struct NormBwdArgs {
    const void *dy, *h, *dh;
    const float *weight, *rstd;
    void *dx;
    float *dweight;
    float *part;                // workspace: norm_bwd_blocks() x [D]
    int M, D;
};
// out[c] = sum over rows of part[row][c], in a fixed order.
cudaError_t launch_sum_rows(const float *part, float *out, int rows, int cols, cudaStream_t stream);
int norm_bwd_blocks(int M, int D);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs &a, cudaStream_t stream);

cudaError_t launch_vector_add(const float *a, const float *b, float *c, long long n,
                              cudaStream_t stream);
cudaError_t launch_wait_selftest(int *status, uint64_t limit_ns, cudaStream_t stream);

}  // namespace attn
