// Linear layers on tcgen05 tensor cores: y = act(x w + b) + r forward, dx = dz w^T and dw = x^T dz
// backward, and the forward in e4m3.  One persistent GEMM skeleton over pairs of CTAs,
// C[256 x BN] = sum over K steps of A B, with operand policies:
//   Fwd   : A = x (K-major), B = w [K, N] (MN-major).
//   FwdQ8 : A = xq, B = wq [N, K], both K-major, e4m3.
//   Dx    : A = dz (K-major), B = w (K-major: the rows of w are the columns of dx).
//   Dw    : A = x^T, B = dz, both MN-major; the K steps are 64 rows each.
// x (and dx) may be split by heads, [G, H, T, dk] with row m = g T + i and column c = h dk + e: a
// 64-column box lies in one head, so only the coordinates of the copies differ.  Row tiles (and, for
// dw, steps) lie in one group g; the copies' zero fill and clipping end a tile at the group's last row.
//
// A cluster of two CTAs computes a 256 x BN tile together (tcgen05 cta_group::2): each loads 128 rows
// of A and BN / 2 columns of B a step, 32 KB for 2 x 128 x 256 x 64 multiply-adds where a single CTA
// with the same tile of its own would load 48 KB, which is what bounds the K loop (L2 bandwidth and
// the reads of shared memory).  Each CTA: warp 0 TMA producer, warp 1 tcgen05 issuer (even CTA),
// warps 4-11 epilogue; the accumulator is double-buffered in TMEM, so a tile's epilogue overlaps the
// products of the next.
//
// Epilogue: a warp owns 32 rows x 64 columns at a time (thread = row): TMEM -> registers, scales,
// bias, activation, residual in fp32, one rounding to bf16, a swizzled 4 KB buffer in shared memory,
// one TMA store.  The residual comes the same way round, by a TMA load into that buffer before the
// accumulator is ready.
#include "act.cuh"
#include "common.cuh"
#include "kernels.h"

#include <atomic>

namespace attn {
namespace {

constexpr int BM = 256;            // rows of a tile (both CTAs)
constexpr int kGroupM = 8;         // row tiles walked side by side, for reuse of B in L2

struct GemmMaps {
    CUtensorMap a, b, y, z, r;
};

struct GemmParams {
    int T, mblocks;                // rows of one group, its row tiles
    int n_mtiles, n_ntiles, N;     // row tiles of all groups, column tiles, columns
    int dk, H;                     // the head split of the side that has one (A; Dx: y)
    int ksteps, steps_per_split, tblocks;   // K steps in all and per item; Dw: steps of one group
    int n_items;
    const float *bias, *x_scale, *w_scale;
    int has_z, has_r, act;
    float *part;                   // Dw split over K: [splits][rows][N] fp32 partial sums
    int *status;
};

enum Policy { Fwd, FwdQ8, Dx, Dw };

template <Policy P, int BN>
struct Cfg {
    static constexpr bool FP8 = P == FwdQ8;
    static constexpr bool A_MN = P == Dw, B_MN = P == Fwd || P == Dw;
    static constexpr int KE = FP8 ? 128 : 64;              // elements of K a step: 128 bytes
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int EPI = 8 * 2 * 4096;               // two buffers for each epilogue warp
    static constexpr int SMEM = STAGES * STAGE + EPI + 1024;
    static constexpr uint32_t TM_COLS = 2 * BN;
};

// K-major rows of 128 bytes: the k-th 32-byte slice starts 32 bytes in.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) { return ptx::sdesc_sw128(base + kk * 32, 16, 1024); }
// MN-major: 64-column blocks of 64 K rows (8 KB each); a slice is 16 K rows.
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk)
{
    return ptx::sdesc_sw128(base + kk * 2048, 8192, 1024);
}

template <Policy P, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    gemm_pair_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p)
{
    using C = Cfg<P, BN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    __shared__ uint64_t bar_full[STAGES], bar_empty[STAGES], bar_acc_full[2], bar_acc_empty[2], bar_res[16];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    const int tiles = p.n_mtiles * p.n_ntiles;
    // item -> K range, row tile, column tile: kGroupM row tiles side by side, column by column
    auto decode = [&](int item, int &ks, int &mt, int &nt, int &k_begin, int &nk) {
        ks = item / tiles;
        const int t = item - ks * tiles, per = kGroupM * p.n_ntiles, first = t / per * kGroupM, q = t % per;
        const int rows = min(kGroupM, p.n_mtiles - first);
        mt = first + q % rows;
        nt = q / rows;
        k_begin = ks * p.steps_per_split;
        nk = min(p.steps_per_split, p.ksteps - k_begin);
    };
    const Guard g{&abort_sh, p.status, kWaitLimitNs};

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&bar_full[s], 1);
            ptx::mbar_init(&bar_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&bar_acc_full[b], 1);
            ptx::mbar_init(&bar_acc_empty[b], 16);   // the epilogue warps of both CTAs
        }
        for (int b = 0; b < 16; ++b) ptx::mbar_init(&bar_res[b], 1);
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&tmem_sh, C::TM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // both CTAs' barriers exist before either signals the other
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh;

    if (warp == 0) {
        if (ptx::elect_one()) {
            int j = 0;   // position in the stage ring, across items
            for (int item = cluster; item < p.n_items; item += n_clusters) {
                int ks, mt, nt, k_begin, nk;
                decode(item, ks, mt, nt, k_begin, nk);
                const int grp = mt / p.mblocks, i0 = (mt % p.mblocks) * BM + (int)rank * 128;
                const int n0 = nt * BN + (int)rank * (BN / 2);
                for (int q = 0; q < nk; ++q, ++j) {
                    const int s = j % STAGES, step = k_begin + q;
                    wait_bounded(&bar_empty[s], ((j / STAGES) & 1) ^ 1, g);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&bar_full[s], 2 * C::STAGE);
                    const uint32_t bar = ptx::cluster_addr(ptx::smem_u32(&bar_full[s]), 0);
                    uint8_t *sa = smem + s * C::STAGE, *sb = sa + C::A_BYTES;
                    if (P == Dw) {
                        const int gk = step / p.tblocks, t0 = (step % p.tblocks) * 64;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = i0 + 64 * h;
                            ptx::tma_load_3d_pair(sa + h * 8192, &maps.a, bar, c % p.dk, t0, gk * p.H + c / p.dk);
                        }
#pragma unroll
                        for (int h = 0; h < BN / 128; ++h)
                            ptx::tma_load_3d_pair(sb + h * 8192, &maps.b, bar, n0 + 64 * h, t0, gk);
                    } else {
                        const int c = step * C::KE;
                        if (P == Dx)
                            ptx::tma_load_3d_pair(sa, &maps.a, bar, c, i0, grp);
                        else
                            ptx::tma_load_3d_pair(sa, &maps.a, bar, c % p.dk, i0, grp * p.H + c / p.dk);
                        if (P == Fwd) {
#pragma unroll
                            for (int h = 0; h < BN / 128; ++h)
                                ptx::tma_load_3d_pair(sb + h * 8192, &maps.b, bar, n0 + 64 * h, c, 0);
                        } else {
                            ptx::tma_load_3d_pair(sb, &maps.b, bar, c, n0, 0);
                        }
                    }
                }
            }
            if (rank == 0)   // both CTAs' copies have landed before either leaves
                for (int q = (j > STAGES ? j - STAGES : 0); q < j; ++q)
                    wait_bounded(&bar_full[q % STAGES], (q / STAGES) & 1, g);
        }
    } else if (warp == 1 && rank == 0) {
        if (ptx::elect_one()) {
            const uint32_t idesc = C::FP8 ? ptx::idesc_f16_f32(BM, BN, false, false)   // format 0: e4m3
                                          : ptx::idesc_bf16_f32(BM, BN, C::A_MN, C::B_MN);
            const uint32_t base = ptx::smem_u32(smem);
            int j = 0, li = 0;
            for (int item = cluster; item < p.n_items; item += n_clusters, ++li) {
                int ks, mt, nt, k_begin, nk;
                decode(item, ks, mt, nt, k_begin, nk);
                const int ab = li & 1;
                wait_bounded<true>(&bar_acc_empty[ab], ((li >> 1) & 1) ^ 1, g);   // epilogues of item li-2 done
                ptx::tc_fence_after();
                for (int q = 0; q < nk; ++q, ++j) {
                    const int s = j % STAGES;
                    wait_bounded<true>(&bar_full[s], (j / STAGES) & 1, g);
                    ptx::tc_fence_after();
                    const uint32_t sa = base + s * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_pair<C::FP8>(tmem + ab * BN, C::A_MN ? desc_mn(sa, kk) : desc_k(sa, kk),
                                              C::B_MN ? desc_mn(sb, kk) : desc_k(sb, kk), idesc,
                                              (q > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit_pair(&bar_empty[s]);
                }
                ptx::mma_commit_pair(&bar_acc_full[ab]);
            }
            // every MMA must have finished before TMEM is released (matters after a timeout)
            for (int b = 0; b < 2 && b < li; ++b) {
                const int last = li - 1 - ((li - 1 - b) & 1);
                wait_bounded(&bar_acc_full[last & 1], (last >> 1) & 1, g);
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, set = (warp - 4) >> 2, ew = warp - 4;
        uint8_t *buf = smem + STAGES * C::STAGE + ew * 8192;
        uint64_t *rbar = bar_res + 2 * ew;
        uint32_t rphase = 0;   // bit b: the parity the next load into buffer b completes
        const uint32_t sbuf = ptx::smem_u32(buf);
        const uint32_t empty0 = ptx::cluster_addr(ptx::smem_u32(&bar_acc_empty[0]), 0);
        const uint32_t empty1 = ptx::cluster_addr(ptx::smem_u32(&bar_acc_empty[1]), 0);
        int li = 0;
        for (int item = cluster; item < p.n_items; item += n_clusters, ++li) {
            int ks, mt, nt, k_begin, nk;
            decode(item, ks, mt, nt, k_begin, nk);
            const int ab = li & 1;
            const int grp = mt / p.mblocks, i0 = (mt % p.mblocks) * BM + (int)rank * 128 + quarter * 32;
            const int n0 = nt * BN;
            const bool rows = i0 < p.T;
            // buffer of chunk j: alternating, or both for y and z
            auto load_res = [&](int col, int b) {
                ptx::mbar_arrive_expect_tx(&rbar[b], 4096);
                ptx::tma_load_3d(buf + b * 4096, &maps.r, &rbar[b], col, i0, grp);
            };
            if (lane == 0) {
                ptx::bulk_wait_group_read<0>();   // the buffers are free again
                if (p.has_r && rows) {
                    if (n0 + set * 64 < p.N) load_res(n0 + set * 64, 0);
                    if (!p.has_z && BN == 256 && n0 + set * 64 + 128 < p.N) load_res(n0 + set * 64 + 128, 1);
                }
            }
            __syncwarp();
            const float xs = (P == FwdQ8 && i0 + lane < p.T) ? p.x_scale[i0 + lane] : 0.f;
            wait_bounded(&bar_acc_full[ab], (li >> 1) & 1, g);
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * BN;
#pragma unroll 1
            for (int j = 0; j < BN / 128; ++j) {
                const int c0 = set * 64 + j * 128, col0 = n0 + c0;
                if (col0 >= p.N || !rows) break;
                const int b = p.has_z ? 0 : j;
                if (p.has_z && j > 0) {
                    if (lane == 0) {
                        ptx::bulk_wait_group_read<0>();
                        if (p.has_r) load_res(col0, 0);
                    }
                    __syncwarp();
                }
                if (p.has_r) {
                    wait_bounded(&rbar[b], (rphase >> b) & 1, g);
                    rphase ^= 1u << b;
                }
                const uint32_t yrow = sbuf + b * 4096 + lane * 128, zrow = sbuf + 4096 + lane * 128;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[32];
                    ptx::tmem_ld32(taddr + c0 + half * 32, v);
                    ptx::tmem_ld_wait();
                    reg_fence(v);
                    if (P == Dw && p.part) {   // fp32 partial sums, a 128-byte line a thread
                        if (i0 + lane < p.T) {
                            float *dst = p.part + ((size_t)ks * p.T + i0 + lane) * p.N + col0 + half * 32;
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (col0 + half * 32 + 4 * q < p.N)
                                    reinterpret_cast<uint4 *>(dst)[q] =
                                        make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        }
                        continue;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {   // 8 columns: 16 bytes of the row
                        const int col = col0 + half * 32 + q * 8;
                        const uint32_t off = (uint32_t)(((half * 4 + q) ^ (lane & 7)) << 4);
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * q + e]);
                        if (P == Fwd || P == FwdQ8) {
                            if (col < p.N) {
                                if (P == FwdQ8) {
                                    const float4 s0 = __ldg(reinterpret_cast<const float4 *>(p.w_scale + col));
                                    const float4 s1 = __ldg(reinterpret_cast<const float4 *>(p.w_scale + col) + 1);
                                    f[0] *= xs * s0.x; f[1] *= xs * s0.y; f[2] *= xs * s0.z; f[3] *= xs * s0.w;
                                    f[4] *= xs * s1.x; f[5] *= xs * s1.y; f[6] *= xs * s1.z; f[7] *= xs * s1.w;
                                }
                                if (p.bias) {
                                    const float4 b0 = __ldg(reinterpret_cast<const float4 *>(p.bias + col));
                                    const float4 b1 = __ldg(reinterpret_cast<const float4 *>(p.bias + col) + 1);
                                    f[0] += b0.x; f[1] += b0.y; f[2] += b0.z; f[3] += b0.w;
                                    f[4] += b1.x; f[5] += b1.y; f[6] += b1.z; f[7] += b1.w;
                                }
                            }
                            if (p.has_z)
                                sts_u128(zrow + off, make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                                                ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7])));
                            if (p.act != ATTN_ACT_NONE) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) f[e] = activate(f[e], p.act);
                            }
                            if (p.has_r) {
                                const uint4 r = lds_u128(yrow + off);
                                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    f[2 * e] += __uint_as_float(w[e] << 16);
                                    f[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
                                }
                            }
                        }
                        sts_u128(yrow + off, make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                                        ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7])));
                    }
                }
                if (!(P == Dw && p.part)) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (P == Dx)
                            ptx::tma_store_3d(&maps.y, buf + b * 4096, col0 % p.dk, i0, grp * p.H + col0 / p.dk);
                        else
                            ptx::tma_store_3d(&maps.y, buf + b * 4096, col0, i0, grp);
                        if (p.has_z) ptx::tma_store_3d(&maps.z, buf + 4096, col0, i0, grp);
                        ptx::bulk_commit_group();
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster(ab ? empty1 : empty0);
        }
        if (lane == 0) ptx::bulk_wait_group<0>();
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // neither CTA leaves while the other may read its shared memory or signal it
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, C::TM_COLS);
    }
}

// dz = dy act'(z) in bf16, and the column sums of the unrounded dz over a block of rows.  A warp
// takes a row's 256 columns at a time (8 a thread, 16 bytes), the block's 8 warps neighbouring rows.
__global__ void __launch_bounds__(256) dz_kernel(const LinBwdArgs a, int blocks)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x * 256 + lane * 8;
    __shared__ float part[8][256];
    float s[8] = {};
    if (n < a.N) {
        const int per = (a.M + blocks - 1) / blocks;
        const long long m_end = min((long long)a.M, (long long)(blockIdx.y + 1) * per);
        for (long long m = (long long)blockIdx.y * per + warp; m < m_end; m += 8) {
            const size_t at = ((size_t)m * a.N + n) / 8;
            const uint4 d4 = static_cast<const uint4 *>(a.dy)[at];
            const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(d[e] << 16);
                f[2 * e + 1] = __uint_as_float(d[e] & 0xffff0000u);
            }
            if (a.z) {
                const uint4 z4 = static_cast<const uint4 *>(a.z)[at];
                const uint32_t z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] *= act_slope(__uint_as_float(z[e] << 16), a.act);
                    f[2 * e + 1] *= act_slope(__uint_as_float(z[e] & 0xffff0000u), a.act);
                }
                static_cast<uint4 *>(a.dz)[at] = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                                            ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7]));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
        }
    }
    if (!a.dbias) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][lane * 8 + e] = s[e];
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.N) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
    a.col_part[(size_t)blockIdx.y * a.N + c] = t;
}

// dw = the sum of the partial sums, in order, rounded once; 4 elements a thread.
__global__ void __launch_bounds__(256) dw_join_kernel(const float *part, void *dw, int splits, long long elems)
{
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= elems) return;
    float4 s = *reinterpret_cast<const float4 *>(part + i);
    for (int k = 1; k < splits; ++k) {
        const float4 t = *reinterpret_cast<const float4 *>(part + k * elems + i);
        s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
    }
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(dw) + i) =
        make_uint2(ptx::pack_bf16x2(s.x, s.y), ptx::pack_bf16x2(s.z, s.w));
}

// ------------------------------------------------------------------ launches
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// The pairs the plans are made for (a function of the sizes alone, so that results and workspaces
// do not depend on where the plan is made): a GB300's 152 SMs.
constexpr int kPlanPairs = 76;

template <Policy P, int BN>
cudaError_t launch_pair(const GemmMaps &m, const GemmParams &p, cudaStream_t stream)
{
    using C = Cfg<P, BN>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(gemm_pair_kernel<P, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    const int pairs = device_sm_count() / 2;
    gemm_pair_kernel<P, BN><<<2 * (p.n_items < pairs ? p.n_items : pairs), 384, C::SMEM, stream>>>(m, p);
    return cudaGetLastError();
}

bool set_items(GemmParams &p, int splits)
{
    const long long items = (long long)p.n_mtiles * p.n_ntiles * splits;
    p.n_items = (int)items;
    return items <= 0x7fffffffLL;
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;

// Whether 256-column tiles give every pair of CTAs a tile; else 128-column ones spread the work
// over more of them.
bool wide_tiles(long long mtiles, int N) { return mtiles * ceil_div(N, 256) >= kPlanPairs; }

struct DwPlan {
    bool wide;
    int splits, steps_per_split;
};

// dw has few tiles (K x N) and a long sum (the rows), so the rows are split over pairs of CTAs where
// the partial sums' traffic costs less than the idle pairs: the plan takes the least of
//   rounds of items per pair x steps per item x time of a step  +  partial sums written and read.
// 0.27 us: a step of a 256 x 256 tile at the tensor cores' rate; 5 bytes/ps: what the join reads at.
DwPlan dw_plan(int G, int T, int K, int N)
{
    const long long steps = (long long)G * ceil_div(T, 64), mt = ceil_div(K, BM);
    DwPlan best{true, 1, (int)steps};
    double best_t = 1e30;
    for (int wide = 1; wide >= 0; --wide) {
        const long long tiles = mt * ceil_div(N, wide ? 256 : 128);
        for (int s = 1; s <= 16 && s <= steps; ++s) {
            const long long per = (steps + s - 1) / s;
            if ((steps + per - 1) / per != s) continue;
            double t = (double)((tiles * s + kPlanPairs - 1) / kPlanPairs) * (per * (wide ? 0.27 : 0.16) + 1.5);
            if (s > 1) t += 2.5 + (double)s * K * N * 8 / 5e6;
            if (t < best_t) {
                best_t = t;
                best = DwPlan{wide == 1, s, (int)per};
            }
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_linear(const LinArgs &a, cudaStream_t stream)
{
    GemmParams p = {};
    p.T = a.T;
    p.mblocks = ceil_div(a.T, BM);
    p.n_mtiles = p.mblocks * a.G;   // at most M
    p.N = a.N;
    p.dk = a.dk;
    p.H = a.H;
    p.bias = a.bias;
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.has_z = a.z != nullptr;
    p.has_r = a.residual != nullptr;
    p.act = a.act;
    p.status = a.status;
    const bool wide = wide_tiles(p.n_mtiles, a.N);
    const int bn = wide ? 256 : 128;
    p.n_ntiles = ceil_div(a.N, bn);
    if (!set_items(p, 1)) return cudaErrorInvalidValue;
    p.ksteps = p.steps_per_split = ceil_div(a.K, a.q8 ? 128 : 64);
    GemmMaps m;
    CUresult r;
    if (a.q8) {
        r = make_map_3d(&m.a, a.x, kU8, 1, a.K, a.M, 1, 128, 128);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kU8, 1, a.K, a.N, 1, 128, bn / 2);
    } else {
        r = make_map_3d(&m.a, a.x, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 128);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kBf16, 2, a.N, a.K, 1, 64, 64);
    }
    if (r == CUDA_SUCCESS) r = make_map_3d(&m.y, a.y, kBf16, 2, a.N, a.T, a.G, 64, 32);
    if (r == CUDA_SUCCESS && a.z) r = make_map_3d(&m.z, a.z, kBf16, 2, a.N, a.T, a.G, 64, 32);
    if (r == CUDA_SUCCESS && a.residual) r = make_map_3d(&m.r, a.residual, kBf16, 2, a.N, a.T, a.G, 64, 32);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    if (a.q8)
        return wide ? launch_pair<FwdQ8, 256>(m, p, stream) : launch_pair<FwdQ8, 128>(m, p, stream);
    return wide ? launch_pair<Fwd, 256>(m, p, stream) : launch_pair<Fwd, 128>(m, p, stream);
}

// Blocks of rows of the column sums: enough for four blocks of threads an SM, at least 16 rows each.
int lin_bwd_row_blocks(int M, int N)
{
    const int strips = ceil_div(N, 256);
    const int want = ceil_div(8 * kPlanPairs, strips), most = ceil_div(M, 16);
    const int b = want < most ? want : most;
    return b > 1 ? b : 1;
}

int lin_dw_splits(int G, int T, int K, int N) { return T > 0 ? dw_plan(G, T, K, N).splits : 1; }

cudaError_t launch_linear_bwd(const LinBwdArgs &a, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (a.dbias || (a.z && (a.dx || a.dw))) {
        const int blocks = lin_bwd_row_blocks(a.M, a.N);
        dz_kernel<<<dim3(ceil_div(a.N, 256), blocks), 256, 0, stream>>>(a, blocks);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (a.dbias) {
            if ((e = launch_sum_rows(a.col_part, a.dbias, blocks, a.N, stream)) != cudaSuccess) return e;
        }
    }
    const void *dz = a.z ? a.dz : a.dy;
    GemmMaps m;
    CUresult r;
    if (a.dx) {
        GemmParams p = {};
        p.T = a.T;
        p.mblocks = ceil_div(a.T, BM);
        p.n_mtiles = p.mblocks * a.G;
        p.N = a.K;
        p.dk = a.dk;
        p.H = a.H;
        p.status = a.status;
        const bool wide = wide_tiles(p.n_mtiles, a.K);
        const int bn = wide ? 256 : 128;
        p.n_ntiles = ceil_div(a.K, bn);
        if (!set_items(p, 1)) return cudaErrorInvalidValue;
        p.ksteps = p.steps_per_split = ceil_div(a.N, 64);
        r = make_map_3d(&m.a, dz, kBf16, 2, a.N, a.T, a.G, 64, 128);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kBf16, 2, a.N, a.K, 1, 64, bn / 2);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.y, a.dx, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 32);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
        e = wide ? launch_pair<Dx, 256>(m, p, stream) : launch_pair<Dx, 128>(m, p, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.dw) {
        const DwPlan plan = dw_plan(a.G, a.T, a.K, a.N);
        GemmParams p = {};
        p.T = a.K;
        p.mblocks = p.n_mtiles = ceil_div(a.K, BM);
        p.N = a.N;
        p.dk = a.dk;
        p.H = a.H;
        p.status = a.status;
        p.n_ntiles = ceil_div(a.N, plan.wide ? 256 : 128);
        p.tblocks = ceil_div(a.T, 64);
        p.ksteps = a.G * p.tblocks;
        p.steps_per_split = plan.steps_per_split;
        if (!set_items(p, plan.splits)) return cudaErrorInvalidValue;
        p.part = plan.splits > 1 ? a.dw_part : nullptr;
        r = make_map_3d(&m.a, a.x, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 64);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, dz, kBf16, 2, a.N, a.T, a.G, 64, 64);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.y, a.dw, kBf16, 2, a.N, a.K, 1, 64, 32);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
        e = plan.wide ? launch_pair<Dw, 256>(m, p, stream) : launch_pair<Dw, 128>(m, p, stream);
        if (e == cudaSuccess && plan.splits > 1) {
            const long long elems = (long long)a.K * a.N;
            dw_join_kernel<<<ceil_div(elems, 1024), 256, 0, stream>>>(a.dw_part, a.dw, plan.splits, elems);
            e = cudaGetLastError();
        }
    }
    return e;
}

}  // namespace attn
