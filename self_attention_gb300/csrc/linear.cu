// Linear layers on tcgen05 tensor cores: y = act(x w + b) + r forward, dx = dz w^T and dw = x^T dz
// backward, and the forward in e4m3.  One persistent GEMM skeleton over pairs of CTAs,
// C[256 x BN] = sum over K steps of A B, with operand policies:
//   Fwd   : A = x (K-major), B = w [K, N] (MN-major).
//   FwdQ8 : A = xq, B = wq [N, K], both K-major, e4m3.
//   Bwd   : dx with A = dz, B = w (both K-major: the rows of w are the columns of dx), and dw with
//           A = x^T, B = dz (both MN-major), its K steps 64 rows each, in one launch.
// x (and dx) may be split by heads, [G, H, T, dk] with row m = g T + i and column c = h dk + e: a
// 64-column box lies in one head, so only the coordinates of the copies differ.  A row block (and, for
// dw, a step) lies in one group g; the copies' zero fill and clipping end it at the group's last row.
//
// A cluster of two CTAs computes a 256 x BN tile together (tcgen05 cta_group::2): each loads 128 rows
// of A and BN / 2 columns of B a step, 32 KB for 2 x 128 x 256 x 64 multiply-adds where a single CTA
// with the same tile of its own would load 48 KB, which is what bounds the K loop (L2 bandwidth and
// the reads of shared memory).  Each CTA: warp 0 TMA producer, warp 1 tcgen05 issuer (even CTA),
// warps 4-19 epilogue; the accumulator is double-buffered in TMEM, so a tile's epilogue overlaps the
// products of the next.
//
// Epilogue: a warp owns 32 rows x 64 columns of a tile (thread = row): TMEM -> registers, scales, bias,
// activation, residual in fp32, one rounding to bf16, a swizzled 4 KB buffer in shared memory, TMA
// stores.  The residual comes the same way round, by a TMA load into that buffer before the accumulator
// is ready.  Sixteen warps, since a warp's chain of loads, MUFU operations and stores is long: with
// eight, GELU with z kept took a tenth longer at 32768 x 1024 x 4096.
//
// What bounds it: the products and, over a second or more of them, the power limit (32768 rows, 1024 x
// 4096, in long runs at 1.5 to 1.6 GHz: 177 us without an activation, 1.55 PFLOP/s, 191 with GELU, 215
// with z kept as well, 194 in short runs; 8192^3 in short runs: 585 us, 1.88 PFLOP/s, e4m3 309 us, 3.56
// PFLOP/s).  Shared memory is nearly full too: operands written (64 B a cycle) and read (64), so each 64
// KB that the epilogue writes and reads back shows.  With short K the epilogue's own chain counts: 1.9
// us a tile (32768 x 64 x 4096: 56 us, 4.9 TB/s).  Measured and not kept: copying the buffers out by
// 128-byte lines instead of TMA (4 % slower with z kept, 2 % without), storing z straight from
// registers (7 %).
#include "act.cuh"
#include "cluster.cuh"
#include "kernels.h"
#include "sum_rows.cuh"

namespace attn {
namespace {

constexpr int BM = 256;            // rows of a tile (both CTAs)
constexpr int kEpiWarps = 16;      // four for each 32 rows of a CTA, each with 64 of 256 columns
constexpr int kGroupM = 8;         // row tiles walked side by side, for reuse of B in L2

// n / d for 0 <= n < 2^31 by a multiplication (the epilogue warps decode an item in their critical path,
// where each integer division takes 0.1 us): q = (hi(n m) + n) >> s with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1.
struct FastDiv {
    unsigned m, s, d;
    __device__ int div(int n) const { return (int)((__umulhi((unsigned)n, m) + (unsigned)n) >> s); }
};

FastDiv fast_div(int d)
{
    unsigned s = 0;
    while ((1ull << s) < (unsigned long long)d) ++s;
    return FastDiv{(unsigned)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, (unsigned)d};
}

struct GemmMaps {
    CUtensorMap a, b, y;       // Fwd, FwdQ8; Bwd: of dx
    CUtensorMap a2, b2, y2;    // Bwd: of dw; Fwd, FwdQ8: a2 the residual, y2 z
};

// One product: rows in groups, tiles, steps.
struct Prob {
    int T;                         // rows of one group
    int rb_log2, n_rblocks;        // rows of a row block, row blocks of all groups
    FastDiv rblocks;               // row blocks of one group
    int n_mtiles, n_ntiles, N;     // row tiles, column tiles, columns
    FastDiv tiles, per_group;      // tiles of a K split, of kGroupM row tiles
    int dk, H;                     // the head split of the side that has one (A; dx: y)
    int ksteps, steps_per_split;   // K steps in all and per item
    int tblocks, T_k;              // dw: steps and rows of one group
    int n_items;
};

struct GemmParams {
    Prob q[2];                     // [0] Fwd, FwdQ8, dx; [1] dw
    const float *bias, *x_scale, *w_scale;
    int has_z, has_r, act;
    // Bwd: items of dx each cluster takes, and how many more those from a_clusters on take first; whether
    // y2 maps [splits][rows][N] fp32 partial sums
    int x_all, x_early, a_clusters, part;
    // Bwd, the bias gradient: either col_rows partial rows to add up into dbias, or (sum_x) rows of dy to
    // add up, per_slice at a time, into `slices` partial rows, or all at once (slices = 0) into dbias
    float *col_part, *dbias;
    int col_rows, col_n;
    const __nv_bfloat16 *sum_x;
    int sum_m, per_slice, slices;
    int *status;
};

enum Policy { Fwd, FwdQ8, Bwd, Dx /* split kernel only */ };

template <Policy P, int BN>
struct Cfg {
    static constexpr bool FP8 = P == FwdQ8;
    static constexpr int KE = FP8 ? 128 : 64;              // elements of K a step: 128 bytes
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int EPI = kEpiWarps * 4096;           // a 32 x 64 bf16 buffer for each epilogue warp
    static constexpr int SMEM = STAGES * STAGE + EPI + 1024;
    static constexpr uint32_t TM_COLS = 2 * BN;
    // The epilogue warps that take an item: with 128 columns half of them, the other half the next item.
    static constexpr int TAKERS = kEpiWarps * BN / 256;
};

// K-major rows of 128 bytes: the k-th 32-byte slice starts 32 bytes in.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) { return ptx::sdesc_sw128(base + kk * 32, 16, 1024); }
// MN-major: 64-column blocks of 64 K rows (8 KB each); a slice is 16 K rows.
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk)
{
    return ptx::sdesc_sw128(base + kk * 2048, 8192, 1024);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

// Four pairs of fp32 -> eight bf16, rounded to nearest even.
__device__ __forceinline__ uint4 pack_bf16x8(const uint64_t *f)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        ptx::f2_unpack(f[e], lo, hi);
        w[e] = ptx::pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 pack_bf16x4(const uint64_t (&f)[2])
{
    float a, b, c, d;
    ptx::f2_unpack(f[0], a, b);
    ptx::f2_unpack(f[1], c, d);
    return make_uint2(ptx::pack_bf16x2(a, b), ptx::pack_bf16x2(c, d));
}

__device__ __forceinline__ void prefetch_l1(const void *p)
{
    asm volatile("prefetch.global.L1 [%0];" ::"l"(__cvta_generic_to_global(p)) : "memory");
}

template <Policy P, int BN>
__global__ void __launch_bounds__(128 + 32 * kEpiWarps, 1)
    gemm_pair_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p)
{
    using C = Cfg<P, BN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    __shared__ uint64_t bar_full[STAGES], bar_empty[STAGES], bar_acc_full[2], bar_acc_empty[2], bar_res[kEpiWarps];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    // The cluster's items: Fwd every n_clusters-th tile.  Bwd: its share of dw's (w = 1), then as many of
    // dx's as fill it up to the others' level.  The clusters with less of dw deal out the first of dx's
    // items among themselves, then all of them deal out the rest: at any time they work on neighbouring
    // tiles, whose operands L2 then holds.
    const int n_dw = P == Bwd && cluster < p.q[1].n_items ? (p.q[1].n_items - cluster - 1) / n_clusters + 1 : 0;
    const int early = P == Bwd && cluster >= p.a_clusters ? p.x_early : 0;
    auto item_at = [&](int li, int &w, int &item) {
        w = li < n_dw;
        if (P != Bwd || w) {
            item = cluster + li * n_clusters;
            return w || item < p.q[0].n_items;
        }
        const int j = li - n_dw;
        if (j >= early + p.x_all) return false;
        const long long at = j < early ? (long long)j * (n_clusters - p.a_clusters) + cluster - p.a_clusters
                                       : (long long)p.x_early * (n_clusters - p.a_clusters) +
                                             (long long)(j - early) * n_clusters + cluster;
        item = (int)min(at, (long long)p.q[0].n_items);
        return item < p.q[0].n_items;
    };
    // item -> K range, row tile, column tile: kGroupM row tiles side by side, column by column
    auto decode = [&](const Prob &q, int item, int &ks, int &mt, int &nt, int &k_begin, int &nk) {
        ks = q.tiles.div(item);
        const int t = item - ks * (int)q.tiles.d, group = q.per_group.div(t);
        const int first = group * kGroupM, r = t - group * (int)q.per_group.d, rows = q.n_mtiles - first;
        if (rows >= kGroupM) {
            nt = r / kGroupM;
            mt = first + r % kGroupM;
        } else {   // the last, smaller group
            nt = r / rows;
            mt = first + r - nt * rows;
        }
        k_begin = ks * q.steps_per_split;
        nk = min(q.steps_per_split, q.ksteps - k_begin);
    };
    // row block -> group, first row
    auto locate = [&](const Prob &q, int block, int &grp, int &row) {
        grp = q.rblocks.div(block);
        row = (block - grp * (int)q.rblocks.d) << q.rb_log2;
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
            ptx::mbar_init(&bar_acc_empty[b], 2 * C::TAKERS);   // the epilogue warps of both CTAs
        }
        for (int b = 0; b < kEpiWarps; ++b) ptx::mbar_init(&bar_res[b], 1);
        ptx::fence_mbar_init();
    }
    if (warp == 2 && ptx::elect_one()) {   // (of the maps that there are)
        if (P != Bwd || p.q[0].n_items > 0) {
            ptx::tma_prefetch_desc(&maps.a);
            ptx::tma_prefetch_desc(&maps.b);
        }
        if (P == Bwd ? p.q[1].n_items > 0 : p.has_r) ptx::tma_prefetch_desc(&maps.a2);
        if (P == Bwd && p.q[1].n_items > 0) ptx::tma_prefetch_desc(&maps.b2);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&tmem_sh, C::TM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // both CTAs' barriers exist before either signals the other
    ptx::tc_fence_after();
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const uint32_t tmem = tmem_sh;

    if (warp == 0) {
        if (ptx::elect_one()) {
            int s = 0;          // place in the stage ring, and the parity of its turn, across items
            uint32_t ph = 0;
            const uint32_t full0 = ptx::cluster_addr(ptx::smem_u32(&bar_full[0]), 0);
            int w, item;
            for (int li = 0; item_at(li, w, item); ++li) {
                const Prob &pr = p.q[P == Bwd ? w : 0];
                int ks, mt, nt, k_begin, nk;
                decode(pr, item, ks, mt, nt, k_begin, nk);
                // this CTA's 128 rows: one block of 128, or four of 32 that may lie in different groups
                const int per_cta = 128 >> pr.rb_log2, block0 = (mt * 2 + (int)rank) * per_cta;
                int grp[4], i0[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) locate(pr, block0 + h, grp[h], i0[h]);
                const int n0 = nt * BN + (int)rank * (BN / 2);
                // K is walked without divisions, which would take this one thread longer than a step
                auto turn = [&] {   // the next stage is free; both CTAs' copies complete on the even one's barrier
                    wait_bounded(&bar_empty[s], ph ^ 1, g);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&bar_full[s], 2 * C::STAGE);
                };
                auto next = [&] {
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                };
                if (P == Bwd && w) {   // dw: 64 rows t0.. of group gk
                    int gk = k_begin / pr.tblocks, t0 = (k_begin - gk * pr.tblocks) * 64, col[2], head[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        head[h] = (i0[0] + 64 * h) / pr.dk;
                        col[h] = i0[0] + 64 * h - head[h] * pr.dk;
                    }
                    for (int q = 0; q < nk; ++q) {
                        turn();
                        const uint32_t bar = full0 + s * 8;
                        uint8_t *sa = smem + s * C::STAGE, *sb = sa + C::A_BYTES;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            ptx::tma_load_3d_pair(sa + h * 8192, &maps.a2, bar, col[h], t0, gk * pr.H + head[h]);
#pragma unroll
                        for (int h = 0; h < BN / 128; ++h)
                            ptx::tma_load_3d_pair(sb + h * 8192, &maps.b2, bar, n0 + 64 * h, t0, gk);
                        t0 += 64;
                        if (t0 >= pr.T_k) {
                            t0 = 0;
                            ++gk;
                        }
                        next();
                    }
                } else {   // column c of A: ce of head ch
                    int c = k_begin * C::KE, ch = P == Fwd ? c / pr.dk : 0, ce = c - ch * pr.dk;
                    if (P != Fwd) ce = c;
                    const int heads = P == Bwd ? 1 : pr.H;
                    for (int q = 0; q < nk; ++q) {
                        turn();
                        const uint32_t bar = full0 + s * 8;
                        uint8_t *sa = smem + s * C::STAGE, *sb = sa + C::A_BYTES;
                        ptx::tma_load_3d_pair(sa, &maps.a, bar, ce, i0[0], grp[0] * heads + ch);
                        if (per_cta == 4)
#pragma unroll
                            for (int h = 1; h < 4; ++h)
                                ptx::tma_load_3d_pair(sa + h * 4096, &maps.a, bar, ce, i0[h], grp[h] * heads + ch);
                        if (P == Fwd) {
#pragma unroll
                            for (int h = 0; h < BN / 128; ++h)
                                ptx::tma_load_3d_pair(sb + h * 8192, &maps.b, bar, n0 + 64 * h, c, 0);
                        } else {
                            ptx::tma_load_3d_pair(sb, &maps.b, bar, c, n0, 0);
                        }
                        c += C::KE;
                        ce += C::KE;
                        if (P == Fwd && ce >= pr.dk) {
                            ce = 0;
                            ++ch;
                        }
                        next();
                    }
                }
            }
            // The last turn of every stage has been consumed (a stage that had none passes at once): no copy
            // is in flight, and no arrival on this CTA's barriers, when it leaves.
            for (int q = 0; q < STAGES; ++q) wait_bounded(&bar_empty[q], q < s ? ph : ph ^ 1, g);
        }
    } else if (warp == 1 && rank == 0) {
        if (ptx::elect_one()) {
            const uint32_t base = ptx::smem_u32(smem);
            int s = 0, li = 0, w, item;
            uint32_t ph = 0;
            for (; item_at(li, w, item); ++li) {
                const Prob &pr = p.q[P == Bwd ? w : 0];
                int ks, mt, nt, k_begin, nk;
                decode(pr, item, ks, mt, nt, k_begin, nk);
                const bool a_mn = P == Bwd && w, b_mn = P == Fwd || a_mn;
                const uint32_t idesc = C::FP8 ? ptx::idesc_f16_f32(BM, BN, false, false)   // format 0: e4m3
                                              : ptx::idesc_bf16_f32(BM, BN, a_mn, b_mn);
                const int ab = li & 1;
                wait_bounded(&bar_acc_empty[ab], ((li >> 1) & 1) ^ 1, g);   // epilogues of item li-2 done
                ptx::tc_fence_after();
                for (int q = 0; q < nk; ++q) {
                    wait_bounded(&bar_full[s], ph, g);
                    ptx::tc_fence_after();
                    const uint32_t sa = base + s * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_pair<C::FP8>(tmem + ab * BN, a_mn ? desc_mn(sa, kk) : desc_k(sa, kk),
                                              b_mn ? desc_mn(sb, kk) : desc_k(sb, kk), idesc,
                                              (q > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit_pair(&bar_empty[s]);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                ptx::mma_commit_pair(&bar_acc_full[ab]);
            }
            // every MMA must have finished before TMEM is released (matters after a timeout), and the last
            // arrivals from the odd CTA must have come in before this one leaves
            for (int b = 0; b < 2 && b < li; ++b) {
                const int last = li - 1 - ((li - 1 - b) & 1);
                wait_bounded(&bar_acc_full[last & 1], (last >> 1) & 1, g);
                wait_bounded(&bar_acc_empty[last & 1], (last >> 1) & 1, g);
            }
        }
    } else if (warp >= 4) {
        // sets of four warps: with 256 columns a set takes 64 of every item, with 128 of every second one
        const int quarter = warp & 3, ew = warp - 4, set = (ew >> 2) % (BN / 64), turn = (ew >> 2) / (BN / 64);
        uint8_t *buf = smem + STAGES * C::STAGE + ew * 4096;
        uint64_t *rbar = bar_res + ew;
        uint32_t rphase = 0;
        const uint32_t sbuf = ptx::smem_u32(buf), row = sbuf + lane * 128;
        const uint32_t empty0 = ptx::cluster_addr(ptx::smem_u32(&bar_acc_empty[0]), 0);
        int w, item;
        for (int li = 0; item_at(li, w, item); ++li) {
            if (BN == 128 && (li & 1) != turn) continue;   // (and so the same accumulator every time)
            const Prob &pr = p.q[P == Bwd ? w : 0];
            int ks, mt, nt, k_begin, nk;
            decode(pr, item, ks, mt, nt, k_begin, nk);
            const int ab = li & 1;
            const int first = mt * BM + (int)rank * 128 + quarter * 32, block = first >> pr.rb_log2;
            int grp, i0;
            locate(pr, block, grp, i0);
            i0 += first & ((1 << pr.rb_log2) - 1);
            const int col0 = nt * BN + set * 64;
            const bool mine = col0 < pr.N && i0 < pr.T && block < pr.n_rblocks;
            // The residual of the warp's 64 columns, or (beside z) of 32 of them behind the half for z.
            auto load_res = [&](int half) {
                ptx::mbar_arrive_expect_tx(rbar, p.has_z ? 2048 : 4096);
                ptx::tma_load_3d(buf + (p.has_z ? 2048 : 0), &maps.a2, rbar, col0 + half * 32, i0, grp);
            };
            auto wait_res = [&] {
                wait_bounded(rbar, rphase, g);
                rphase ^= 1;
            };
            // f += the residual's 8 columns at `addr`
            auto add_res = [&](uint64_t *f, uint32_t addr) {
                const uint4 r = lds_u128(addr);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = ptx::add_f32x2(f[e], ptx::f2_pack(__uint_as_float(w[e] << 16),
                                                             __uint_as_float(w[e] & 0xffff0000u)));
            };
            // Leaves the buffer to a TMA store.
            auto store = [&](const CUtensorMap *map, int c, int slice) {
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_3d(map, buf, c, i0, slice);
                    ptx::bulk_commit_group();
                }
            };
            // The buffer is free again.
            auto reclaim = [&] {
                if (lane == 0) ptx::bulk_wait_group_read<0>();
                __syncwarp();
            };
            reclaim();
            if (lane == 0 && p.has_r && mine) load_res(0);
            // what load_z reads is on its way to L1 while the warp waits for the accumulator
            if (P == Fwd || P == FwdQ8) {
                const int c = col0 + (lane & 1) * 32;
                if (lane < 2 && mine && c < pr.N) {
                    if (p.bias) prefetch_l1(p.bias + c);
                    if (P == FwdQ8) prefetch_l1(p.w_scale + c);
                }
            }
            const uint64_t xs = f2_both((P == FwdQ8 && mine && i0 + lane < pr.T) ? p.x_scale[i0 + lane] : 0.f);
            wait_bounded(&bar_acc_full[ab], (li >> 1) & 1, g);
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * BN + set * 64;
            auto release = [&] {   // this warp has read its part of the accumulator
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_remote(empty0 + ab * 8);
            };
            if (!mine) {
                release();
                continue;
            }
            if (P == Bwd && w && p.part) {   // fp32 partial sums: 32 columns are a 128-byte row
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[32];
                    ptx::tmem_ld32(taddr + half * 32, v);
                    ptx::tmem_ld_wait();
                    reg_fence(v);
                    if (half) {
                        release();
                        reclaim();
                    }
                    if (col0 + half * 32 >= pr.N) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        sts_u128(row + ((q ^ (lane & 7)) << 4),
                                 make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
                    store(&maps.y2, col0 + half * 32, ks);
                }
                continue;
            }
            // z (or, without scales and bias, the sums) of 32 columns, as pairs
            auto load_z = [&](int half, uint64_t (&f)[16]) {
                uint32_t v[32];
                ulonglong2 bias[8];
                if constexpr (P == Fwd) {   // asked for ahead of the wait for the accumulator
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int col = col0 + half * 32 + q * 4;
                        bias[q] = p.bias && col < pr.N ? *reinterpret_cast<const ulonglong2 *>(p.bias + col)
                                                       : make_ulonglong2(0, 0);
                    }
                }
                ptx::tmem_ld32(taddr + half * 32, v);
                ptx::tmem_ld_wait();
                reg_fence(v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    f[i] = ptx::f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
#pragma unroll
                for (int q = 0; q < 8; ++q) {   // 4 columns
                    if constexpr (P == FwdQ8) {
                        const int col = col0 + half * 32 + q * 4;
                        ulonglong2 b = make_ulonglong2(0, 0), ws = b;
                        if (p.bias && col < pr.N) b = *reinterpret_cast<const ulonglong2 *>(p.bias + col);
                        if (col < pr.N) ws = *reinterpret_cast<const ulonglong2 *>(p.w_scale + col);
                        f[2 * q] = ptx::fma_f32x2(f[2 * q], ptx::mul_f32x2(ws.x, xs), b.x);
                        f[2 * q + 1] = ptx::fma_f32x2(f[2 * q + 1], ptx::mul_f32x2(ws.y, xs), b.y);
                    } else if constexpr (P == Fwd) {
                        f[2 * q] = ptx::add_f32x2(f[2 * q], bias[q].x);
                        f[2 * q + 1] = ptx::add_f32x2(f[2 * q + 1], bias[q].y);
                    }
                }
            };
            if (P == Fwd && p.has_z) {
                // 32 columns at a time: z in the buffer's first half, y in the second (rows of 64 bytes, the
                // 16-byte chunk c of row r at c ^ (r / 2 & 3)); reading the accumulator costs too much beside
                // the products to take z in a pass of its own
                const uint32_t zrow = sbuf + lane * 64, swz = (lane >> 1) & 3;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint64_t f[16];
                    uint4 z[4];
                    load_z(half, f);
                    if (half) release();
                    if (col0 + half * 32 >= pr.N) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) z[q] = pack_bf16x8(f + 4 * q);
                    activate(f, p.act);
                    if (half) {
                        reclaim();
                        if (p.has_r && lane == 0) load_res(1);
                    }
                    if (p.has_r) wait_res();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at = zrow + ((q ^ swz) << 4);
                        sts_u128(at, z[q]);
                        if (p.has_r) add_res(f + 4 * q, at + 2048);
                        sts_u128(at + 2048, pack_bf16x8(f + 4 * q));
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_3d(&maps.y2, buf, col0 + half * 32, i0, grp);
                        ptx::tma_store_3d(&maps.y, buf + 2048, col0 + half * 32, i0, grp);
                        ptx::bulk_commit_group();
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                uint64_t f[16];
                load_z(half, f);
                if (half) release();
                if (P == Fwd || P == FwdQ8) activate(f, p.act);
                if ((P == Fwd || P == FwdQ8) && p.has_r && half == 0) wait_res();
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // 8 columns: 16 bytes of the row
                    const uint32_t at = row + (((half * 4 + q) ^ (lane & 7)) << 4);
                    if ((P == Fwd || P == FwdQ8) && p.has_r) add_res(f + 4 * q, at);
                    sts_u128(at, pack_bf16x8(f + 4 * q));
                }
            }
            if (P == Bwd && w)
                store(&maps.y2, col0, 0);
            else if (P == Bwd) {
                const int head = pr.H > 1 ? col0 >> (pr.dk == 64 ? 6 : 7) : 0;   // heads are 64 or 128 wide
                store(&maps.y, col0 - head * pr.dk, grp * pr.H + head);
            }
            else
                store(&maps.y, col0, grp);
        }
        if (lane == 0) ptx::bulk_wait_group<0>();   // complete before the CTA exits
    } else if (P == Bwd && warp >= 2) {
        // the bias gradient, by the two warps that have no other work, while the products run
        const int first = blockIdx.x * 2 + warp - 2, warps = gridDim.x * 2;
        if (p.sum_x && p.slices == 0) {   // dz is dy, of few rows: 64 columns a warp, 64 rows in flight
            const int from = lane >> 3;
            for (int c = first * 64; c < p.col_n; c += warps * 64) {
                const int n = c + (lane & 7) * 8;
                float s[8] = {};
                for (int m = from; m < p.sum_m; m += 64) {
                    uint4 v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[k] = m + 4 * k < p.sum_m && n < p.col_n
                                   ? *reinterpret_cast<const uint4 *>(p.sum_x + (size_t)(m + 4 * k) * p.col_n + n)
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float f[8];
                        unpack_bf16x8(v[k], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) s[e] += f[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[e] += __shfl_xor_sync(~0u, s[e], 8);
                    s[e] += __shfl_xor_sync(~0u, s[e], 16);
                }
                if (from == 0 && n < p.col_n) {
                    float4 *dst = reinterpret_cast<float4 *>(p.dbias + n);
                    dst[0] = make_float4(s[0], s[1], s[2], s[3]);
                    dst[1] = make_float4(s[4], s[5], s[6], s[7]);
                }
            }
        } else if (p.sum_x) {   // dz is dy: sums over slices of its rows, 8 columns a lane, 16 rows in flight
            for (int sl = first; sl < p.slices; sl += warps) {
                const long long m0 = (long long)sl * p.per_slice, m1 = min((long long)p.sum_m, m0 + p.per_slice);
                for (int n = lane * 8; n < p.col_n; n += 256) {
                    float s[8] = {};
                    for (long long m = m0; m < m1; m += 16) {
                        uint4 v[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            v[k] = m + k < m1 ? *reinterpret_cast<const uint4 *>(p.sum_x + (size_t)(m + k) * p.col_n + n)
                                              : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float f[8];
                            unpack_bf16x8(v[k], f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) s[e] += f[e];
                        }
                    }
                    float4 *dst = reinterpret_cast<float4 *>(p.col_part + (size_t)sl * p.col_n + n);
                    dst[0] = make_float4(s[0], s[1], s[2], s[3]);
                    dst[1] = make_float4(s[4], s[5], s[6], s[7]);
                }
            }
        } else {   // the partial sums of dz_kernel, 32 columns a warp
            for (int c = first * 32 + lane; c < p.col_n; c += warps * 32) {
                float s = 0.f;
#pragma unroll 16
                for (int r = 0; r < p.col_rows; ++r) s += p.col_part[(size_t)r * p.col_n + c];
                p.dbias[c] = s;
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    // neither CTA leaves while the other may read its shared memory or signal it (each has waited for what it
    // was sent: the even one for the accumulators' release, the odd one's producer for every stage's)
    ptx::cluster_sync_relaxed();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, C::TM_COLS);
    }
}

// Few rows: the weights are the large operand, and the time is what it takes to stream them.  The
// product is turned round, C^T[128 columns of y x TN rows] with the weights as the MMA's A operand, so
// that TN follows the number of rows, and K is split over the CTAs of a cluster, so that many SMs
// read (one 2048 x 8192 matrix is 64 column tiles).  Each CTA sends the rows of its partial tile to the
// CTAs that own them (row r to rank r mod splits), straight from tensor memory into their shared memory;
// after one cluster barrier each sums its rows over the ranks in order, applies the epilogue and stores.
// Where K is not split, each warp finishes its strip of the tile from tensor memory.
// (Leaving the partial tiles in place and fetching them takes a second barrier, and remote loads that
// are waited for: 1 us of 7 more.)  Up to TN = 64 two CTAs fit an SM.
struct SplitParams {
    int T, rb, rblocks, n_rblocks; // rows as in GemmParams, in tiles of TN
    int N, n_ntiles;               // columns of y, tiles of 128
    int dk, H;                     // the head split of A's side (Dx: of y)
    int ksteps, steps_per_cta;
    const float *bias, *x_scale, *w_scale;
    const __nv_bfloat16 *residual;
    __nv_bfloat16 *y, *z;
    int act;
    int *status;
};

template <Policy P, int TN>
struct SplitCfg {
    static constexpr bool FP8 = P == FwdQ8;
    static constexpr int KE = FP8 ? 128 : 64;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = TN * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int RECV = TN * 512;   // partial rows sent here: [rank][row of this CTA][128] fp32
    static constexpr int STAGES = TN <= 16 ? 5 : TN <= 32 ? 4 : TN <= 64 ? 3 : 5;
    static constexpr int SMEM = STAGES * STAGE + RECV + 1024;
    static constexpr uint32_t TM_COLS = TN < 32 ? 32 : TN;
};

// After every CTA of the cluster has arrived: sums this CTA's rows over the S ranks, in order, and finishes
// them, a warp a row, 4 columns a lane (b, ws: their bias and scales).  What a row's epilogue reads is asked
// for a row ahead, the first row's before the wait for the cluster.
template <Policy P, int TN, int S>
__device__ __forceinline__ void join_rows(const SplitParams &p, uint32_t recv, int rank, int mt, int n0, ulonglong2 b,
                                          ulonglong2 ws)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = n0 + lane * 4;
    struct Row {
        bool mine;
        size_t out;
        uint2 res;
        float xs;
    };
    const bool one_group = p.n_rblocks == p.rblocks;
    const int head = P == Dx ? col / p.dk : 0, in_head = P == Dx ? col - head * p.dk : 0;
    auto ask = [&](int l) {
        Row w{};
        const int at = mt * TN + l * S + rank;
        int grp = 0, i = at;
        bool there = true;
        if (!one_group) {
            const int block = at / p.rb;
            grp = block / p.rblocks;
            i = (block - grp * p.rblocks) * p.rb + at % p.rb;
            there = block < p.n_rblocks;
        }
        w.mine = there && l < TN / S && i < p.T && col < p.N;
        if (!w.mine) return w;
        const size_t row = (size_t)grp * p.T + i;
        w.out = P == Dx ? (((size_t)grp * p.H + head) * p.T + i) * p.dk + in_head : row * p.N + col;
        if (P != Dx && p.residual) w.res = *reinterpret_cast<const uint2 *>(p.residual + w.out);
        if (P == FwdQ8) w.xs = p.x_scale[row];
        return w;
    };
    Row next = ask(warp);
    __syncwarp();
    ptx::cluster_wait();
    for (int l = warp; l < TN / S; l += 8) {
        const Row w = next;
        next = ask(l + 8);
        if (!w.mine) continue;
        ulonglong2 f = lds_f32x4(recv + l * 512 + lane * 16);
#pragma unroll
        for (int k = 1; k < S; ++k) {
            const ulonglong2 t = lds_f32x4(recv + (k * (TN / S) + l) * 512 + lane * 16);
            f.x = ptx::add_f32x2(f.x, t.x);
            f.y = ptx::add_f32x2(f.y, t.y);
        }
        uint64_t v[2] = {f.x, f.y};
        if (P != Dx) {
            if (P == FwdQ8) {
                const uint64_t xs = f2_both(w.xs);
                v[0] = ptx::fma_f32x2(v[0], ptx::mul_f32x2(ws.x, xs), b.x);
                v[1] = ptx::fma_f32x2(v[1], ptx::mul_f32x2(ws.y, xs), b.y);
            } else if (p.bias) {
                v[0] = ptx::add_f32x2(v[0], b.x);
                v[1] = ptx::add_f32x2(v[1], b.y);
            }
            if (p.z) *reinterpret_cast<uint2 *>(p.z + w.out) = pack_bf16x4(v);
            activate(v, p.act);
            if (p.residual) {
                v[0] = ptx::add_f32x2(v[0], ptx::f2_pack(__uint_as_float(w.res.x << 16), __uint_as_float(w.res.x & 0xffff0000u)));
                v[1] = ptx::add_f32x2(v[1], ptx::f2_pack(__uint_as_float(w.res.y << 16), __uint_as_float(w.res.y & 0xffff0000u)));
            }
        }
        *reinterpret_cast<uint2 *>(p.y + w.out) = pack_bf16x4(v);
    }
}

// The two columns that a lane finishes where K is not split (p.N is even).
__device__ __forceinline__ int lane_col(int n0) { return n0 + (threadIdx.x & 126); }

// K is not split: each warp finishes a 32-column strip of the tile from tensor memory, W rows at a time, warps
// w + 4, which have had no other work, and w in turn.  Neighbouring lanes exchange values, so that a lane holds
// two columns of every second row.  b, ws: bias and scales of the columns.
template <Policy P, int TN>
__device__ __forceinline__ void finish_rows(const SplitParams &p, uint32_t tmem, int mt, int n0, uint64_t b, uint64_t ws,
                                            uint64_t *bar_acc, const Guard &g)
{
    constexpr int W = TN < 64 ? 16 : 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, odd = lane & 1;
    const int col = lane_col(n0);
    const bool cols = col < p.N;
    const int head = P == Dx ? col / p.dk : 0, in_head = P == Dx ? col - head * p.dk : 0;
    bool ready = false;
#pragma unroll 1
    for (int c = (warp >> 2 ^ 1) * W; c < TN; c += 2 * W) {   // (rb >= W: W rows lie in one block)
        const int at = mt * TN + c, block = at / p.rb, grp = block / p.rblocks;
        const int i0 = (block - grp * p.rblocks) * p.rb + at % p.rb + odd;
        const int rows = block < p.n_rblocks && cols ? min(W, p.T - i0) : 0;   // of this lane: 0, 2, 4.. below it
        const size_t step = P == Dx ? p.dk : p.N;
        const size_t out = P == Dx ? (((size_t)grp * p.H + head) * p.T + i0) * p.dk + in_head
                                   : ((size_t)grp * p.T + i0) * p.N + col;
        uint32_t res[W / 2] = {};
        float xs[W / 2] = {};
#pragma unroll
        for (int k = 0; k < W / 2; ++k)
            if (2 * k < rows) {
                if (P != Dx && p.residual) res[k] = *reinterpret_cast<const uint32_t *>(p.residual + out + 2 * k * step);
                if (P == FwdQ8) xs[k] = p.x_scale[(size_t)grp * p.T + i0 + 2 * k];
            }
        if (!ready) {
            wait_bounded(bar_acc, 0, g);
            ptx::tc_fence_after();
            ready = true;
        }
        uint32_t v[W];
        if constexpr (W == 16)
            ptx::tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
        else
            ptx::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
        ptx::tmem_ld_wait();
        reg_fence(v);
        uint64_t f[W / 2];
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            const uint32_t other = __shfl_xor_sync(~0u, odd ? v[2 * k] : v[2 * k + 1], 1);
            f[k] = odd ? ptx::f2_pack(__uint_as_float(other), __uint_as_float(v[2 * k + 1]))
                       : ptx::f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(other));
            if (P == FwdQ8) f[k] = ptx::fma_f32x2(f[k], ptx::mul_f32x2(ws, f2_both(xs[k])), b);
            if (P == Fwd) f[k] = ptx::add_f32x2(f[k], b);
        }
        auto put = [&](__nv_bfloat16 *to) {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                float lo, hi;
                ptx::f2_unpack(f[k], lo, hi);
                if (2 * k < rows) *reinterpret_cast<uint32_t *>(to + out + 2 * k * step) = ptx::pack_bf16x2(lo, hi);
            }
        };
        if (P == Fwd && p.z) put(p.z);
        if (P != Dx) {
            activate(f, p.act);
            if (p.residual) {
#pragma unroll
                for (int k = 0; k < W / 2; ++k)
                    f[k] = ptx::add_f32x2(f[k], ptx::f2_pack(__uint_as_float(res[k] << 16),
                                                             __uint_as_float(res[k] & 0xffff0000u)));
            }
        }
        put(p.y);
    }
}

template <Policy P, int TN>
__global__ void __launch_bounds__(256) gemm_split_kernel(const __grid_constant__ CUtensorMap map_w,
                                                         const __grid_constant__ CUtensorMap map_x,
                                                         const __grid_constant__ SplitParams p)
{
    using C = SplitCfg<P, TN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    __shared__ uint64_t bar_full[STAGES], bar_empty[STAGES], bar_acc;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_rank(), splits = (int)ptx::cluster_size();
    const int tile = blockIdx.x / splits, mt = tile / p.n_ntiles, n0 = tile % p.n_ntiles * 128;
    const int k_begin = rank * p.steps_per_cta, nk = max(0, min(p.steps_per_cta, p.ksteps - k_begin));
    const Guard g{&abort_sh, p.status, kWaitLimitNs};

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&bar_full[s], 1);
            ptx::mbar_init(&bar_empty[s], 1);
        }
        ptx::mbar_init(&bar_acc, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 2 && ptx::elect_one()) {
        ptx::tma_prefetch_desc(&map_w);
        ptx::tma_prefetch_desc(&map_x);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&tmem_sh, C::TM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh, recv = ptx::smem_u32(smem + STAGES * C::STAGE);
    if (splits > 1) ptx::cluster_arrive();
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    // asked for ahead of the roles: their latency is behind the first copies'
    ulonglong2 b = make_ulonglong2(0, 0), ws = b;   // of two or four columns (see finish_rows, join_rows)
    if (P != Dx) {
        const int c2 = lane_col(n0), c4 = n0 + lane * 4;
        if (splits == 1 && c2 < p.N) {
            if (p.bias) b.x = *reinterpret_cast<const uint64_t *>(p.bias + c2);
            if (P == FwdQ8) ws.x = *reinterpret_cast<const uint64_t *>(p.w_scale + c2);
        } else if (splits > 1 && c4 < p.N) {
            if (p.bias) b = *reinterpret_cast<const ulonglong2 *>(p.bias + c4);
            if (P == FwdQ8) ws = *reinterpret_cast<const ulonglong2 *>(p.w_scale + c4);
        }
    }

    if (warp == 0) {
        if (ptx::elect_one()) {
            // Everything that takes a division is worked out ahead of the loop (see the pair kernel).
            constexpr int BOXES = TN <= 32 ? 1 : TN / 32;
            const int boxes = TN / p.rb, heads = P == Dx ? 1 : p.H;
            int c = k_begin * C::KE, ch = P == Fwd ? c / p.dk : 0, ce = c - ch * p.dk, row[BOXES], slice[BOXES];
            if (P != Fwd) ce = c;
#pragma unroll
            for (int h = 0; h < BOXES; ++h) {
                const int block = mt * boxes + h, grp = block / p.rblocks;
                row[h] = (block - grp * p.rblocks) * p.rb;
                slice[h] = grp * heads;
            }
            int s = 0;
            uint32_t ph = 0;
            for (int q = 0; q < nk; ++q) {
                wait_bounded(&bar_empty[s], ph ^ 1, g);
                ptx::mbar_arrive_expect_tx(&bar_full[s], C::STAGE);
                uint8_t *sa = smem + s * C::STAGE, *sb = sa + C::A_BYTES;
                if (P == Fwd) {
                    ptx::tma_load_3d(sa, &map_w, &bar_full[s], n0, c, 0);
                    ptx::tma_load_3d(sa + 8192, &map_w, &bar_full[s], n0 + 64, c, 0);
                } else {
                    ptx::tma_load_3d(sa, &map_w, &bar_full[s], c, n0, 0);
                }
#pragma unroll
                for (int h = 0; h < BOXES; ++h)
                    if (h < boxes)
                        ptx::tma_load_3d(sb + h * p.rb * 128, &map_x, &bar_full[s], ce, row[h], slice[h] + ch);
                c += C::KE;
                ce += C::KE;
                if (P == Fwd && ce >= p.dk) {
                    ce = 0;
                    ++ch;
                }
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            for (int q = (nk > STAGES ? nk - STAGES : 0); q < nk; ++q)   // no copy outlives the CTA
                wait_bounded(&bar_full[q % STAGES], (q / STAGES) & 1, g);
        }
    } else if (warp == 1) {
        if (ptx::elect_one() && nk > 0) {
            const uint32_t idesc =
                C::FP8 ? ptx::idesc_f16_f32(128, TN, false, false) : ptx::idesc_bf16_f32(128, TN, P == Fwd, false);
            const uint32_t base = ptx::smem_u32(smem);
            for (int q = 0; q < nk; ++q) {
                const int s = q % STAGES;
                wait_bounded(&bar_full[s], (q / STAGES) & 1, g);
                ptx::tc_fence_after();
                const uint32_t sa = base + s * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t da = P == Fwd ? desc_mn(sa, kk) : desc_k(sa, kk);
                    if (C::FP8)
                        ptx::mma_ss_e4m3(tmem, da, desc_k(sb, kk), idesc, (q > 0 || kk > 0) ? 1u : 0u);
                    else
                        ptx::mma_ss(tmem, da, desc_k(sb, kk), idesc, (q > 0 || kk > 0) ? 1u : 0u);
                }
                ptx::mma_commit(&bar_empty[s]);
            }
            ptx::mma_commit(&bar_acc);
            wait_bounded(&bar_acc, 0, g);
        }
    } else if (warp >= 4 && splits > 1) {
        // the rows of the partial tile to their owners: row r to rank r mod splits as its row r / splits
        const int quarter = warp & 3, log2s = 31 - __clz(splits);
        const uint32_t mine = recv + ((uint32_t)(rank * (TN / splits)) * 128 + quarter * 32 + lane) * 4;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16);
        // rows that there are (with several groups a tile may have gaps: all are sent)
        const int valid = p.n_rblocks == p.rblocks ? min(TN, p.T - mt * TN) : TN;
        if (nk > 0) wait_bounded(&bar_acc, 0, g);
        ptx::tc_fence_after();
        __syncwarp();
        ptx::cluster_wait();   // every CTA of the cluster runs
        constexpr int W = TN < 32 ? 16 : 32;   // columns read at a time
#pragma unroll 1
        for (int c = 0; c < valid; c += W) {
            uint32_t v[W] = {};
            if (nk > 0) {
                if constexpr (W == 16)
                    ptx::tmem_ld16(taddr + c, v);
                else
                    ptx::tmem_ld32(taddr + c, v);
                ptx::tmem_ld_wait();
                reg_fence(v);
            }
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (c + e < valid)
                    ptx::st_cluster_b32(ptx::cluster_addr(mine + ((c + e) >> log2s) * 512, (c + e) & (splits - 1)), v[e]);
        }
        ptx::tc_fence_before();
    }
    __syncwarp();
    if (splits == 1) {
        finish_rows<P, TN>(p, tmem, mt, n0, b.x, ws.x, &bar_acc, g);
        ptx::tc_fence_before();
        __syncthreads();
    } else {
        if (warp < 4) ptx::cluster_wait();
        ptx::cluster_arrive();   // this CTA's rows are sent
        switch (splits) {        // (the wait for the others is in there)
        case 2: join_rows<P, TN, 2>(p, recv, rank, mt, n0, b, ws); break;
        case 4: join_rows<P, TN, 4>(p, recv, rank, mt, n0, b, ws); break;
        default: join_rows<P, TN, 8>(p, recv, rank, mt, n0, b, ws); break;
        }
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TM_COLS);
    }
}

// dz = dy act'(z) in bf16, and the column sums of the unrounded dz over a block of rows.  A warp
// takes a row's 256 columns at a time (8 a thread, 16 bytes), the block's 8 warps neighbouring rows.  Bound
// by HBM: 32768 x 4096 with GELU 124 us, 6.5 TB/s (0.96 of the measured copy).  The rounding is the price of bf16
// tensor cores in the two products, which take dz as an operand: dx and dw are then off by 2.3e-3 of their norm,
// with the last rounding alone 1.7e-3.  Operands of more bits (tf32, or dz as two bf16 terms) would take the
// products twice as long and dz's memory twice over; the column sums cost nothing unrounded, and are.
__global__ void __launch_bounds__(256) dz_kernel(const LinBwdArgs a, int blocks)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x * 256 + lane * 8;
    __shared__ float part[8][256];
    float s[8] = {};
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (n < a.N) {
        const long long per = ((long long)a.M + blocks - 1) / blocks;
        const long long m_end = min((long long)a.M, (blockIdx.y + 1) * per);
        // two rows at a time: their loads are in flight together
        for (long long m = blockIdx.y * per + warp; m < m_end; m += 16) {
            uint4 d4[2], z4[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (m + 8 * k < m_end) {
                    const size_t at = ((size_t)(m + 8 * k) * a.N + n) / 8;
                    d4[k] = static_cast<const uint4 *>(a.dy)[at];
                    if (a.z) z4[k] = static_cast<const uint4 *>(a.z)[at];
                }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (m + 8 * k < m_end) {
                    float f[8], z[8];
                    unpack_bf16x8(d4[k], f);
                    if (a.z) {
                        unpack_bf16x8(z4[k], z);
                        times_slope(f, z, a.act);
                        static_cast<uint4 *>(a.dz)[((size_t)(m + 8 * k) * a.N + n) / 8] =
                            make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                       ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7]));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] += f[e];
                }
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

// What is left after the products: dw = the sum of its partial sums, in order, rounded once, 4 elements a
// thread, in the first `dw_blocks` blocks; the bias gradient's partial sums in the others.
__global__ void __launch_bounds__(256) bwd_join_kernel(const float *part, void *dw, int splits, long long elems,
                                                       int dw_blocks, const float *col_part, float *dbias, int slices,
                                                       int N)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if ((int)blockIdx.x >= dw_blocks) {
        sum_columns(col_part, dbias, slices, N, ((int)blockIdx.x - dw_blocks) * kSumCols);
        return;
    }
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
cudaError_t launch_pair(const GemmMaps &m, const GemmParams &p, int clusters, cudaStream_t stream)
{
    using C = Cfg<P, BN>;
    static std::atomic<bool> set[64];
    const cudaError_t e = raise_smem((const void *)gemm_pair_kernel<P, BN>, C::SMEM, set);
    if (e != cudaSuccess) return e;
    return launch_overlapped(gemm_pair_kernel<P, BN>, 2 * clusters, 128 + 32 * kEpiWarps, C::SMEM, 2, stream, m, p);
}

template <Policy P, int TN>
cudaError_t launch_split_tn(const CUtensorMap &w, const CUtensorMap &x, const SplitParams &p, int tiles, int splits,
                            cudaStream_t stream)
{
    using C = SplitCfg<P, TN>;
    static std::atomic<bool> set[64];
    cudaError_t e = raise_smem((const void *)gemm_split_kernel<P, TN>, C::SMEM, set);
    if (e != cudaSuccess) return e;
    return launch_overlapped(gemm_split_kernel<P, TN>, tiles * splits, 256, C::SMEM, splits, stream, w, x, p);
}

// How few-row products are laid out: rows a tile, CTAs a tile.
struct SplitPlan {
    int tn, splits, tiles;
    double us;   // estimated time
};

// CTAs of the split kernel that the GPU holds at once: two an SM up to 64 rows, else one; clusters of
// four and eight leave some of a GPC's SMs over (from cudaOccupancyMaxActiveClusters on a GB300).
int split_slots(int tn, int s)
{
    if (tn <= 64) return s == 8 ? 288 : s == 4 ? 296 : 304;
    return s == 8 ? 120 : s == 4 ? 144 : 152;
}

// The plan with the least estimated time, in us.  The terms are fitted to a sweep of every plan over 1
// to 8192 rows at sixteen sizes of K and N from 64 to 8192 (the chosen plan takes 0.5 % more than the best
// one there on average, 11 % at most): start, join and end; a K step 0.26, or what the ring of stages leaves of
// the memory's latency once all SMs load, or the steps' bytes at L2's rate of 20 TB/s, or the weights at HBM's
// and L2's.
SplitPlan split_plan(int G, int T, int N, int ksteps)
{
    SplitPlan best{};
    best.us = 1e30;
    const long long M = (long long)G * T;
    for (int tn = 16; tn <= 128; tn *= 2) {
        const int rb = G > 1 && tn > 32 ? 32 : tn;
        const long long tiles = (long long)ceil_div((long long)ceil_div(T, rb) * G, tn / rb) * ceil_div(N, 128);
        if (tiles >= 0x7fffffff / 8) continue;
        for (int s = 1; s <= 8 && s <= ksteps; s *= 2) {
            const long long ctas = tiles * s;
            if (ctas > split_slots(tn, s)) break;   // all at once, or not at all
            const int steps = ceil_div(ksteps, s);
            const bool two = ctas > 2 * kPlanPairs;   // on some SMs
            const int stages = tn == 64 ? 3 : tn == 32 ? 4 : 5;
            const double ring = 1.106 / stages * (ctas < 2 * kPlanPairs ? ctas / (2.0 * kPlanPairs) : 1.0);
            const double l2 = (double)steps * ctas * (16384 + tn * 128) / 20.3e6;
            const double hbm = (double)ksteps * 128 * N / (two ? 10.2e6 : 9.2e6);
            double loop = steps * (ring > 0.258 ? ring : 0.258);
            loop = loop > l2 ? loop : l2;
            loop = loop > hbm ? loop : hbm;
            const double ends = s == 1 ? 3.4 + tn * 0.0272 + (two ? 0.195 : 0.0)
                                       : 3.72 + tn * (0.0281 + 0.0369 / (s * s)) + (two ? 0.56 : 0.0);
            const double us = ends + loop;
            if (us < best.us) best = SplitPlan{tn, s, (int)tiles, us};
        }
        if (tn >= M) break;
    }
    return best;
}

template <Policy P>
cudaError_t launch_split(const CUtensorMap &w, const CUtensorMap &x, SplitParams &p, const SplitPlan &s,
                         cudaStream_t stream)
{
    p.n_ntiles = ceil_div(p.N, 128);
    p.steps_per_cta = ceil_div(p.ksteps, s.splits);
    switch (s.tn) {
    case 16: return launch_split_tn<P, 16>(w, x, p, s.tiles, s.splits, stream);
    case 32: return launch_split_tn<P, 32>(w, x, p, s.tiles, s.splits, stream);
    case 64: return launch_split_tn<P, 64>(w, x, p, s.tiles, s.splits, stream);
    default: return launch_split_tn<P, 128>(w, x, p, s.tiles, s.splits, stream);
    }
}

// Row blocks: 128 rows of the only group, or 32 rows of one of several groups, so that a tile spans
// groups and wastes at most 31 rows a group (576 rows a group: 18 blocks, 256-row tiles would take
// 768 rows).
int row_block(int G) { return G > 1 ? 32 : 128; }

long long row_tiles(int G, int T)
{
    const long long blocks = (long long)ceil_div(T, row_block(G)) * G, per = BM / row_block(G);
    return (blocks + per - 1) / per;
}

// Fills in the rows and the tiles; false if there are too many to count in an int (see lin_rows_fit: the entry
// points refuse such rows).
bool set_tiles(Prob &q, int G, int T, int N, int bn, int splits)
{
    const int rb = row_block(G), rblocks = ceil_div(T, rb);
    const long long mtiles = row_tiles(G, T), tiles = mtiles * ceil_div(N, bn);
    // the kernel counts rows, those that pad a block included, and items in ints
    if (!lin_rows_fit(G, T) || tiles * splits > 0x7fffffffLL) return false;
    q.T = T;
    q.rb_log2 = rb == 32 ? 5 : 7;
    q.rblocks = fast_div(rblocks);
    q.n_rblocks = rblocks * G;
    q.n_mtiles = (int)mtiles;
    q.N = N;
    q.n_ntiles = ceil_div(N, bn);
    q.tiles = fast_div((int)tiles);
    q.per_group = fast_div(kGroupM * q.n_ntiles);
    q.n_items = (int)(tiles * splits);
    return true;
}

void set_split_rows(SplitParams &p, int G, int T, int tn)
{
    p.T = T;
    p.rb = G > 1 && tn > 32 ? 32 : tn;
    p.rblocks = ceil_div(T, p.rb);
    p.n_rblocks = p.rblocks * G;
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;

// Tiles of 256 or 128 columns, whichever is estimated to take less: rounds of tiles per pair x (K
// steps x time of a step + a tile's fill and drain).
struct PairPlan {
    bool wide;
    double us;
};

constexpr double kStepWide = 0.298, kStepNarrow = 0.219;   // us a K step (the sweep of split_plan)

PairPlan pair_plan(long long mtiles, int N, int ksteps)
{
    auto rounds = [&](int bn) { return (double)((mtiles * ceil_div(N, bn) + kPlanPairs - 1) / kPlanPairs); };
    const double w = 5.58 + rounds(256) * ksteps * kStepWide, n = 4.975 + rounds(128) * ksteps * kStepNarrow;
    return w <= n ? PairPlan{true, w} : PairPlan{false, n};
}

// The backward runs both products in one launch, so that one's tiles fill the pairs that the other's
// leave idle and there is one start and end (18432 rows, 768 x 768: 42 us apart, 33 together; 1111 rows,
// 1000 x 520: 20 and 12; 32768 rows, 1024 x 4096: 307 and 295, 1.86 PFLOP/s).
//
// How `clusters` share nd items of dw, of a steps each, and nx of dx, of b.
struct Shares {
    long long nd, nx, a, b, whole, rest, clusters;   // rest clusters have whole + 1 items of dw
    Shares(long long nd, long long nx, long long a, long long b, int clusters)
        : nd(nd), nx(nx), a(a), b(b), whole(nd / clusters), rest(nd % clusters), clusters(clusters)
    {
    }
    // dx's items that fit up to step t beside `dw` items of dw
    long long room(long long t, long long dw) const { return t > dw * a ? (t - dw * a) / b : 0; }
    long long even() const { return (nd * a + nx * b + clusters - 1) / clusters; }
    long long longest_dw() const { return (whole + (rest > 0)) * a; }
    // The least level t >= lo at which dx's items fit: all clusters end at about that step.  (They do at
    // even() + b, where no cluster wastes an item's room.)
    long long level(long long lo) const
    {
        long long hi = even() + b;
        while (lo < hi) {
            const long long t = (lo + hi) / 2;
            if (rest * room(t, whole + 1) + (clusters - rest) * room(t, whole) >= nx)
                hi = t;
            else
                lo = t + 1;
        }
        return lo;
    }
};

// dw has few tiles (K x N) and a long sum (the rows), which is split over items where that pays for the
// partial sums' join.  The estimate is fitted to a sweep of every plan over 64 to 18432 rows at twelve sizes
// of K and N from 256 to 4096 (the chosen plan takes 1 % more than the best one there on average); an item's
// fill and drain counts as one more step of dx, two of dw.
struct BwdPlan {
    bool wide;
    int splits, steps_per_split;
    double us, dw_us;   // of both, of dw alone
};

BwdPlan bwd_plan(int G, int T, int K, int N)
{
    constexpr double kStart = 3.8, kStep[2] = {0.222, 0.335}, kJoin = 2.2, kJoinRate = 9.4e6;
    const long long steps = (long long)G * ceil_div(T, 64), mx = row_tiles(G, T), mw = ceil_div(K, BM);
    const int ksteps = ceil_div(N, 64);
    BwdPlan best{};
    best.us = 1e30;
    for (int wide = 1; wide >= 0; --wide) {
        const int bn = wide ? 256 : 128;
        for (int s = 1; s <= 16 && s <= steps; ++s) {
            const long long per = (steps + s - 1) / s;
            if ((steps + per - 1) / per != s) continue;
            const double fixed = kStart + (s > 1 ? kJoin + (double)s * K * N * 8 / kJoinRate : 0.0);
            if (fixed >= best.us) break;
            const Shares h(mw * ceil_div(N, bn) * s, mx * ceil_div(K, bn), per + 2, ksteps + 1, kPlanPairs);
            const long long even = h.even(), dw = h.longest_dw();
            if (fixed + (even > dw ? even : dw) * kStep[wide] >= best.us) continue;
            const long long level = h.level(even), last = level > dw ? level : dw;
            const double us = fixed + last * kStep[wide];
            if (us < best.us) best = BwdPlan{wide == 1, s, (int)per, us, fixed + dw * kStep[wide]};
        }
    }
    return best;
}

// How many of dx's items each cluster takes.  (Beside other items a fill and drain counts twice that; the
// sweep was run with these.)
void level_items(GemmParams &p, int clusters)
{
    const Shares h(p.q[1].n_items, p.q[0].n_items, p.q[1].steps_per_split + 4, p.q[0].ksteps + 2, clusters);
    const long long t = h.level(0);
    p.a_clusters = (int)h.rest;
    p.x_all = (int)h.room(t, h.rest ? h.whole + 1 : h.whole);
    p.x_early = (int)h.room(t, h.whole) - p.x_all;
}

// Which of the two kernels takes a forward product.
struct FwdPlan {
    bool few;          // the few-row kernel, by `split`; else the pair kernel
    SplitPlan split;
    bool wide;
};

FwdPlan fwd_plan(int G, int T, int K, int N, bool q8)
{
    const int ksteps = ceil_div(K, q8 ? 128 : 64);
    const PairPlan pair = pair_plan(row_tiles(G, T), N, ksteps);
    const SplitPlan split = split_plan(G, T, N, ksteps);
    return FwdPlan{split.us < pair.us, split, pair.wide};
}

// How a backward runs: the plan of the products in one launch, whether dx goes to the few-row kernel beside dw
// alone, and how the bias gradient is taken where dz is dy: where dw is taken too, the two idle warps of the
// product kernel's CTAs read dy for it.  Each adds up whole columns where that (0.8 us for 64 rows) ends with the
// products or within a join's time (196 x 768 x 768: 6.2 us, with the join 7.7; 16 x 1024 x 4096 10.3 and 17.8;
// 1024 x 768 x 768 11.8 and 8.7).  Else slices of rows, which costs nothing while the products take longer, from
// K of about 450 on (16 KB in flight a CTA against 4 K flops an element); else a pass of its own.
enum BiasBy { kPass, kColumns, kSlices };
struct BwdChoice {
    BwdPlan plan;
    SplitPlan split;
    bool dx_split;
    BiasBy bias;
};

BwdChoice bwd_choice(int G, int T, int K, int N, bool has_act, bool need_dx, bool need_dw)
{
    BwdChoice c{bwd_plan(G, T, K, N), SplitPlan{}, false, kPass};
    if (need_dx) c.split = split_plan(G, T, K, ceil_div(N, 64));
    c.dx_split = need_dx && c.split.us + c.plan.dw_us < c.plan.us;
    if (has_act || !need_dw) return c;
    const int col_warps = 4 * (N < 256 * kPlanPairs ? ceil_div(N, 256) : kPlanPairs);   // at least
    const double direct_us = 0.8 * ceil_div((long long)G * T, 64) * ceil_div(ceil_div(N, 64), col_warps);
    if (direct_us <= (need_dx && !c.dx_split ? c.plan.us : c.plan.dw_us) + 0.5)
        c.bias = kColumns;
    else if (K >= 512)
        c.bias = kSlices;
    return c;
}

}  // namespace

void lin_plan(int G, int T, int K, int N, int q8, int plan[5])
{
    const FwdPlan f = fwd_plan(G, T, K, N, q8 != 0);
    plan[0] = f.few ? f.split.tn : 0;
    plan[1] = f.few ? f.split.splits : 0;
    plan[2] = f.few ? 0 : f.wide ? 256 : 128;
    plan[3] = plan[4] = 0;
}

void lin_bwd_plan(int G, int T, int K, int N, int has_act, int plan[5])
{
    const BwdChoice c = bwd_choice(G, T, K, N, has_act != 0, true, true);
    plan[0] = c.dx_split ? c.split.tn : 0;
    plan[1] = c.dx_split ? c.split.splits : 0;
    plan[2] = c.plan.wide ? 256 : 128;
    plan[3] = c.plan.splits;
    plan[4] = c.bias;
}

bool lin_rows_fit(int G, int T) { return row_tiles(G, T) * BM <= 0x7fffffffLL; }

cudaError_t launch_linear(const LinArgs &a, cudaStream_t stream)
{
    const int ksteps = ceil_div(a.K, a.q8 ? 128 : 64);
    const FwdPlan plan = fwd_plan(a.G, a.T, a.K, a.N, a.q8 != 0);
    const SplitPlan &split = plan.split;
    GemmMaps m = {};
    CUresult r;
    if (plan.few) {
        SplitParams sp = {};
        set_split_rows(sp, a.G, a.T, split.tn);
        sp.N = a.N;
        sp.dk = a.dk;
        sp.H = a.H;
        sp.ksteps = ksteps;
        sp.bias = a.bias;
        sp.x_scale = a.x_scale;
        sp.w_scale = a.w_scale;
        sp.residual = static_cast<const __nv_bfloat16 *>(a.residual);
        sp.y = static_cast<__nv_bfloat16 *>(a.y);
        sp.z = static_cast<__nv_bfloat16 *>(a.z);
        sp.act = a.act;
        sp.status = a.status;
        if (a.q8) {
            r = make_map_3d(&m.a, a.x, kU8, 1, a.K, a.M, 1, 128, sp.rb);
            if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kU8, 1, a.K, a.N, 1, 128, 128);
        } else {
            r = make_map_3d(&m.a, a.x, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, sp.rb);
            if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kBf16, 2, a.N, a.K, 1, 64, 64);
        }
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
        return a.q8 ? launch_split<FwdQ8>(m.b, m.a, sp, split, stream) : launch_split<Fwd>(m.b, m.a, sp, split, stream);
    }
    const int bn = plan.wide ? 256 : 128;
    GemmParams p = {};
    Prob &q = p.q[0];
    if (!set_tiles(q, a.G, a.T, a.N, bn, 1)) return cudaErrorInvalidValue;
    q.dk = a.dk;
    q.H = a.H;
    q.ksteps = q.steps_per_split = ksteps;
    p.bias = a.bias;
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.has_z = a.z != nullptr;
    p.has_r = a.residual != nullptr;
    p.act = a.act;
    p.status = a.status;
    if (a.q8) {
        r = make_map_3d(&m.a, a.x, kU8, 1, a.K, a.M, 1, 128, 128);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kU8, 1, a.K, a.N, 1, 128, bn / 2);
    } else {
        r = make_map_3d(&m.a, a.x, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 1 << q.rb_log2);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kBf16, 2, a.N, a.K, 1, 64, 64);
    }
    const int oc = a.z ? 32 : 64;   // columns of a store (see the epilogue)
    if (r == CUDA_SUCCESS) r = make_map_3d(&m.y, a.y, kBf16, 2, a.N, a.T, a.G, oc, 32);
    if (r == CUDA_SUCCESS && a.z) r = make_map_3d(&m.y2, a.z, kBf16, 2, a.N, a.T, a.G, oc, 32);
    if (r == CUDA_SUCCESS && a.residual) r = make_map_3d(&m.a2, a.residual, kBf16, 2, a.N, a.T, a.G, oc, 32);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    const int pairs = device_sm_count() / 2, clusters = q.n_items < pairs ? q.n_items : pairs;
    if (a.q8)
        return plan.wide ? launch_pair<FwdQ8, 256>(m, p, clusters, stream) : launch_pair<FwdQ8, 128>(m, p, clusters, stream);
    return plan.wide ? launch_pair<Fwd, 256>(m, p, clusters, stream) : launch_pair<Fwd, 128>(m, p, clusters, stream);
}

// Blocks of rows of the column sums: four blocks of threads an SM, at least 16 rows each, and no more
// than two warps of each CTA can add up behind the products.
static int lin_bwd_row_blocks(int M, int N)
{
    const int strips = ceil_div(N, 256);
    int b = ceil_div(8 * kPlanPairs, strips);
    if (b > 256) b = 256;
    if (b > ceil_div(M, 16)) b = ceil_div(M, 16);
    return b > 1 ? b : 1;
}

// Slices of rows of the same sums where dz is dy: one for each of the warps that take them beside the
// products, at least 16 rows each.
int lin_bwd_slices(int M)
{
    const int most = ceil_div(M, 16);
    return most < 4 * kPlanPairs ? (most > 1 ? most : 1) : 4 * kPlanPairs;
}

int lin_bwd_col_rows(int M, int N)
{
    const int b = lin_bwd_row_blocks(M, N), s = lin_bwd_slices(M);
    return b > s ? b : s;
}

int lin_dw_splits(int G, int T, int K, int N) { return T > 0 ? bwd_plan(G, T, K, N).splits : 1; }

cudaError_t launch_linear_bwd(const LinBwdArgs &a, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    const int blocks = lin_bwd_row_blocks(a.M, a.N);
    const BwdChoice choice = bwd_choice(a.G, a.T, a.K, a.N, a.z != nullptr, a.dx != nullptr, a.dw != nullptr);
    const BwdPlan &plan = choice.plan;
    const int ksteps = ceil_div(a.N, 64);
    const SplitPlan &split = choice.split;
    const bool dx_split = choice.dx_split, direct = a.dbias && choice.bias == kColumns,
               beside = a.dbias && choice.bias != kPass;
    if ((a.dbias && !beside) || (a.z && (a.dx || a.dw))) {
        e = launch_overlapped(dz_kernel, dim3(ceil_div(a.N, 256), blocks), 256, 0, 1, stream, a, blocks);
        if (e != cudaSuccess) return e;
    }
    const void *dz = a.z ? a.dz : a.dy;
    CUresult r = CUDA_SUCCESS;
    const bool dx_left = a.dx && !dx_split;
    if (dx_split) {
        SplitParams sp = {};
        set_split_rows(sp, a.G, a.T, split.tn);
        sp.N = a.K;
        sp.dk = a.dk;
        sp.H = a.H;
        sp.ksteps = ksteps;
        sp.y = static_cast<__nv_bfloat16 *>(a.dx);
        sp.status = a.status;
        CUtensorMap mx, mw;
        r = make_map_3d(&mx, dz, kBf16, 2, a.N, a.T, a.G, 64, sp.rb);
        if (r == CUDA_SUCCESS) r = make_map_3d(&mw, a.w, kBf16, 2, a.N, a.K, 1, 64, 128);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
        if ((e = launch_split<Dx>(mw, mx, sp, split, stream)) != cudaSuccess) return e;
    }
    if (!dx_left && !a.dw) return a.dbias ? launch_sum_rows(a.col_part, a.dbias, blocks, a.N, stream) : e;

    const int bn = plan.wide ? 256 : 128;
    GemmMaps m = {};
    GemmParams p = {};
    p.status = a.status;
    if (dx_left) {
        Prob &q = p.q[0];
        if (!set_tiles(q, a.G, a.T, a.K, bn, 1)) return cudaErrorInvalidValue;
        q.dk = a.dk;
        q.H = a.H;
        q.ksteps = q.steps_per_split = ksteps;
        r = make_map_3d(&m.a, dz, kBf16, 2, a.N, a.T, a.G, 64, 1 << q.rb_log2);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b, a.w, kBf16, 2, a.N, a.K, 1, 64, bn / 2);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.y, a.dx, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 32);
    }
    if (a.dw && r == CUDA_SUCCESS) {
        Prob &q = p.q[1];
        if (!set_tiles(q, 1, a.K, a.N, bn, plan.splits)) return cudaErrorInvalidValue;
        q.dk = a.dk;
        q.H = a.H;
        q.tblocks = ceil_div(a.T, 64);
        q.T_k = a.T;
        q.ksteps = a.G * q.tblocks;
        q.steps_per_split = plan.steps_per_split;
        p.part = plan.splits > 1;
        r = make_map_3d(&m.a2, a.x, kBf16, 2, a.dk, a.T, (long long)a.G * a.H, 64, 64);
        if (r == CUDA_SUCCESS) r = make_map_3d(&m.b2, dz, kBf16, 2, a.N, a.T, a.G, 64, 64);
        if (r == CUDA_SUCCESS)
            r = p.part ? make_map_3d(&m.y2, a.dw_part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.N, a.K, plan.splits, 32, 32)
                       : make_map_3d(&m.y2, a.dw, kBf16, 2, a.N, a.K, 1, 64, 32);
    }
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    if (a.dbias) {
        p.col_part = a.col_part;
        p.dbias = a.dbias;
        p.col_rows = blocks;
        p.col_n = a.N;
        if (beside) {
            p.sum_x = static_cast<const __nv_bfloat16 *>(a.dy);
            p.sum_m = a.M;
            p.slices = direct ? 0 : lin_bwd_slices(a.M);
            p.per_slice = direct ? 0 : ceil_div(a.M, p.slices);
        }
    }
    const long long items = (long long)p.q[0].n_items + p.q[1].n_items;
    const int pairs = device_sm_count() / 2, clusters = items < pairs ? (int)items : pairs;
    level_items(p, clusters);
    e = plan.wide ? launch_pair<Bwd, 256>(m, p, clusters, stream) : launch_pair<Bwd, 128>(m, p, clusters, stream);
    if (e == cudaSuccess && (p.part || p.slices)) {
        const long long elems = p.part ? (long long)a.K * a.N : 0;
        const int dw_blocks = ceil_div(elems, 1024), sum_blocks = p.slices ? a.N / kSumCols : 0;   // N % 8 == 0
        e = launch_overlapped(bwd_join_kernel, dw_blocks + sum_blocks, 256, 0, 1, stream, (const float *)a.dw_part, a.dw,
                              plan.splits, elems, dw_blocks, (const float *)a.col_part, a.dbias, p.slices, a.N);
    }
    return e;
}

}  // namespace attn
