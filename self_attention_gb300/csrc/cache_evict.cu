// Eviction from a cache by accumulated attention weight.
//
// Per sequence and head, n = min(length, keep) slots stay: those of the `recent` newest positions first, then
// the ones of the largest weights, equal ones by the lower slot.  Kept slots at or behind n move into evicted
// ones before n, both in ascending order, so that sources and targets never meet, every move can run at once
// and a slot that stays in place costs nothing but its rank.
//
// select_kernel: a cluster of 1 to 8 blocks a sequence and head, each with a run of its slots; more where the blocks
// fill the GPU no better (one pass over a slot is some 30 instructions a warp, and there are six: 16384 slots of 32
// heads, most of them evicted, take 27 us by clusters of four and took 35 by single blocks).  A slot's rank is its
// weight's bits (weights count as zero where they are negative or NaN), all ones for the newest positions.  The n-th
// largest rank is found by up to three histograms of 11, 11 and 10 bits over ranks that stay in shared memory (from L2
// where they do not fit), each added up over the cluster; two are enough where no rank that goes begins with the bits of
// one that stays (a third takes 32 heads of 16384 slots 2 us).
// Then each warp takes a run of neighbouring slots and numbers its ties, its holes and its movers by ballots, with
// sums over the warps and the cluster in between: in order without a barrier a step.  move_kernel: the rows, 16 bytes
// a lane, over the whole GPU.
// Bound by HBM (8 bytes a slot, 8 d a moved slot) once there are enough sequences and heads, by the select's
// latency before.
#include "cluster.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kBins = 2048;
constexpr int kMaxInSmem = 48 * 1024;    // ranks a block keeps in shared memory (192 KB)
constexpr int kPlanSms = 152;
constexpr int kOwnBlocks = 128;          // blocks from which on they move what they select,
constexpr int kOwnElements = 128 * 1024; // up to these elements of k a block, and
constexpr int kOwnMoves = 256;           // moves a block up to which fewer do
constexpr int kSmallSlots = 8192;        // up to which two blocks of 512 threads share an SM
constexpr int kListMoves = 3 * kBins / 2; // moves a block's own list has room for, and one more
constexpr int kMoveRows = 32;            // moves a block of move_kernel takes

struct SelShared {
    alignas(16) uint32_t bins[3][kBins]; // of each pass, then a short list of moves
    uint32_t warp[4][32];
    uint32_t prefix;                     // rank bits found so far
    uint32_t need;                       // how many are still to be taken among those with this prefix
    uint32_t have;                       // and how many there are
    uint32_t sums[4];                    // this block's, read by the others: newest, ties, holes, movers
};

// Sum over the lanes before this one and this one.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, uint32_t lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= (uint32_t)o) v += t;
    }
    return v;
}

// Sum of `v` over the warps before this one, `total` over all of them; v is the same in all lanes of a warp.
template <int WARPS>
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t *buf, uint32_t &total)
{
    const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) buf[w] = v;
    __syncthreads();
    const uint32_t part = lane < WARPS ? buf[lane] : 0u, sums = warp_scan(part, lane);
    total = __shfl_sync(0xffffffffu, sums, 31);
    return __shfl_sync(0xffffffffu, sums - part, w);
}

__device__ __forceinline__ uint32_t rank_of(float w, int pos, long long oldest)
{
    if (pos > oldest) return 0xffffffffu;
    return w > 0.f ? __float_as_uint(w) : 0u;
}

// Moves first, first + step ... of a list: each by LANES lanes (16 bytes each) of d = 8 LANES columns, N at once.
template <int LANES, int N>
__device__ __forceinline__ void move_rows(const EvictArgs &a, int bh, const int *moves, int count, int first, int step)
{
    const int lane = threadIdx.x % LANES;
    const long long row = (long long)bh * a.C;
    uint4 *k = static_cast<uint4 *>(a.k) + row * LANES, *v = static_cast<uint4 *>(a.v) + row * LANES;
    int2 at[N];                                     // (to, from)
    uint4 x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int m = first + i * step;
        at[i] = m < count ? *reinterpret_cast<const int2 *>(moves + 2 + 2 * m) : make_int2(-1, -1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (at[i].x >= 0) {
            x[i] = k[(long long)at[i].y * LANES + lane];
            y[i] = v[(long long)at[i].y * LANES + lane];
        }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (at[i].x < 0) continue;
        const long long dst = at[i].x, src = at[i].y;
        k[dst * LANES + lane] = x[i];
        v[dst * LANES + lane] = y[i];
        if (lane == 0) {
            a.weights_out[row + dst] = a.weights[row + src];
            a.weights_out[row + src] = 0.f;
        }
        if (lane == 1) {
            a.positions_out[row + dst] = a.slot_positions[row + src];
            a.positions_out[row + src] = -1;
        }
    }
}

// LANES > 0: the blocks move the rows themselves, 0: move_kernel does.
template <int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(EvictArgs a, int stride, int in_smem, int blocks)
{
    extern __shared__ __align__(16) uint32_t ranks[];
    __shared__ SelShared s;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bh = blockIdx.x / blocks, b = bh / a.H;
    const int me = blockIdx.x % blocks;          // (= the rank in the cluster)
    const long long row = (long long)bh * a.C;
    const float *w = a.weights + row;
    const int *pos = a.slot_positions + row;
    // up to 4096 slots wait in registers for the newest position, more are read again; those of a single block are asked
    // for along with the length
    constexpr int WARPS = THREADS / 32, HELD = 4096 / THREADS;
    float wr[HELD];
    int pr[HELD];
    auto hold = [&](int from, int to) {
#pragma unroll
        for (int e = 0; e < HELD; ++e) {
            const int j = from + e * THREADS + tid;
            wr[e] = j < to ? w[j] : 0.f;
            pr[e] = j < to ? pos[j] : INT32_MIN;
        }
    };
    const bool early = blocks == 1 && in_smem && a.C <= HELD * THREADS;
    if (early) hold(0, a.C);
    const int L = min(max(a.lengths[b], 0), a.C), n = min(L, a.keep);
    float *w_out = a.weights_out + row;
    int *pos_out = a.positions_out + row;
    int *moves = a.moves + (long long)bh * stride;
    if (bh % a.H == 0 && me == 0 && tid == 0) a.lengths_out[b] = n;
    // what lies behind the kept slots is empty; sources of moves are emptied by those who read them
    if (n == L) {
#pragma unroll 4
        for (int j = me * THREADS + tid; j < a.C; j += blocks * THREADS) {
            const float x = j < n ? w[j] : 0.f;
            const int p = j < n ? pos[j] : -1;
            w_out[j] = x;
            pos_out[j] = p;
        }
        if (LANES == 0 && me == 0 && tid == 0) moves[0] = 0;
        return;
    }
    const int share = ((L + blocks - 1) / blocks + 31) / 32 * 32;       // slots [begin, end) are this block's
    const int begin = min(me * share, L), end = min(begin + share, L);
    auto sync = [&] {
        __syncwarp();                // (a warp arrives as one)
        if (blocks > 1) ptx::cluster_sync();
        else __syncthreads();
    };
    auto other = [&](const void *p, int block) { return ptx::cluster_addr(ptx::smem_u32(p), (uint32_t)block); };
    // the sum of the others' s.sums[i] ahead of this block's, and over all; lane k reads block k's
    auto blocks_before = [&](int i, uint32_t &total) {
        const uint32_t x = lane < blocks ? ptx::ld_cluster_b32(other(&s.sums[i], lane)) : 0u;
        total = __reduce_add_sync(0xffffffffu, x);
        return __reduce_add_sync(0xffffffffu, lane < me ? x : 0u);
    };

    // the newest position
    for (int i = tid; i < 3 * kBins; i += THREADS) (&s.bins[0][0])[i] = 0;
    int newest = INT32_MIN;
    const bool held = in_smem && share <= HELD * THREADS;
    if (held) {
        if (!early) hold(begin, end);
#pragma unroll
        for (int e = 0; e < HELD; ++e)
            if (begin + e * THREADS + tid < end) newest = max(newest, pr[e]);
    } else {
#pragma unroll 8
        for (int j = begin + tid; j < end; j += THREADS) newest = max(newest, pos[j]);
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) s.warp[0][warp] = (uint32_t)newest;
    __syncthreads();
    newest = __reduce_max_sync(0xffffffffu, lane < WARPS ? (int)s.warp[0][lane] : INT32_MIN);
    if (blocks > 1) {
        if (tid == 0) s.sums[0] = (uint32_t)newest;
        sync();
        newest = __reduce_max_sync(0xffffffffu, lane < blocks ? (int)ptx::ld_cluster_b32(other(&s.sums[0], lane)) : newest);
    }
    const long long oldest = (long long)newest - a.recent;   // positions above it are safe
    auto rank = [&](int j) { return in_smem ? ranks[j - begin] : rank_of(w[j], pos[j], oldest); };

    // the n-th largest rank
    constexpr uint32_t kAll = 0xffffffffu;
    uint32_t prefix = 0, need = (uint32_t)n;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
        uint32_t *bins = s.bins[pass];
        auto count = [&](uint32_t r, bool there) {
            const uint32_t bin = there && (r & mask) == prefix ? r >> shift & ((1u << bits) - 1) : 0xffffffffu;
            // ties (zeros, the newest) often fill a warp: one addition for all of them
            const uint32_t b0 = __shfl_sync(0xffffffffu, bin, 0);
            if (__all_sync(0xffffffffu, bin == b0)) {
                if (lane == 0 && bin != 0xffffffffu) atomicAdd(&bins[bin], 32u);
            } else if (bin != 0xffffffffu) {
                atomicAdd(&bins[bin], 1u);
            }
        };
        if (pass == 0 && held) {
#pragma unroll
            for (int e = 0; e < HELD; ++e) {
                const int j = begin + e * THREADS + tid;
                const uint32_t r = rank_of(wr[e], pr[e], oldest);
                if (j < end) ranks[j - begin] = r;
                if (begin + e * THREADS < end) count(r, j < end);
            }
        } else if (pass == 0) {
#pragma unroll 4
            for (int j0 = begin; j0 < end; j0 += THREADS) {
                const int j = j0 + tid;
                const uint32_t r = j < end ? rank_of(w[j], pos[j], oldest) : 0u;
                if (in_smem && j < end) ranks[j - begin] = r;
                count(r, j < end);
            }
        } else {
            for (int j0 = begin; j0 < end; j0 += THREADS) {
                const int j = j0 + tid;
                count(j < end ? rank(j) : 0u, j < end);
            }
        }
        sync();
        // bins from the top: thread t holds PER of them
        constexpr int PER = kBins / THREADS;
        const int base = PER * (THREADS - 1 - tid);
        uint32_t c[PER], sum = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) c[e] = bins[base + e];
        if (PER == 2 && blocks > 1) {
            uint2 x[7];
#pragma unroll
            for (int k = 1; k < 8; ++k)
                x[k - 1] = k < blocks ? ptx::ld_cluster_b64(other(&bins[base], me ^ k)) : make_uint2(0, 0);
#pragma unroll
            for (int k = 0; k < 7; ++k) {
                c[0] += x[k].x;
                c[1] += x[k].y;
            }
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) sum += c[e];
        const uint32_t inc = warp_scan(sum, lane);
        uint32_t total;
        uint32_t above = warps_before<WARPS>(__shfl_sync(0xffffffffu, inc, 31), s.warp[1], total) + inc - sum;
#pragma unroll
        for (int e = PER - 1; e >= 0; --e) {
            if (above < need && need <= above + c[e]) {
                s.prefix = prefix | (uint32_t)(base + e) << shift;
                s.need = need - above;
                s.have = c[e];
            }
            above += c[e];
        }
        __syncthreads();
        prefix = s.prefix;
        need = s.have == s.need ? kAll : s.need;
        if (need == kAll) break;         // all that begin with these bits stay: two passes where weights differ
    }

    // In order: ranks above `prefix` stay, and the first `need` that equal it.  A warp takes slots [from, to).
    const int run = (end - begin + THREADS - 1) / THREADS * 32, from = min(begin + warp * run, end), to = min(from + run, end);
    uint32_t ties0 = 0, holes = 0, movers = 0, total;
    if (need != kAll) {              // the order of the ties matters: some of them go
        uint32_t ties = 0;
        for (int j0 = from; j0 < to; j0 += 32) {
            const int j = j0 + lane;
            ties += __popc(__ballot_sync(0xffffffffu, j < to && rank(j) == prefix));
        }
        ties0 = warps_before<WARPS>(ties, s.warp[0], total);
        if (blocks > 1) {
            if (tid == 0) s.sums[1] = total;
            sync();
            ties0 += blocks_before(1, total);
        }
    }
    const uint32_t below = (1u << lane) - 1;
    auto kept = [&](int j, uint32_t &t) {          // by a whole warp; t: ties so far
        const uint32_t r = j < to ? rank(j) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, j < to && r == prefix);
        const bool k = j < to && (r > prefix || (r == prefix && t + __popc(eq & below) < need));
        t += __popc(eq);
        return k;
    };
    uint32_t t = ties0;
    for (int j0 = from; j0 < to; j0 += 32) {
        const int j = j0 + lane;
        const bool k = kept(j, t);
        holes += __popc(__ballot_sync(0xffffffffu, j < n && j < to && !k));
        movers += __popc(__ballot_sync(0xffffffffu, j >= n && k));
    }
    uint32_t hole = warps_before<WARPS>(holes, s.warp[2], total), mover = warps_before<WARPS>(movers, s.warp[3], movers);
    if (blocks > 1) {
        if (tid == 0) {
            s.sums[2] = total;
            s.sums[3] = movers;
        }
        sync();
        mover += blocks_before(3, movers);
        hole += blocks_before(2, total);
    }
    if (LANES == 0 && me == 0 && tid == 0) moves[0] = (int)total;
    int *list = LANES > 0 && blocks == 1 && total < kListMoves ? reinterpret_cast<int *>(&s.bins[0][0]) : moves;
    t = ties0;
#pragma unroll 2
    for (int j0 = from; j0 < to; j0 += 32) {
        const int j = j0 + lane;
        const bool k = kept(j, t);
        const uint32_t hb = __ballot_sync(0xffffffffu, j < n && j < to && !k);
        const uint32_t mb = __ballot_sync(0xffffffffu, j >= n && k);
        if (hb >> lane & 1) list[2 + 2 * (hole + __popc(hb & below))] = j;
        if (mb >> lane & 1) list[3 + 2 * (mover + __popc(mb & below))] = j;
        hole += __popc(hb);
        mover += __popc(mb);
        if (j < n ? k : j < to && !k) {
            const float x = j < n ? w[j] : 0.f;
            const int p = j < n ? pos[j] : -1;
            w_out[j] = x;
            pos_out[j] = p;
        }
    }
    for (int j = L + me * THREADS + tid; j < a.C; j += blocks * THREADS) {
        w_out[j] = 0.f;
        pos_out[j] = -1;
    }
    if (LANES > 0) {
        // the list is complete, and nothing of the sources' numbers is needed any more but by those who move them
        sync();
        constexpr int AT_ONCE = THREADS / (LANES > 0 ? LANES : 1), N = 2;
        for (int m = me * AT_ONCE + tid / (LANES > 0 ? LANES : 1); m < (int)total; m += N * blocks * AT_ONCE)
            move_rows<(LANES > 0 ? LANES : 1), N>(a, bh, list, (int)total, m, blocks * AT_ONCE);
    } else {
        __syncwarp();
        if (blocks > 1) ptx::cluster_sync_relaxed();     // nobody leaves while its sums are read
    }
}

template <int LANES>
__global__ void __launch_bounds__(256) move_kernel(EvictArgs a, int stride, int blocks)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int bh = blockIdx.x / blocks;
    const int *moves = a.moves + (long long)bh * stride;
    constexpr int STEP = 256 / LANES;
    move_rows<LANES, kMoveRows / STEP>(a, bh, moves, moves[0], blockIdx.x % blocks * kMoveRows + threadIdx.x / LANES, STEP);
}

int most_moves(int C, int keep) { return keep < C - keep ? keep : C - keep > 0 ? C - keep : 0; }
int moves_stride(int C, int keep) { return (2 + 2 * most_moves(C, keep) + 3) / 4 * 4; }

// Blocks of select_kernel a sequence and head: as many as keep the GPU's SMs from idling, 1024 slots each at least.
int select_blocks(int heads, int C)
{
    int n = 1;
    while (n < 8 && (long long)heads * n * 2 <= kPlanSms && C / (n * 2) >= 1024) n *= 2;
    return n;
}

// The selecting blocks move the rows too where there are enough of them to keep HBM busy, or little to move (one launch
// less, and no hand-over of the list: 128 heads of 2049 slots less one 6.8 us, by two kernels 1.5 more).  A few leave that
// to the whole GPU (8 heads of 100000 slots less half 75 us, themselves 114), and so do all of them where it takes longer
// than the select (d = 128: 32 heads 16384 -> 8192 slots 38.7 us, themselves 43.4; 128 heads 8192 -> 4096 65.7 and 69.1).
bool own_moves(int heads, int split, int C, int d, int keep)
{
    const long long blocks = (long long)heads * split, moves = (long long)most_moves(C, keep) * heads;
    return (blocks >= kOwnBlocks && moves * d <= kOwnElements * blocks) || moves <= kOwnMoves * blocks;
}

}  // namespace

size_t evict_workspace(int B, int H, int C, int d, int keep)
{
    const int split = select_blocks(B * H, C);
    // single blocks that move a short list keep it in shared memory
    if (split == 1 && own_moves(B * H, split, C, d, keep) && most_moves(C, keep) < kListMoves) return 0;
    return (size_t)B * H * moves_stride(C, keep) * 4;
}

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream)
{
    const int split = select_blocks(a.B * a.H, a.C), share = (a.C + split - 1) / split + 32;
    const int in_smem = share <= kMaxInSmem, bytes = in_smem ? (share + 3) / 4 * 16 : 0;
    const int stride = moves_stride(a.C, a.keep), most = most_moves(a.C, a.keep), blocks = a.B * a.H * split;
    const bool own = own_moves(a.B * a.H, split, a.C, a.d, a.keep);
    // Two smaller blocks an SM where larger ones would come in waves (512 heads of 2049 slots less one 15.0 us, by 1024
    // threads 22.4; 256 heads 4096 -> 2048 62.9 and 66.5); not for long runs (160 heads of 20000 slots 109, and 105 as it is).
    const bool small = split == 1 && blocks > kPlanSms && a.C <= kSmallSlots;
    static std::atomic<bool> set[6][64];
    const int which = (!own ? 0 : a.d == 64 ? 1 : 2) + (small ? 3 : 0);
    auto *const kernel = which == 0   ? select_kernel<0, 1024>
                         : which == 1 ? select_kernel<8, 1024>
                         : which == 2 ? select_kernel<16, 1024>
                         : which == 3 ? select_kernel<0, 512>
                         : which == 4 ? select_kernel<8, 512>
                                      : select_kernel<16, 512>;
    cudaError_t e = raise_smem(reinterpret_cast<const void *>(kernel), kMaxInSmem * 4, set[which]);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(kernel, dim3((unsigned)blocks), dim3(small ? 512 : 1024), (size_t)bytes, (unsigned)split, stream, a,
                          stride, in_smem, split);
    if (e != cudaSuccess || most == 0 || own) return e;
    const int each = (most + kMoveRows - 1) / kMoveRows;     // blocks a sequence and head
    const dim3 grid((unsigned)each * (unsigned)(a.B * a.H));
    return a.d == 64 ? launch_overlapped(move_kernel<8>, grid, dim3(256), 0, 1, stream, a, stride, each)
                     : launch_overlapped(move_kernel<16>, grid, dim3(256), 0, 1, stream, a, stride, each);
}

}  // namespace attn
