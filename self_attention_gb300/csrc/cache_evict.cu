// Eviction from a cache by accumulated attention weight.
//
// Per sequence and head, n = min(length, keep) slots stay: those of the `recent` newest positions first, then
// the ones of the largest weights, equal ones by the lower slot.  Kept slots at or behind n move into evicted
// ones before n, both in ascending order, so that sources and targets never meet, every move can run at once
// and a slot that stays in place costs nothing but its rank.
//
// select_kernel: one block a sequence and head.  A slot's rank is its weight's bits (weights count as zero where
// they are negative or NaN), all ones for the newest positions.  The n-th largest rank is found by three
// histograms of 11, 11 and 10 bits over ranks that stay in shared memory (from L2 where they do not fit), then
// one ordered pass over the slots numbers the ties, the holes and the movers.  move_kernel: the rows, 16 bytes
// a lane, over the whole GPU.
// Bound by HBM (8 bytes a slot, 8 d a moved slot) once there are enough sequences and heads, by the select's
// latency before.
#include "cluster.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxInSmem = 48 * 1024;    // ranks kept in shared memory (192 KB)
constexpr int kMoveRows = 32;            // moves a block of move_kernel takes

struct SelShared {
    uint32_t bins[kBins];
    uint32_t warp[32];
    uint32_t warp2[32];
    uint32_t prefix;                     // rank bits found so far
    uint32_t need;                       // how many are still to be taken among those with this prefix
    int newest;
};

// Sum over the lanes before this one, and over all of the warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, uint32_t lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= (uint32_t)o) v += t;
    }
    return v;
}

// Exclusive sum over the block's threads; `total` over all of them.  `buf` is free again after the next barrier.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *buf, uint32_t &total)
{
    const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t inc = warp_scan(v, lane);
    if (lane == 31) buf[w] = inc;
    __syncthreads();
    const uint32_t part = buf[lane];
    const uint32_t sums = warp_scan(part, lane);
    total = __shfl_sync(0xffffffffu, sums, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, sums - part, w);
    return before + inc - v;
}

__device__ __forceinline__ uint32_t rank_of(float w, int pos, long long oldest)
{
    if (pos > oldest) return 0xffffffffu;
    return w > 0.f ? __float_as_uint(w) : 0u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(EvictArgs a, int stride, int in_smem)
{
    extern __shared__ __align__(16) uint32_t ranks[];
    __shared__ SelShared s;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tid = threadIdx.x, bh = blockIdx.x, b = bh / a.H;
    const int L = min(max(a.lengths[b], 0), a.C), n = min(L, a.keep);
    const long long row = (long long)bh * a.C;
    const float *w = a.weights + row;
    const int *pos = a.slot_positions + row;
    float *w_out = a.weights_out + row;
    int *pos_out = a.positions_out + row;
    int *moves = a.moves + (long long)bh * stride;
    if (bh % a.H == 0 && tid == 0) a.lengths_out[b] = n;
    // what lies behind the kept slots is empty; sources of moves are emptied by those who read them
    if (n == L) {
        for (int j = tid; j < a.C; j += kSelThreads) {
            const float x = w[j];
            const int p = pos[j];
            w_out[j] = j < n ? x : 0.f;
            pos_out[j] = j < n ? p : -1;
        }
        if (tid == 0) moves[0] = 0;
        return;
    }

    // the newest position
    int newest = INT32_MIN;
    for (int j = tid; j < L; j += kSelThreads) newest = max(newest, pos[j]);
    newest = __reduce_max_sync(0xffffffffu, newest);
    if ((tid & 31) == 0) s.warp[tid >> 5] = (uint32_t)newest;
    __syncthreads();
    newest = __reduce_max_sync(0xffffffffu, (int)s.warp[tid & 31]);
    const long long oldest = (long long)newest - a.recent;   // positions above it are safe
    if (in_smem)
        for (int j = tid; j < L; j += kSelThreads) ranks[j] = rank_of(w[j], pos[j], oldest);
    auto rank = [&](int j) { return in_smem ? ranks[j] : rank_of(w[j], pos[j], oldest); };

    // the n-th largest rank
    uint32_t prefix = 0, need = (uint32_t)n;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
        for (int i = tid; i < kBins; i += kSelThreads) s.bins[i] = 0;
        __syncthreads();
        for (int j0 = 0; j0 < L; j0 += kSelThreads) {
            const int j = j0 + tid;
            const uint32_t r = j < L ? rank(j) : 0u;
            const bool in = j < L && (r & mask) == prefix;
            const uint32_t bin = r >> shift & ((1u << bits) - 1);
            // neighbours often share a bin (weights of one magnitude, ties of zero): one addition for all of them
            const uint32_t same = __match_any_sync(0xffffffffu, in ? bin : 0xffffffffu);
            if (in && (same & ((1u << (tid & 31)) - 1)) == 0) atomicAdd(&s.bins[bin], (uint32_t)__popc(same));
        }
        __syncthreads();
        // bins from the top: thread t holds bins 2 (1023 - t) + 1 and 2 (1023 - t)
        const int top = 2 * (kSelThreads - 1 - tid) + 1;
        const uint32_t c1 = s.bins[top], c0 = s.bins[top - 1];
        uint32_t total;
        const uint32_t above = block_scan(c0 + c1, s.warp2, total);
        if (above < need && need <= above + c0 + c1) {
            const bool first = need <= above + c1;
            s.prefix = prefix | (uint32_t)(first ? top : top - 1) << shift;
            s.need = need - above - (first ? 0 : c1);
        }
        __syncthreads();
        prefix = s.prefix;
        need = s.need;
    }

    // In order: ranks above `prefix` stay, and the first `need` that equal it.
    uint32_t ties = 0, holes = 0, movers = 0;
    for (int j0 = 0; j0 < L; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t r = j < L ? rank(j) : 0u;
        const bool eq = j < L && r == prefix;
        uint32_t total;
        const uint32_t t = ties + block_scan(eq, s.warp, total);
        ties += total;
        const bool kept = j < L && (r > prefix || (eq && t < need));
        const bool hole = j < n && !kept, mover = j >= n && kept;
        const uint32_t at = block_scan((uint32_t)hole | (uint32_t)mover << 16, s.warp2, total);
        if (hole) moves[1 + 2 * (holes + (at & 0xffff))] = j;
        if (mover) moves[2 + 2 * (movers + (at >> 16))] = j;
        holes += total & 0xffff;
        movers += total >> 16;
        if (j < L && j < n ? kept : j < L && !mover) {
            const float x = w[j];
            const int p = pos[j];
            w_out[j] = j < n ? x : 0.f;
            pos_out[j] = j < n ? p : -1;
        }
    }
    for (int j = L + tid; j < a.C; j += kSelThreads) {
        w_out[j] = 0.f;
        pos_out[j] = -1;
    }
    if (tid == 0) moves[0] = (int)holes;
}

// LANES lanes a row of d = 8 LANES columns.
template <int LANES>
__global__ void __launch_bounds__(256) move_kernel(EvictArgs a, int stride, int blocks)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int bh = blockIdx.x / blocks, lane = threadIdx.x % LANES;
    const int *moves = a.moves + (long long)bh * stride;
    const int count = moves[0], first = blockIdx.x % blocks * kMoveRows;
    const int last = min(first + kMoveRows, count);
    const long long row = (long long)bh * a.C;
    uint4 *k = static_cast<uint4 *>(a.k) + row * LANES, *v = static_cast<uint4 *>(a.v) + row * LANES;
    constexpr int STEP = 256 / LANES;
    for (int m = first + threadIdx.x / LANES; m < last; m += STEP) {
        const long long dst = moves[1 + 2 * m], src = moves[2 + 2 * m];
        const uint4 x = k[src * LANES + lane], y = v[src * LANES + lane];
        k[dst * LANES + lane] = x;
        v[dst * LANES + lane] = y;
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

int most_moves(int C, int keep) { return keep < C - keep ? keep : C - keep > 0 ? C - keep : 0; }
int moves_stride(int C, int keep) { return (1 + 2 * most_moves(C, keep) + 3) / 4 * 4; }

}  // namespace

size_t evict_workspace(int B, int H, int C, int keep) { return (size_t)B * H * moves_stride(C, keep) * 4; }

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream)
{
    const int in_smem = a.C <= kMaxInSmem, bytes = in_smem ? (a.C + 3) / 4 * 16 : 0;
    const int stride = moves_stride(a.C, a.keep);
    static std::atomic<bool> set[64];
    cudaError_t e = raise_smem(reinterpret_cast<const void *>(select_kernel), kMaxInSmem * 4, set);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(select_kernel, dim3((unsigned)(a.B * a.H)), dim3(kSelThreads), (size_t)bytes, 1, stream, a,
                          stride, in_smem);
    const int most = most_moves(a.C, a.keep);
    if (e != cudaSuccess || most == 0) return e;
    const int blocks = (most + kMoveRows - 1) / kMoveRows;     // a sequence and head
    const dim3 grid((unsigned)blocks * (unsigned)(a.B * a.H));
    return a.d == 64 ? launch_overlapped(move_kernel<8>, grid, dim3(256), 0, 1, stream, a, stride, blocks)
                     : launch_overlapped(move_kernel<16>, grid, dim3(256), 0, 1, stream, a, stride, blocks);
}

}  // namespace attn
