// Attention of one token, a chain or a tree of drafted tokens over a cache:
//   o = sum_j p_j v_j,  p_j = exp(scale q.k_j - lse),  lse = log sum_j exp(scale q.k_j),
// over the slots j < length and, of the T tokens that follow them in the cache, those that the token's mask
// word names.  Bound by HBM: each slot's K and V (4 d bytes) meet the few rows of the heads that share them; short
// caches by latency.  The rows of a (sequence, cached head), r = g T + t, are one contiguous block of q and o; a unit is 8,
// 16, 128 or 256 of them.
//
// Up to 16 rows (unit_kernel, few_kernel; more where the cache is short).  The products are turned round so that the
// slots are the 16-row operand of mma.sync and the few query rows its 8 columns: S^T = K Q^T, O^T = V^T P^T (a tcgen05
// tile would be nearly empty with so few rows, and its result is a round trip through tensor memory away; the tensor pipe
// is at 15 % as it is).  A warp takes 16 slots a step, from a ring that TMA fills for it alone:
//   K   thread (g, q) = (lane / 4, lane % 4) reads chunks 4 c + q of slots g and g + 8; the sum over d runs in the
//       order that these chunks give, the same for Q.
//   V   it reads chunk g (and g + 8) of slots 2 q, 2 q + 1, 2 q + 8, 2 q + 9; two slots' values of a column
//       are put side by side by byte permutes, and column 8 g + j is row g of the j-th 16-row tile.
//   P   leaves S^T's accumulator as pairs of rows; movmatrix turns it into pairs of slots.
// No barrier of the CTA in the loop: each warp keeps its own running maximum and sum, and asks for a step as soon as it
// has used one up.  Eight warps with three steps each (192 KB an SM on their way at d = 128) draw 6.4 TB/s (32 sequences
// of 16000 slots and 4 cached heads, 160 us); loads into registers, twelve warps with one step ahead, 6.1 (170 us), and
// the same ring by cp.async 5.2 (201 us: the copies' instructions sit on each warp's chain).  P meets V as two bf16
// terms (its upper bits and the rest), 2^-15 of it: one term alone would cost 2^-8 of each weight, and the pipe has room.
//
// Work is shared out in blocks of 128 slots over all units (few_kernel, many_kernel), the same number for each CTA or
// nearly so (the lengths are on the device: each CTA finds its share itself).  A unit that one CTA has whole is finished
// there; the others' parts go to the workspace with their maximum and sum, and a second kernel adds them in the order of
// their slots.  Where a unit's slots are few enough for one CTA or cluster (unit_kernel, many_kernel by whole units)
// nothing is joined through memory.  choose() takes the kernels by the sizes.  Nothing depends on timing: results are
// bitwise reproducible.
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kBlock = 16 * kFewWarps;   // slots of a block of work
constexpr int kAbortBytes = 16;          // of the word that says a wait has given up, behind the barriers

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Cached keys and values are read once (by one CTA): no room in L1 for them.
__device__ __forceinline__ uint4 stream16(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Values that are not finite.
__device__ __forceinline__ bool odd_value(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ bool odd_pair(uint32_t w) { return odd_value(lo(w)) || odd_value(hi(w)); }
__device__ __forceinline__ bool any_odd(const uint4 &v)
{
    return odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w);
}
__device__ __forceinline__ void drop_odd(uint32_t &w)
{
    if (odd_value(lo(w))) w &= 0xffff0000u;
    if (odd_value(hi(w))) w &= 0x0000ffffu;
}
__device__ __forceinline__ void drop_odd(uint4 &v)
{
    drop_odd(v.x);
    drop_odd(v.y);
    drop_odd(v.z);
    drop_odd(v.w);
}

// How the work of all units is shared out.  Sequence b has H * tiles units of blocks(b) blocks each.
struct Plan {
    int H, tiles, T, C;
    int block;       // slots a block of work
    int whole;       // a CTA takes one unit whole (and nothing is shared out)
    int slack;       // blocks that a CTA may have more if it then has one unit's alone
};

// Slots of the cache ahead of the new tokens.
__device__ __forceinline__ int length_of(const int *lengths, int b, int T, int C)
{
    return min(max(lengths[b], 0), C - T);
}

__device__ __forceinline__ int blocks_of(int length, const Plan &p) { return (length + p.T + p.block - 1) / p.block; }

// a / b, by a 32-bit division where both fit.
__device__ __forceinline__ long long divide(long long a, int b)
{
    return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// What a CTA's share is: `per` blocks in the order of the units; or, where that takes at most `slack` blocks more, up to
// `per` blocks of one unit alone (apart), since the end of a unit costs about two blocks' time.
struct Shares {
    long long per;
    bool apart;
};

// From the blocks n of the lane's own sequence (up to 32 of them); by a whole warp.
__device__ __forceinline__ Shares shares_of(int n, const Plan &p, int ctas)
{
    const long long units = (long long)p.H * p.tiles;
    const long long all = (long long)__reduce_add_sync(0xffffffffu, n) * units;
    const int per = (int)min(divide(all + ctas - 1, ctas), 0x7ffffff0ll);
    for (int k = 0; k <= p.slack; ++k)
        if ((long long)__reduce_add_sync(0xffffffffu, (n + per + k - 1) / (per + k)) * units <= ctas) return {per + k, true};
    return {per, false};
}

// Blocks of all sequences, and of those ahead of sequence `upto`; by a whole warp, the same in every lane.
__device__ __forceinline__ long long count_blocks(const int *lengths, int B, int upto, const Plan &p, long long &before)
{
    long long all = 0, ahead = 0;
    for (int b = threadIdx.x & 31; b < B; b += 32) {
        const int n = blocks_of(length_of(lengths, b, p.T, p.C), p);
        all += n;
        ahead += b < upto ? n : 0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    }
    before = ahead * p.H * p.tiles;
    return all * p.H * p.tiles;
}

// A run of blocks of one unit, that one CTA works on.
struct Segment {
    long long head;         // b H + h
    int b, tile, first, last, nb, length;
    bool there;
    __device__ __forceinline__ bool whole() const { return first == 0 && last == nb; }
};

// Walks over a CTA's share of the blocks, the same number for each.
struct Walk {
    long long x, end, before;
    int b, length, nb;
    // By a whole warp.
    __device__ __forceinline__ bool begin(const int *lengths, int B, const Plan &p)
    {
        const uint32_t lane = threadIdx.x & 31;
        const long long per_unit = (long long)p.H * p.tiles;
        if (p.whole) {
            b = (int)(blockIdx.x / (unsigned)per_unit);
            length = length_of(lengths, b, p.T, p.C);
            nb = blocks_of(length, p);
            before = 0;
            x = (long long)(blockIdx.x % (unsigned)per_unit) * nb;
            end = x + nb;
            return true;
        }
        int len = (int)lane < B ? length_of(lengths, (int)lane, p.T, p.C) : 0, inc;
        int n = (int)lane < B ? blocks_of(len, p) : 0;
        auto scan = [&](int v) {         // the sum of v over the lanes up to this one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= (uint32_t)o) v += t;
            }
            return v;
        };
        if (B <= 32) {
            const Shares sh = shares_of(n, p, (int)gridDim.x);
            if (sh.apart) {
                const int per = (int)sh.per, mine = (n + per - 1) / per;       // CTAs a unit of this sequence
                inc = scan(mine);
                const uint32_t hit = __ballot_sync(0xffffffffu, blockIdx.x < inc * per_unit);
                if (!hit) return false;
                const int l = __ffs(hit) - 1, k = __shfl_sync(0xffffffffu, mine, l);
                const int at = (int)(blockIdx.x - __shfl_sync(0xffffffffu, inc - mine, l) * per_unit), u = at / k;
                length = __shfl_sync(0xffffffffu, len, l);
                nb = blocks_of(length, p);
                b = l;
                before = 0;
                x = (long long)u * nb + (long long)(at - u * k) * per;
                end = min(x + per, (long long)(u + 1) * nb);
                return true;
            }
            end = (long long)__reduce_add_sync(0xffffffffu, n) * per_unit;
            x = sh.per * blockIdx.x;
            end = min(x + sh.per, end);
        } else {
            long long ignored;
            const long long all = count_blocks(lengths, B, 0, p, ignored), per = divide(all + gridDim.x - 1, (int)gridDim.x);
            x = per * blockIdx.x;
            end = min(x + per, all);
        }
        if (x >= end) return false;
        inc = scan(n);
        long long sum = 0;
        for (int b0 = 0;;) {          // ends: x lies before `all`
            const uint32_t hit = __ballot_sync(0xffffffffu, x < (sum + inc) * per_unit);
            if (hit) {
                const int l = __ffs(hit) - 1;
                before = (sum + __shfl_sync(0xffffffffu, inc - n, l)) * per_unit;
                length = __shfl_sync(0xffffffffu, len, l);
                nb = blocks_of(length, p);
                b = b0 + l;
                return true;
            }
            sum += __shfl_sync(0xffffffffu, inc, 31);
            b0 += 32;
            len = b0 + (int)lane < B ? length_of(lengths, b0 + (int)lane, p.T, p.C) : 0;
            n = b0 + (int)lane < B ? blocks_of(len, p) : 0;
            inc = scan(n);
        }
    }
    // By any thread.
    __device__ __forceinline__ bool next(const int *lengths, const Plan &p, Segment &s)
    {
        s.there = x < end;
        if (!s.there) return false;
        while (x >= before + (long long)nb * p.H * p.tiles) {
            before += (long long)nb * p.H * p.tiles;
            ++b;
            length = length_of(lengths, b, p.T, p.C);
            nb = blocks_of(length, p);
        }
        const long long u = divide(x - before, nb);          // unit of the sequence
        s.first = (int)(x - before - u * nb);
        s.last = (int)min((long long)nb, s.first + (end - x));
        const long long h = divide(u, p.tiles);
        s.tile = (int)(u - h * p.tiles);
        s.b = b;
        s.nb = nb;
        s.length = length;
        s.head = (long long)b * p.H + h;
        x += s.last - s.first;
        return true;
    }
};

// Which tokens token t sees, as bits.
__device__ __forceinline__ uint64_t word_of(const uint64_t *tree, int b, int T, int t)
{
    return tree ? tree[(long long)b * T + t] : (2ull << t) - 1;
}

// Partial results: slot 2 c for the part that CTA c begins inside a unit, 2 c + 1 for the one it begins a unit with.
struct Parts {
    float *o;          // [2 grid][rows][d]; many_kernel's [2 grid][d / 4][rows][4], so that its threads, one a row, write runs
    float2 *ml;        // [2 grid][rows]: maximum (of scores times log2 e) and sum
    float *scores;     // null, or [B H][G T][C]: scores times log2 e, -infinity where a row does not see a slot
};

// Lanes that differ in `bit` change places: the one without it gives b for the other's a.
__device__ __forceinline__ void exchange(uint4 &a, uint4 &b, int bit)
{
    const bool up = (threadIdx.x & bit) != 0;
    const uint4 give = up ? a : b;
    const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, bit), __shfl_xor_sync(0xffffffffu, give.y, bit),
                                 __shfl_xor_sync(0xffffffffu, give.z, bit), __shfl_xor_sync(0xffffffffu, give.w, bit));
    if (up) a = got;
    else b = got;
}

// Waits for what is already on its way, for a second at most, whether or not the CTA has given up.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > 1000000000ull) return;
}

struct KvMaps {
    CUtensorMap k, v;         // [B H][C][d], boxes of 64 columns x 16 slots
};

// A warp's state: 8 NT rows of one unit against 16 slots a step.  K and V of the steps ahead come by TMA into a ring of
// STAGES steps that is the warp's own (64 columns a box, 128-byte swizzle: V is read without bank conflicts, K with two
// ways), each stage with a barrier that nobody but this warp waits on.
template <int D, int NT, int STAGES_>
struct Rows {
    static constexpr int STAGES = STAGES_;
    static constexpr int KC = D / 32;           // chunks of a K row a thread holds
    static constexpr int VC = D / 64;           // chunks of a V row a thread holds
    static constexpr int MT = D / 16;           // 16-row tiles of O^T
    static constexpr uint32_t BOX = 16 * 128, STAGE = 2 * (D / 64) * BOX, RING = STAGES * STAGE;    // bytes
    uint4 qf[NT][KC];
    uint64_t word[NT][2];                       // what rows 2 q and 2 q + 1 see of the tokens
    float acc[NT][MT][4], m[NT][2], l[NT][2], s[NT][4];
    int g, q;
    uint8_t *ring;                              // 1024-byte aligned
    uint64_t *bars;
    uint32_t asked, taken;                      // steps

    __device__ __forceinline__ Rows(uint8_t *warp_ring, uint64_t *warp_bars)
        : g((threadIdx.x & 31) >> 2), q(threadIdx.x & 3), ring(warp_ring), bars(warp_bars), asked(0), taken(0)
    {
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
        }
    }
    // Q's rows from r0 on as the 8-column operand, and their mask words (the last step needs them at once)
    __device__ __forceinline__ void load_q(const CacheAttnArgs &a, long long head, int b, int r0)
    {
        const int R = a.G * a.T;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 8 * t + 2 * q + e;
                word[t][e] = r < R ? word_of(a.tree, b, a.T, r % a.T) : 0;
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 8 * t + g;
            const uint4 *qp = static_cast<const uint4 *>(a.q) + (head * R + r) * (D / 8);
#pragma unroll
            for (int c = 0; c < KC; ++c) qf[t][c] = r < R ? qp[4 * c + q] : make_uint4(0, 0, 0, 0);
        }
    }
    // Asks for 16 slots from `key` on.
    __device__ __forceinline__ void load(const KvMaps &maps, long long head, int key)
    {
        __syncwarp();                           // the stage's last step has been read by every lane
        if ((threadIdx.x & 31) == 0) {
            const uint32_t st = asked % STAGES;
            uint8_t *to = ring + st * STAGE;
            ptx::mbar_arrive_expect_tx(&bars[st], STAGE);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                ptx::tma_load_3d(to + c * BOX, &maps.k, &bars[st], 64 * c, key, (int)head);
                ptx::tma_load_3d(to + (D / 64 + c) * BOX, &maps.v, &bars[st], 64 * c, key, (int)head);
            }
        }
        ++asked;
    }
    // Nothing stays on its way when the warp leaves (matters only after a timeout).
    __device__ __forceinline__ void finish()
    {
        for (; taken < asked; ++taken) drain(&bars[taken % STAGES], taken / STAGES & 1);
    }
    // S^T = K Q^T of the step that was asked for first; two sums, whose products need not wait for one another.
    __device__ __forceinline__ void scores(const Guard &guard)
    {
        const uint32_t st = taken % STAGES, at = ptx::smem_u32(ring) + st * STAGE + g * 128;
        wait_bounded(&bars[st], taken / STAGES & 1, guard);
        uint4 kr[2][KC];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kr[i][c] = lds_u128(at + i * 1024 + (c >> 1) * BOX + (((q ^ g) ^ (c & 1) * 4) << 4));
        float s1[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) s1[t][0] = s1[t][1] = s1[t][2] = s1[t][3] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t a0[4] = {kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y};
            const uint32_t a1[4] = {kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mma16816(s[t], a0, qf[t][c].x, qf[t][c].y);
                mma16816(s1[t], a1, qf[t][c].z, qf[t][c].w);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] += s1[t][e];
    }
    // The rest of the step at `key`: weights, and O^T += V^T P^T.  kept: see Parts::scores
    __device__ __forceinline__ void step(const CacheAttnArgs &a, long long head, int r0, int key, int length, float to_log2,
                                         float *kept)
    {
        const int T = a.T, R = a.G * T;
        const bool tail = key + 16 > length;
        uint4 vr[4][VC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int j = 2 * q + (i & 1);
                vr[i][c] = lds_u128(ptx::smem_u32(ring) + taken % STAGES * STAGE + (D / 64 + c) * BOX + (j + 8 * (i >> 1)) * 128 +
                                    ((g ^ j) << 4));
            }
        ++taken;
        if (tail) {          // whatever lies behind the last slot is not a value
            const int left = length + T - key - 2 * q;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    if ((i & 1) + 8 * (i >> 1) >= left) vr[i][c] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] *= to_log2;
            if (tail) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = key + g + 8 * i - length;
                        if (j >= 0 && !(j < T && (word[t][e] >> j & 1))) s[t][e + 2 * i] = -INFINITY;
                    }
                }
            }
            if (kept) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r0 + 8 * t + 2 * q + (e & 1), j = key + g + 8 * (e >> 1);
                    if (r < R && j < length + T) kept[(head * R + r) * a.C + j] = s[t][e];
                }
            }
            // The maximum is brought up to date only where some score exceeds it.
            const float top[2] = {fmaxf(s[t][0], s[t][2]), fmaxf(s[t][1], s[t][3])};
            if (__any_sync(0xffffffffu, top[0] > m[t][0] || top[1] > m[t][1])) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float w = fmaxf(m[t][e], top[e]);
                    w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 4));
                    w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 8));
                    w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 16));
                    const float f = w == -INFINITY ? 1.f : ptx::ex2(m[t][e] - w);
                    m[t][e] = w;
                    l[t][e] *= f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[t][i][e] *= f;
                        acc[t][i][e + 2] *= f;
                    }
                }
            }
        }
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float base = m[t][e & 1] == -INFINITY ? 0.f : m[t][e & 1];
                p[e] = ptx::ex2(s[t][e] - base);
                l[t][e & 1] += p[e];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // the upper bits and the rest, at least 2^-24 of p: it is of p's sign, and 0 only where p is (or below 2^-100),
                // so that an infinite value keeps its sign under both
                const uint32_t w = __byte_perm(__float_as_uint(p[2 * i]), __float_as_uint(p[2 * i + 1]), 0x7632);
                const float x0 = fmaxf(p[2 * i] - lo(w), p[2 * i] * 0x1p-24f);
                const float x1 = fmaxf(p[2 * i + 1] - hi(w), p[2 * i + 1] * 0x1p-24f);
                ph[t][i] = transpose8x8(w);
                pl[t][i] = transpose8x8(ptx::pack_bf16x2(x0, x1));
            }
        }
        // A token's value that is not finite may reach the rows that see it alone, but 0 times it is NaN in a
        // product: such values are added one by one and leave the operand.  Rare, and only among the T tokens (a mask word
        // may leave out a single one; without masks it sees itself).
        if (tail && (T > 1 || a.tree)) {
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    odd |= key + 2 * q + (i & 1) + 8 * (i >> 1) >= length && any_odd(vr[i][c]);
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    for (int from = 0; from < 4; ++from) {      // slot 2 from + (i & 1) + 8 (i >> 1)
                        const int j = 2 * from + (i & 1) + 8 * (i >> 1);
                        if (key + j < length) continue;
#pragma unroll
                        for (int c = 0; c < VC; ++c) {
                            const uint32_t w[4] = {__shfl_sync(0xffffffffu, vr[i][c].x, 4 * g + from),
                                                   __shfl_sync(0xffffffffu, vr[i][c].y, 4 * g + from),
                                                   __shfl_sync(0xffffffffu, vr[i][c].z, 4 * g + from),
                                                   __shfl_sync(0xffffffffu, vr[i][c].w, 4 * g + from)};
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float seen = __shfl_sync(0xffffffffu, s[t][e + 2 * (i >> 1)], 4 * (j % 8) + q);
#pragma unroll
                                    for (int x = 0; x < 8; ++x) {
                                        const float v = x & 1 ? hi(w[x / 2]) : lo(w[x / 2]);
                                        if (seen != -INFINITY && odd_value(v))
                                            acc[t][D == 128 ? x : x & 3][e + 2 * (D == 128 ? c : x >> 2)] += v;
                                    }
                                }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < VC; ++c)
                        if (key + 2 * q + (i & 1) + 8 * (i >> 1) >= length) drop_odd(vr[i][c]);
            }
        }
        // O^T += V^T P^T.  Tile j of 16 rows: columns 8 g + j of one chunk, and of the other (d = 64: the other half of
        // the one).
        uint32_t af[MT][4];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)          // a slot pair
#pragma unroll
                for (int c = 0; c < 2; ++c) {    // rows g and g + 8 of the tile
                    const int e = D == 128 ? j : j + 4 * c;     // column of the chunk
                    const uint4 &x = vr[2 * i][D == 128 ? c : 0], &y = vr[2 * i + 1][D == 128 ? c : 0];
                    const uint32_t u = e / 2 == 0 ? x.x : e / 2 == 1 ? x.y : e / 2 == 2 ? x.z : x.w;
                    const uint32_t w = e / 2 == 0 ? y.x : e / 2 == 1 ? y.y : e / 2 == 2 ? y.z : y.w;
                    af[j][2 * i + c] = __byte_perm(u, w, e & 1 ? 0x7632 : 0x5410);
                }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < MT; ++j) mma16816(acc[t][j], af[j], ph[t][0], ph[t][1]);
#pragma unroll
            for (int j = 0; j < MT; ++j) mma16816(acc[t][j], af[j], pl[t][0], pl[t][1]);
        }
    }
    // A warp's results into shared memory as they lie in its registers, and into those of another warp.
    __device__ __forceinline__ void hand_over(float *to)          // [NT (4 MT + 4)][32]
    {
        float *x = to + (threadIdx.x & 31);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[((t * MT + i) * 4 + e) * 32] = acc[t][i][e];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[(NT * MT * 4 + t * 4 + e) * 32] = m[t][e];
                x[(NT * MT * 4 + t * 4 + 2 + e) * 32] = l[t][e];
            }
        }
    }
    __device__ __forceinline__ void take_over(const float *from)
    {
        const float *x = from + (threadIdx.x & 31);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float other = x[(NT * MT * 4 + t * 4 + e) * 32], top = fmaxf(m[t][e], other);
                const float base = top == -INFINITY ? 0.f : top;
                const float f = ptx::ex2(m[t][e] - base), p = ptx::ex2(other - base);
                m[t][e] = top;
                l[t][e] = l[t][e] * f + x[(NT * MT * 4 + t * 4 + 2 + e) * 32] * p;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    acc[t][i][e] = acc[t][i][e] * f + x[((t * MT + i) * 4 + e) * 32] * p;
                    acc[t][i][e + 2] = acc[t][i][e + 2] * f + x[((t * MT + i) * 4 + e + 2) * 32] * p;
                }
            }
    }
    // The warp's results into shared memory, rows of D + 4 floats.
    __device__ __forceinline__ void leave(float *o, float2 *ml)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
                const int r = 8 * t + 2 * q + e;
                if (g == 0) ml[r] = make_float2(m[t][e], l[t][e]);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < MT; j += 4)
                        *reinterpret_cast<float4 *>(o + r * (D + 4) + (D == 128 ? 64 * c + 8 * g + j : 8 * g + 4 * c)) =
                            make_float4(acc[t][j][e + 2 * c], acc[t][j + 1][e + 2 * c], acc[t][j + 2][e + 2 * c],
                                        acc[t][j + 3][e + 2 * c]);
            }
    }
};

// What the warps left of a unit's rows.
template <int D, int NT, int WARPS>
struct Left {
    float o[WARPS][8 * NT][D + 4];
    float2 ml[WARPS][8 * NT];
};

// Row r, columns c ... c + 7 over the warps: maximum and sum, o unnormalised.
template <int D, int NT, int WARPS>
__device__ __forceinline__ float2 gather(const Left<D, NT, WARPS> &sm, int r, int c, float (&o)[8])
{
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sm.ml[w][r].x);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const float2 ml = sm.ml[w][r];
        const float f = ptx::ex2(ml.x - base);
        sum += f * ml.y;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += f * sm.o[w][r][c + e];
    }
    return make_float2(top, sum);
}

// A row that sees nothing has a sum of zero.
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float top, float sum)
{
    return sum == 0.f ? -INFINITY : (top + log2f(sum)) * (1.f / kLog2e);
}

__device__ __forceinline__ void write_o8(const CacheAttnArgs &a, long long row, int c, const float (&o)[8], float inv)
{
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + row * a.d + c) =
        make_uint4(ptx::pack_bf16x2(o[0] * inv, o[1] * inv), ptx::pack_bf16x2(o[2] * inv, o[3] * inv),
                   ptx::pack_bf16x2(o[4] * inv, o[5] * inv), ptx::pack_bf16x2(o[6] * inv, o[7] * inv));
}

template <int D, int NT>
struct FewCfg {
    static constexpr int BLOCKS = D == 64 && NT == 1 ? 2 : 1;    // CTAs an SM
    static constexpr int STAGES = NT == 1 ? 3 : D == 64 ? 5 : 2;
    using R = Rows<D, NT, STAGES>;
    static constexpr int HALF = kFewWarps / 2;
    using L = Left<D, NT, HALF>;
    static constexpr int HELD = NT * (D / 4 + 4) * 32;        // floats a warp hands over
    static constexpr int RINGS = kFewWarps * (int)R::RING, HANDED = HALF * HELD * 4;
    static constexpr int JOIN = HANDED > (int)sizeof(L) ? HANDED : (int)sizeof(L);
    static constexpr int SMEM = RINGS + JOIN + kFewWarps * STAGES * 8 + kAbortBytes + 1024;
    static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "");
};

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, FewCfg<D, NT>::BLOCKS)
    few_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ CacheAttnArgs a, Plan plan, Parts parts)
{
    using C = FewCfg<D, NT>;
    constexpr int R8 = 8 * NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    typename C::L &left = *reinterpret_cast<typename C::L *>(smem + C::RINGS);
    float *handed = reinterpret_cast<float *>(smem + C::RINGS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::RINGS + C::JOIN);
    int *abort = reinterpret_cast<int *>(bars + kFewWarps * C::STAGES);
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, T = a.T, R = a.G * T;
    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < kFewWarps * C::STAGES; ++i) ptx::mbar_init(&bars[i], 1);
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&maps.k);
        ptx::tma_prefetch_desc(&maps.v);
    }
    __syncthreads();
    ptx::grid_dep_wait();
    Walk walk;
    if (!walk.begin(a.lengths, a.B, plan)) return;
    const Guard guard{abort, a.status, kWaitLimitNs};
    const float to_log2 = a.scale * kLog2e;
    typename C::R w(smem + warp * C::R::RING, bars + warp * C::STAGES);
    auto first_key = [&](const Segment &s) { return s.first * kBlock + 16 * warp; };
    // What is asked for runs ahead of what is worked on, over the ends of segments.
    Walk walk_ahead = walk;
    Segment seg, ahead;
    walk_ahead.next(a.lengths, plan, ahead);
    int key_ahead = first_key(ahead);
    auto ask = [&] {
        if (!ahead.there) return;
        w.load(maps, ahead.head, key_ahead);
        key_ahead += kBlock;
        if (key_ahead >= ahead.last * kBlock && walk_ahead.next(a.lengths, plan, ahead)) key_ahead = first_key(ahead);
    };
    ask();
    walk.next(a.lengths, plan, seg);
    w.load_q(a, seg.head, seg.b, seg.tile * R8);
#pragma unroll
    for (int i = 1; i < C::STAGES; ++i) ask();

    while (seg.there) {
        const int r0 = seg.tile * R8, end = seg.last * kBlock;
        Segment nxt;
        walk.next(a.lengths, plan, nxt);
        w.clear();
        for (int key = first_key(seg); key < end; key += kBlock) {       // (a warp's share of the last block may be empty)
            w.scores(guard);
            w.step(a, seg.head, r0, key, seg.length, to_log2, parts.scores);
            ask();
            if (key + kBlock >= end && nxt.there) w.load_q(a, nxt.head, nxt.b, nxt.tile * R8);
        }
        // half of the warps take the others' results over, then the rows are put together
        if (warp >= C::HALF) w.hand_over(handed + (warp - C::HALF) * C::HELD);
        __syncthreads();
        if (warp < C::HALF) {
            w.take_over(handed + warp * C::HELD);
            ptx::named_bar(1, 32 * C::HALF);
            w.leave(&left.o[warp][0][0], left.ml[warp]);
        }
        __syncthreads();
        const long long slot = 2 * (long long)blockIdx.x + (seg.first == 0 ? 1 : 0);
        constexpr int PER = D / 8;       // threads a row, 8 columns each
        for (int i = threadIdx.x; i < R8 * PER; i += kFewThreads) {
            const int r = i / PER, c = i % PER * 8;
            float o[8];
            const float2 ml = gather(left, r, c, o);
            if (r0 + r >= R) continue;
            if (seg.whole()) {
                const long long at = seg.head * R + r0 + r;
                write_o8(a, at, c, o, inverse_of(ml.y));
                if (c == 0) a.lse[at] = lse_of(ml.x, ml.y);
            } else {
                float4 *to = reinterpret_cast<float4 *>(parts.o + (slot * R8 + r) * D + c);
                to[0] = make_float4(o[0], o[1], o[2], o[3]);
                to[1] = make_float4(o[4], o[5], o[6], o[7]);
                if (c == 0) parts.ml[slot * R8 + r] = ml;
            }
        }
        __syncthreads();
        seg = nxt;
    }
    w.finish();
}

// unit_kernel: the same where a unit's slots, as many as the cache has room for, are few enough for one cluster of 1
// to 8 CTAs: each warp takes every (8 cluster)-th run of 16, the CTAs' results meet in distributed shared memory, and
// there are no parts and no join_kernel (the two launches' hand-over, the lengths a second time and the parts' way
// through L2 take 4 us).
constexpr int kUnitWarps = 8;

template <int D, int NT>
struct UnitCfg {
    static constexpr int STAGES = 3;
    static constexpr int BLOCKS = D == 128 ? 1 : 2;
    using R = Rows<D, NT, STAGES>;
    using L = Left<D, NT, kUnitWarps>;
    struct Sum {
        float o[8 * NT][D];              // the CTA's sum, read by the cluster
        float2 ml[8 * NT];
    };
    // what the warps leave goes over their rings
    static constexpr int RINGS = kUnitWarps * (int)R::RING;
    static_assert(sizeof(L) <= RINGS, "");
    static constexpr int SMEM = RINGS + (int)sizeof(Sum) + kUnitWarps * STAGES * 8 + kAbortBytes + 1024;
    static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "");
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * kUnitWarps, UnitCfg<D, NT>::BLOCKS)
    unit_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ CacheAttnArgs a, int tiles, float *kept)
{
    using C = UnitCfg<D, NT>;
    constexpr int R8 = 8 * NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    typename C::L &left = *reinterpret_cast<typename C::L *>(smem);
    typename C::Sum &sm = *reinterpret_cast<typename C::Sum *>(smem + C::RINGS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::RINGS + sizeof(typename C::Sum));
    int *abort = reinterpret_cast<int *>(bars + kUnitWarps * C::STAGES);
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, T = a.T, R = a.G * T;
    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < kUnitWarps * C::STAGES; ++i) ptx::mbar_init(&bars[i], 1);
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&maps.k);
        ptx::tma_prefetch_desc(&maps.v);
    }
    const int ctas = (int)ptx::cluster_size(), rank = (int)ptx::cluster_rank();
    const unsigned unit = blockIdx.x / (unsigned)ctas;
    const long long head = unit / (unsigned)tiles;
    const int r0 = (int)(unit % (unsigned)tiles) * R8, b = (int)(head / a.H);
    const int stride = 16 * kUnitWarps * ctas;
    int key = 16 * (rank * kUnitWarps + warp);
    __syncthreads();
    ptx::grid_dep_wait();
    const Guard guard{abort, a.status, kWaitLimitNs};
    typename C::R w(smem + warp * C::R::RING, bars + warp * C::STAGES);
    if (key < a.C) w.load(maps, head, key);     // along with the length: what lies behind it is masked or dropped
    const int length = length_of(a.lengths, b, T, a.C), valid = length + T;
    w.load_q(a, head, b, r0);
    int ahead = key + stride;
    auto ask = [&] {
        if (ahead < valid) w.load(maps, head, ahead);
        ahead += stride;
    };
#pragma unroll
    for (int i = 1; i < C::STAGES; ++i) ask();
    const float to_log2 = a.scale * kLog2e;
    w.clear();
    for (; key < valid; key += stride) {
        w.scores(guard);
        w.step(a, head, r0, key, length, to_log2, kept);
        ask();
    }
    w.finish();
    __syncthreads();                 // every ring is empty
    w.leave(&left.o[warp][0][0], left.ml[warp]);
    __syncthreads();
    constexpr int PER = D / 8;
    for (int i = threadIdx.x; i < R8 * PER; i += 32 * kUnitWarps) {
        const int r = i / PER, c = i % PER * 8;
        float o[8];
        const float2 ml = gather(left, r, c, o);
        if (ctas == 1) {
            if (r0 + r >= R) continue;
            const long long at = head * R + r0 + r;
            write_o8(a, at, c, o, inverse_of(ml.y));
            if (c == 0) a.lse[at] = lse_of(ml.x, ml.y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4 *>(&sm.o[r][c + e]) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            if (c == 0) sm.ml[r] = ml;
        }
    }
    if (ctas == 1) return;
    __syncwarp();
    ptx::cluster_sync();
    // each CTA finishes its share of the rows' pieces of four columns
    constexpr int QUADS = D / 4, ALL = R8 * QUADS;
    const int share = (ALL + ctas - 1) / ctas;
    for (int i = rank * share + threadIdx.x; i < min((rank + 1) * share, ALL); i += 32 * kUnitWarps) {
        const int r = i / QUADS, c = i % QUADS * 4;
        if (r0 + r >= R) break;
        float2 ml[8];
        float4 o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < ctas) {
                const uint2 x = ptx::ld_cluster_b64(ptx::cluster_addr(ptx::smem_u32(&sm.ml[r]), (uint32_t)k));
                ml[k] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
                o[k] = ptx::ld_cluster_f32x4(ptx::cluster_addr(ptx::smem_u32(&sm.o[r][c]), (uint32_t)k));
            }
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < ctas) top = fmaxf(top, ml[k].x);
        const float base = top == -INFINITY ? 0.f : top;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < ctas) {
                const float f = ptx::ex2(ml[k].x - base);
                sum += f * ml[k].y;
                v.x += f * o[k].x;
                v.y += f * o[k].y;
                v.z += f * o[k].z;
                v.w += f * o[k].w;
            }
        const long long at = head * R + r0 + r;
        const float inv = inverse_of(sum);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + c) =
            make_uint2(ptx::pack_bf16x2(v.x * inv, v.y * inv), ptx::pack_bf16x2(v.z * inv, v.w * inv));
        if (c == 0) a.lse[at] = lse_of(top, sum);
    }
    __syncwarp();                      // (a warp arrives as one)
    ptx::cluster_sync_relaxed();       // nobody leaves while its sums are read
}

// ------------------------------------------------------------------------------------------
// many_kernel: more than 16 rows a cached head, on tcgen05.  One CTA an SM with two streams that alternate on the
// tensor core, so that one's softmax overlaps the other's products.  Up to 128 rows (MODE 1) both streams have the
// same rows, and every other tile of 128 slots each, with maxima, sums and O of their own that meet at the end; up
// to 256 (MODE 2) each has 128 rows, over the same tiles, so that K and V are still read once.
//   warps 0-7   softmax: stream warp / 4, thread = row (= TMEM lane): S from TMEM, running maximum (moved when a tile
//               raises it by more than kTau) and sum, P back over S, O rescaled where the maximum moved.
//   warp 8      TMA: Q, then K and V tiles through one ring, in the order in which the products take them.
//   warp 9      tcgen05: per job (a stream's tile) O += P V, then S of the stream's next job.
//   warps 10-11 the tiles that end behind the cache: V's rows behind the last token are zeroed, and what is not
//               finite among the tokens' own (0 times it would be NaN in rows that do not see it; the rows that do
//               get it when O is written).
// P is bf16, as V is (the operands of a product share their type): up to 2^-8 of each weight, 2.3e-3 of o's norm off where
// o's own rounding is 1.7e-3.  A second term for the rest, as with few rows, costs 128 rows 9 to 25 % and 256 rows 25 to
// 35 % (64000 slots of 16 cached heads 112 -> 152 us), since the softmax's chain and the products set the pace here:
// 5.8 TB/s are drawn at 256 rows, 6.4 at 128.  TMEM columns: S_0, S_1, O_0, O_1.
constexpr int kManyTile = 128;
constexpr float kTau = 8.0f;

template <int D, int MODE>
struct ManyCfg {
    static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = kManyTile * D * 2;
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int SMEM = MODE * Q_BYTES + STAGES * KV_BYTES + 1024;
    static_assert(SMEM <= 227 * 1024 - 1280 - (MODE == 1 ? 2048 : 0), "dynamic + static shared memory over 227 KB");
    static constexpr int TMA_WARP = 8, MMA_WARP = 9, FIX_WARP = 10, THREADS = 384;
    static constexpr uint32_t TM_O = 256;
};

struct ManyMaps {
    CUtensorMap q, k, v;      // [B H][G T][d] in boxes of 128 rows, [B H][C][d] in tiles; 64 columns each
};

// Places of tile j's K and V among the n tiles' loads of a segment.
template <int MODE>
__device__ __forceinline__ int k_place(int j) { return MODE == 1 ? (j == 0 ? 0 : 2 * j - 1) : 2 * j; }
template <int MODE>
__device__ __forceinline__ int v_place(int j, int n) { return MODE == 1 ? (j == n - 1 ? 2 * n - 1 : 2 * j + 2) : 2 * j + 1; }

template <int D, int MODE>
__global__ void __launch_bounds__(384, 1)
    many_kernel(const __grid_constant__ ManyMaps maps, const __grid_constant__ CacheAttnArgs a, Plan plan, Parts parts)
{
    using C = ManyCfg<D, MODE>;
    constexpr int ROWS = MODE * 128, NS = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sQ = align1024(smem_raw);
    uint8_t *sKV = sQ + MODE * C::Q_BYTES;
    __shared__ uint64_t bar_q, bar_qe, bar_full[NS], bar_empty[NS], bar_s[2], bar_p[2], bar_o[2], bar_go, bar_fix, bar_done;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh, odd_sh[4];
    __shared__ Walk walk_sh[8];
    __shared__ Segment seg_sh[8];
    __shared__ float2 ml_sh[MODE == 1 ? 2 : 1][MODE == 1 ? 128 : 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Guard g{&abort_sh, a.status, kWaitLimitNs};
    if (threadIdx.x == 0) {
        abort_sh = 0;
        ptx::mbar_init(&bar_q, 1);
        ptx::mbar_init(&bar_qe, 1);
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(&bar_full[s], 1);
            ptx::mbar_init(&bar_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(&bar_s[t], 1);
            ptx::mbar_init(&bar_p[t], 128);
            ptx::mbar_init(&bar_o[t], 1);
        }
        ptx::mbar_init(&bar_go, 1);
        ptx::mbar_init(&bar_fix, 64);
        ptx::mbar_init(&bar_done, 1);
        ptx::fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        ptx::tmem_alloc(&tmem_sh, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh;
    if (threadIdx.x == 32 * C::TMA_WARP) {
        ptx::tma_prefetch_desc(&maps.q);
        ptx::tma_prefetch_desc(&maps.k);
        ptx::tma_prefetch_desc(&maps.v);
    }
    ptx::grid_dep_launch();      // (not before tensor memory is this kernel's)
    ptx::grid_dep_wait();

    Walk walk;
    Segment seg;
    const bool any = walk.begin(a.lengths, a.B, plan);
    const int T = a.T, R = a.G * T;
    if (!any) {
        // nothing to do: the same for the whole CTA
    } else if (warp == C::TMA_WARP) {
        // ---------------------------------------------------------------- TMA producer
        if (ptx::elect_one()) {
            uint32_t seq = 0;
            uint32_t segs = 0;       // whose Q was asked for
            bool ok = true;          // nothing more is asked for once a wait has given up
            for (uint32_t i = 0; ok && walk.next(a.lengths, plan, seg); ++i) {
                if (i > 0 && !(ok = wait_bounded(&bar_qe, (i - 1) & 1, g))) break;
                ptx::mbar_arrive_expect_tx(&bar_q, MODE * C::Q_BYTES);
                for (int t = 0; t < MODE; ++t)
                    for (int hf = 0; hf < D / 64; ++hf)
                        ptx::tma_load_3d(sQ + t * C::Q_BYTES + hf * 128 * 128, &maps.q, &bar_q, hf * 64,
                                         seg.tile * ROWS + t * 128, (int)seg.head);
                segs = i + 1;
                const int n = seg.last - seg.first;
                auto load = [&](const CUtensorMap *map, int j) {
                    const uint32_t st = seq % NS;
                    if (!ok || !(ok = wait_bounded(&bar_empty[st], ((seq / NS) & 1) ^ 1, g))) return;
                    ptx::mbar_arrive_expect_tx(&bar_full[st], C::KV_BYTES);
                    for (int hf = 0; hf < D / 64; ++hf)
                        ptx::tma_load_3d(sKV + st * C::KV_BYTES + hf * kManyTile * 128, map, &bar_full[st], hf * 64,
                                         (seg.first + j) * kManyTile, (int)seg.head);
                    ++seq;
                };
                load(&maps.k, 0);
                for (int j = 0; j < n; ++j) {      // in the order of k_place() and v_place()
                    if (MODE == 1 && j + 1 < n) load(&maps.k, j + 1);
                    load(&maps.v, j);
                    if (MODE == 2 && j + 1 < n) load(&maps.k, j + 1);
                }
            }
            // do not leave with copies in flight (matters only after a timeout)
            if (segs > 0) drain(&bar_q, (segs - 1) & 1);
            for (uint32_t x = seq > (uint32_t)NS ? seq - NS : 0; x < seq; ++x) drain(&bar_full[x % NS], (x / NS) & 1);
        }
    } else if (warp == C::MMA_WARP) {
        // ---------------------------------------------------------------- tensor core issuer
        if (ptx::elect_one()) {
            const uint32_t idS = ptx::idesc_bf16_f32(128, kManyTile, false, false);
            const uint32_t idO = ptx::idesc_bf16_f32(128, D, false, true);
            const uint32_t q_base = ptx::smem_u32(sQ), kv_base = ptx::smem_u32(sKV);
            uint32_t base = 0, jobs[2] = {0, 0}, fixes = 0;
            bool ok = true;          // no product is issued once a wait has given up
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && wait_bounded(bar, parity, g);
                ptx::tc_fence_after();
                return ok;
            };
            for (uint32_t i_seg = 0; ok && walk.next(a.lengths, plan, seg); ++i_seg) {
                const int n = seg.last - seg.first, J = MODE == 1 ? n : 2 * n;
                // Every load is waited for here, in the order of the loads: a wait by parity must not skip a phase.
                auto issue_s = [&](int i) {
                    const int t = i & 1, j = MODE == 1 ? i : i >> 1;
                    const uint32_t at = base + k_place<MODE>(j), st = at % NS;
                    if ((MODE == 1 || t == 0) && !wait(&bar_full[st], (at / NS) & 1)) return;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
                        ptx::mma_ss(tmem + t * 128,
                                    ptx::sdesc_sw128(q_base + (MODE == 2 ? t * C::Q_BYTES : 0) + off, 16, 1024),
                                    ptx::sdesc_sw128(kv_base + st * C::KV_BYTES + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(&bar_s[t]);
                    if (MODE == 1 || t == 1) ptx::mma_commit(&bar_empty[st]);
                    if (i == J - 1) ptx::mma_commit(&bar_qe);
                };
                if (!wait(&bar_q, i_seg & 1)) break;
                for (int i = 0; i < 2 && i < J && ok; ++i) issue_s(i);
                bool tail = false;           // this tile is being repaired meanwhile
                for (int i = 0; i < J && ok; ++i) {
                    const int t = i & 1, j = MODE == 1 ? i : i >> 1;
                    const uint32_t at = base + v_place<MODE>(j, n), st = at % NS;
                    if (MODE == 1 || t == 0) {
                        if (!wait(&bar_full[st], (at / NS) & 1)) break;
                        tail = (seg.first + j + 1) * kManyTile > seg.length;
                        if (tail) ptx::mbar_arrive(&bar_go);
                    }
                    if (!wait(&bar_p[t], jobs[t]++ & 1)) break;
                    if (tail && (MODE == 1 || t == 0) && !wait(&bar_fix, fixes++ & 1)) break;
#pragma unroll
                    for (int kk = 0; kk < kManyTile / 16; ++kk)
                        ptx::mma_ts(tmem + C::TM_O + t * D, tmem + t * 128 + kk * 8,
                                    ptx::sdesc_sw128(kv_base + st * C::KV_BYTES + kk * 2048, kManyTile * 128, 1024), idO,
                                    i >= 2 || kk > 0 ? 1u : 0u);
                    if (MODE == 1 || t == 1) ptx::mma_commit(&bar_empty[st]);
                    if (i + 2 < J) issue_s(i + 2);
                    else ptx::mma_commit(&bar_o[t]);
                }
                if (J == 1 && ok) ptx::mma_commit(&bar_o[1]);
                base += 2 * n;
            }
            // every product is done before shared and tensor memory are given back (matters after a timeout)
            ptx::mma_commit(&bar_done);
            drain(&bar_done, 0);
        }
    } else if (warp >= C::FIX_WARP) {
        // ---------------------------------------------------------------- V's last rows
        const int ft = (warp - C::FIX_WARP) * 32 + lane;
        uint32_t base = 0, fixes = 0;
        for (uint32_t i_seg = 0; walk.next(a.lengths, plan, seg); ++i_seg) {
            const int n = seg.last - seg.first;
            bool begun = false;
            for (int j = max(0, seg.length / kManyTile - seg.first); j < n; ++j) {
                const int k0 = (seg.first + j) * kManyTile;
                const uint32_t at = base + v_place<MODE>(j, n), st = at % NS;
                if (!begun) {
                    if (ft == 0) odd_sh[i_seg & 3] = 0;
                    ptx::named_bar(1, 64);
                    begun = true;
                }
                wait_bounded(&bar_go, fixes++ & 1, g);     // the tile has landed (the issuer saw it)
                const uint32_t v = ptx::smem_u32(sKV + st * C::KV_BYTES);
                const int own = max(seg.length - k0, 0), behind = min(seg.length + T - k0, kManyTile);
                bool odd = false;
                for (int hf = 0; hf < D / 64; ++hf) {                  // 8 chunks a row of each half
                    const uint32_t half = v + hf * kManyTile * 128;
#pragma unroll 4
                    for (int c = own * 8 + ft; c < behind * 8; c += 64) {
                        uint4 w = lds_u128(half + c * 16);
                        if (any_odd(w)) {
                            odd = true;
                            drop_odd(w);
                            sts_u128(half + c * 16, w);
                        }
                    }
                    for (int c = behind * 8 + ft; c < kManyTile * 8; c += 64) sts_u128(half + c * 16, make_uint4(0, 0, 0, 0));
                }
                if (odd) odd_sh[i_seg & 3] = 1;
                __threadfence_block();
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&bar_fix);
            }
            base += 2 * n;
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int t = warp >> 2, quarter = warp & 3, r_tile = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + C::TM_O;
        const float scale_log2 = a.scale * kLog2e;
        uint32_t jobs = 0;
        // the walk and the segment wait in shared memory: S takes the registers
        const Segment &seg = seg_sh[warp];
        if (lane == 0) walk_sh[warp] = walk;
        for (uint32_t i_seg = 0;; ++i_seg) {
            __syncwarp();
            if (lane == 0) walk_sh[warp].next(a.lengths, plan, seg_sh[warp]);
            __syncwarp();
            if (!seg.there) break;
            const int n = seg.last - seg.first;
            const int row = seg.tile * ROWS + (MODE == 2 ? t * 128 : 0) + r_tile;
            const bool idle = row - lane >= R;          // a warp without rows
            uint64_t word = row < R ? word_of(a.tree, seg.b, T, row % T) : 0;    // (the last tile needs it at once)
            if (T < 64) word &= (1ull << T) - 1;
            float m = -INFINITY, l = 0.f;
            bool begun = false;
            for (int j = MODE == 1 ? t : 0; j < n; j += MODE == 1 ? 2 : 1, ++jobs) {
                wait_bounded(&bar_s[t], jobs & 1, g);
                ptx::tc_fence_after();
                if (!idle) {
                    uint32_t r[128];
                    ptx::tmem_ld32_at<0>(tS + 0, r);
                    ptx::tmem_ld32_at<32>(tS + 32, r);
                    ptx::tmem_ld32_at<64>(tS + 64, r);
                    ptx::tmem_ld32_at<96>(tS + 96, r);
                    ptx::tmem_ld_wait();
                    reg_fence(r);
                    const int u0 = (seg.first + j) * kManyTile - seg.length;    // the tile's first slot, from the first token's
                    if (u0 + kManyTile > 0) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int u = u0 + 32 * c;
                            uint32_t bits;
                            if (u >= 64) bits = 0;
                            else if (u >= 0) bits = (uint32_t)(word >> u);
                            else if (u > -32) bits = (uint32_t)(word << -u) | ((1u << -u) - 1);
                            else bits = 0xffffffffu;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(bits >> i & 1)) r[32 * c + i] = __float_as_uint(-INFINITY);
                        }
                    }
                    float mx[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) mx[u] = __uint_as_float(r[u]);
#pragma unroll
                    for (int i = 8; i < 128; i += 2)
                        mx[(i >> 1) & 7] = ptx::max3(mx[(i >> 1) & 7], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                    const float smax = ptx::max3(ptx::max3(mx[0], mx[1], mx[2]), ptx::max3(mx[3], mx[4], mx[5]),
                                                 fmaxf(mx[6], mx[7]));
                    const float mt = smax * scale_log2;
                    float m_new = m, alpha = 1.f;
                    bool rescale = false;
                    if (!begun) {
                        m_new = mt;
                    } else if (__any_sync(0xffffffffu, mt > m + kTau)) {
                        m_new = fmaxf(m, mt);
                        alpha = m_new == -INFINITY ? 1.f : ptx::ex2(m - m_new);
                        rescale = true;
                    }
                    begun = true;
                    const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
                    const uint64_t c2 = ptx::f2_pack(scale_log2, scale_log2), nm2 = ptx::f2_pack(neg_m, neg_m);
                    uint64_t sum2[2] = {ptx::f2_pack(0.f, 0.f), ptx::f2_pack(0.f, 0.f)};
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const uint64_t x = ptx::fma_f32x2(
                                ptx::f2_pack(__uint_as_float(r[ch * 32 + i]), __uint_as_float(r[ch * 32 + i + 1])), c2, nm2);
                            float t0, t1;
                            ptx::f2_unpack(x, t0, t1);
                            const float p0 = ptx::ex2(t0), p1 = ptx::ex2(t1);
                            sum2[(i >> 1) & 1] = ptx::add_f32x2(sum2[(i >> 1) & 1], ptx::f2_pack(p0, p1));
                            pk[i >> 1] = ptx::pack_bf16x2(p0, p1);
                        }
                        ptx::tmem_st16(tS + ch * 16, pk);
                    }
                    float sum[4];
                    ptx::f2_unpack(sum2[0], sum[0], sum[1]);
                    ptx::f2_unpack(sum2[1], sum[2], sum[3]);
                    l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
                    m = m_new;
                    if (rescale) {
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t ov[32];
                            ptx::tmem_ld32(tO + t * D + c, ov);
                            ptx::tmem_ld_wait();
                            reg_fence(ov);
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            ptx::tmem_st32(tO + t * D + c, ov);
                        }
                    }
                    ptx::tmem_st_wait();
                }
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bar_p[t]);
            }

            // The rows' results: both streams' (MODE 1, each warp half of the columns) or their own.
            float f[2] = {1.f, 0.f};
            if (MODE == 1) {
                ml_sh[t][r_tile] = make_float2(m, l);
                ptx::named_bar(2, 256);
                const float2 other = ml_sh[t ^ 1][r_tile];
                const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
                const float mine = ptx::ex2(m - ref), its = ptx::ex2(other.x - ref);
                f[0] = t == 0 ? mine : its;
                f[1] = t == 0 ? its : mine;
                l = t == 0 ? l * mine + other.y * its : other.y * its + l * mine;
                m = top;
            }
            wait_bounded(&bar_o[t], i_seg & 1, g);
            if (MODE == 1) wait_bounded(&bar_o[t ^ 1], i_seg & 1, g);
            ptx::tc_fence_after();
            const bool whole = seg.whole();
            const bool tail = seg.last * kManyTile > seg.length;
            const bool odd = tail && odd_sh[i_seg & 3];
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long at = seg.head * R + row;
            const long long slot = 2 * (long long)blockIdx.x + (seg.first == 0 ? 1 : 0);
            constexpr int COLS = MODE == 1 ? D / 2 : D;
            if (!idle) {
#pragma unroll
                for (int c0 = 0; c0 < COLS; c0 += 32) {
                    const int c = MODE == 1 ? t * COLS + c0 : c0;
                    uint32_t ov[32];
                    ptx::tmem_ld32(tO + (MODE == 1 ? 0 : t * D) + c, ov);
                    ptx::tmem_ld_wait();
                    reg_fence(ov);
                    if (MODE == 1) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(f[0] * __uint_as_float(ov[i]));
                        if (n > 1) {             // (with one tile the second stream has no O)
                            uint32_t o2[32];
                            ptx::tmem_ld32(tO + D + c, o2);
                            ptx::tmem_ld_wait();
                            reg_fence(o2);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                ov[i] = __float_as_uint(__uint_as_float(ov[i]) + f[1] * __uint_as_float(o2[i]));
                        }
                    }
                    if (odd && row < R) {
                        for (int u = 0; u < T; ++u) {
                            const int key = seg.length + u;
                            if (!(word >> u & 1) || key < seg.first * kManyTile || key >= seg.last * kManyTile) continue;
                            const uint4 *from = static_cast<const uint4 *>(a.v) + (seg.head * a.C + key) * (D / 8) + c / 8;
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint4 w = from[x];
                                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int y = 0; y < 8; ++y) {
                                    const float v = y & 1 ? hi(ws[y / 2]) : lo(ws[y / 2]);
                                    if (odd_value(v)) ov[8 * x + y] = __float_as_uint(__uint_as_float(ov[8 * x + y]) + v);
                                }
                            }
                        }
                    }
                    if (whole) {
                        // Four neighbouring lanes write 64 bytes of one row after another: their 16-byte pieces change
                        // places in two steps (a lane's own row a store would touch 32 lines a time).
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = ptx::pack_bf16x2(__uint_as_float(ov[8 * i + 2 * y]) * inv,
                                                        __uint_as_float(ov[8 * i + 2 * y + 1]) * inv);
                            x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        exchange(x[0], x[1], 1);
                        exchange(x[2], x[3], 1);
                        exchange(x[0], x[2], 2);
                        exchange(x[1], x[3], 2);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = row - (lane & 3) + i;
                            if (r < R)
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + (seg.head * R + r) * D + c +
                                                           8 * (lane & 3)) = x[i];
                        }
                    } else if (row < R) {
                        uint4 *dst = reinterpret_cast<uint4 *>(parts.o) + (slot * (D / 4) + c / 4) * ROWS + row % ROWS;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x * ROWS] = make_uint4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
                    }
                }
                if (row < R && (MODE == 2 || t == 0)) {
                    if (whole) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
                    else parts.ml[slot * ROWS + row % ROWS] = make_float2(m, l);
                }
            }
            ptx::tc_fence_before();
            if (MODE == 1) ptx::named_bar(2, 256);     // both streams' O has been read
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Adds up the parts of a unit that was split, each with its maximum and sum, in the order of their slots.
struct Sum {
    float top = -INFINITY, l = 0.f;
    // Takes a part in: the factors of what is there and of the part.
    __device__ __forceinline__ void take(float2 ml, float &old, float &part)
    {
        const float t = fmaxf(top, ml.x), ref = t == -INFINITY ? 0.f : t;
        old = ptx::ex2(top - ref);
        part = ptx::ex2(ml.x - ref);
        l = l * old + ml.y * part;
        top = t;
    }
    __device__ __forceinline__ float inverse() const { return inverse_of(l); }
    __device__ __forceinline__ float lse() const { return lse_of(top, l); }
};

// Where a unit's parts are.  By a whole warp.
struct Pieces {
    long long c0;
    int count;
    __device__ __forceinline__ Pieces(const CacheAttnArgs &a, const Plan &plan, int ctas, int b, int h, int tile)
    {
        long long before, per;
        if (a.B <= 32) {
            const int l = threadIdx.x & 31, n = l < a.B ? blocks_of(length_of(a.lengths, l, a.T, a.C), plan) : 0;
            const Shares sh = shares_of(n, plan, ctas);
            per = sh.per;
            if (sh.apart) {
                const int mine = (n + (int)per - 1) / (int)per;
                count = __shfl_sync(0xffffffffu, mine, b);
                c0 = (long long)__reduce_add_sync(0xffffffffu, l < b ? mine : 0) * plan.H * plan.tiles +
                     ((long long)h * plan.tiles + tile) * count;
                return;
            }
            before = (long long)__reduce_add_sync(0xffffffffu, l < b ? n : 0) * plan.H * plan.tiles;
        } else {
            per = divide(count_blocks(a.lengths, a.B, b, plan, before) + ctas - 1, ctas);
        }
        const int nb = blocks_of(length_of(a.lengths, b, a.T, a.C), plan);
        const long long u0 = before + ((long long)h * plan.tiles + tile) * nb;
        if (per <= 0x7fffffff) {
            c0 = divide(u0, (int)per);
            count = (int)(divide(u0 + nb - 1, (int)per) - c0) + 1;
        } else {
            c0 = u0 / per;
            count = (int)((u0 + nb - 1) / per - c0) + 1;
        }
    }
    // the first part begins the unit, the others inside it
    __device__ __forceinline__ long long slot(int i) const { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); }
};

// few_kernel's parts: a block a row, a warp every eighth part, a lane D / 32 columns.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(CacheAttnArgs a, Plan plan, int rows, int ctas, Parts parts)
{
    __shared__ float so[kJoinWarps][D];
    __shared__ float2 sml[kJoinWarps];
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = a.G * a.T;
    const int head = (int)(blockIdx.x / (unsigned)R), r = (int)(blockIdx.x % (unsigned)R);
    const int b = head / plan.H, h = head % plan.H;
    ptx::grid_dep_wait();
    const Pieces pieces(a, plan, ctas, b, h, r / rows);
    if (pieces.count == 1) return;
    constexpr int PER = D / 32;
    Sum sum;
    float o[PER] = {};
#pragma unroll 4
    for (int i = warp; i < pieces.count; i += kJoinWarps) {
        const long long at = pieces.slot(i) * rows + r % rows;
        const float2 ml = parts.ml[at];
        const float *from = parts.o + at * D + lane * PER;
        float v[PER], f, p;
        if (PER == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(from);
        else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(from);
        sum.take(ml, f, p);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = o[e] * f + v[e] * p;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = o[e];
    if (lane == 0) sml[warp] = make_float2(sum.top, sum.l);
    __syncthreads();
    if (warp > 0) return;
    Sum all;
    float v[PER] = {};
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        float f, p;
        all.take(sml[w], f, p);
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = v[e] * f + so[w][lane * PER + e] * p;
    }
    const float inv = all.inverse();
    uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.o) + (long long)blockIdx.x * D + lane * PER);
#pragma unroll
    for (int e = 0; e < PER; e += 2) to[e / 2] = ptx::pack_bf16x2(v[e] * inv, v[e + 1] * inv);
    if (lane == 0) a.lse[blockIdx.x] = all.lse();
}

// many_kernel's parts: a block 32 rows and, `sweep` times, 32 / GROUPS columns of them, a warp four columns and every
// GROUPS-th part, six at once.
constexpr int kJoinAtOnce = 6;
constexpr unsigned kJoinBlocks = 4 * 152;    // 4 an SM

template <int D, int GROUPS>
__global__ void __launch_bounds__(256, 4) join_many_kernel(CacheAttnArgs a, Plan plan, int rows, int ctas, Parts parts,
                                                           int sweep)
{
    constexpr int QUADS = 8 / GROUPS;
    __shared__ float4 so[GROUPS][QUADS][32];
    __shared__ float2 sml[GROUPS][32];
    __shared__ uint2 out[32][QUADS + 1];
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp % QUADS, share = warp / QUADS;
    const unsigned groups = rows / 32, sweeps = D / (4 * QUADS) / sweep;
    const int first = (int)(blockIdx.x % sweeps) * sweep * 4 * QUADS, group = (int)(blockIdx.x / sweeps % groups);
    const unsigned unit = blockIdx.x / (sweeps * groups);
    const int tile = (int)(unit % (unsigned)plan.tiles), head = (int)(unit / (unsigned)plan.tiles);
    const int b = head / plan.H, h = head % plan.H, R = a.G * a.T;
    const int r0 = tile * rows + group * 32, r = group * 32 + lane;
    ptx::grid_dep_wait();
    if (r0 >= R) return;
    const Pieces pieces(a, plan, ctas, b, h, tile);
    if (pieces.count == 1) return;
    for (int col = first; col < first + sweep * 4 * QUADS; col += 4 * QUADS) {
        Sum sum;
        float o[4] = {};
        auto take = [&](float2 ml, float4 v) {
            float f, p;
            sum.take(ml, f, p);
            o[0] = o[0] * f + v.x * p;
            o[1] = o[1] * f + v.y * p;
            o[2] = o[2] * f + v.z * p;
            o[3] = o[3] * f + v.w * p;
        };
        for (int i0 = share; i0 < pieces.count; i0 += GROUPS * kJoinAtOnce) {  // (a part that is not there changes nothing)
            float2 ml[kJoinAtOnce];
            float4 v[kJoinAtOnce];
#pragma unroll
            for (int e = 0; e < kJoinAtOnce; ++e) {
                const int i = i0 + GROUPS * e;
                const long long slot = pieces.slot(i);
                const bool there = i < pieces.count;
                ml[e] = there ? parts.ml[slot * rows + r] : make_float2(-INFINITY, 0.f);
                v[e] = there ? reinterpret_cast<const float4 *>(parts.o)[(slot * (D / 4) + col / 4 + quad) * rows + r]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int e = 0; e < kJoinAtOnce; ++e) take(ml[e], v[e]);
        }
        if (GROUPS > 1) {
            so[share][quad][lane] = make_float4(o[0], o[1], o[2], o[3]);
            if (quad == 0) sml[share][lane] = make_float2(sum.top, sum.l);
            __syncthreads();
            if (share == 0) {
#pragma unroll
                for (int g = 1; g < GROUPS; ++g) take(sml[g][lane], so[g][quad][lane]);
            }
        }
        if (share == 0) {
            const float inv = sum.inverse();
            out[lane][quad] =
                make_uint2(ptx::pack_bf16x2(o[0] * inv, o[1] * inv), ptx::pack_bf16x2(o[2] * inv, o[3] * inv));
            if (col == 0 && quad == 0 && r0 + lane < R) a.lse[(long long)head * R + r0 + lane] = sum.lse();
        }
        __syncthreads();
        const int row = threadIdx.x / QUADS, part = threadIdx.x % QUADS;
        if (row < 32 && r0 + row < R)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + ((long long)head * R + r0 + row) * D + col +
                                       part * 4) = out[row][part];
        if (col + 4 * QUADS < first + sweep * 4 * QUADS) __syncthreads();      // `out` is used again
    }
}

// weights_out = weights + the weights that the counted rows give each slot, from the scores that were kept: four slots a
// thread, 256 apart.  At up to 16 rows the scores (4 bytes a row and slot, twice, mostly in L2) are less than K (2 d
// bytes) a second time.
constexpr int kKeptSlots = 1024;     // a block

template <int AT_ONCE>
__global__ void __launch_bounds__(256) kept_weights_kernel(const __grid_constant__ CacheAttnArgs a, int blocks,
                                                           const float *scores)
{
    __shared__ float lse[16];
    ptx::grid_dep_launch();
    const int head = (int)(blockIdx.x / (unsigned)blocks), b = head / a.H, T = a.T, R = a.G * T;
    const int j0 = (int)(blockIdx.x % (unsigned)blocks) * kKeptSlots + threadIdx.x;
    ptx::grid_dep_wait();
    const int valid = length_of(a.lengths, b, T, a.C) + T;
    const long long at = (long long)head * a.C + j0;
    const float *from = scores + (long long)head * R * a.C + j0;
    float was[4], s[AT_ONCE][4], sum[4] = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][e] = r0 + i < R && j0 + 256 * e < valid ? from[(long long)(r0 + i) * a.C + 256 * e] : -INFINITY;
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) was[e] = j0 + 256 * e < a.C ? a.weights[at + 256 * e] : 0.f;
    load(0);
    if (threadIdx.x < 16) {
        const bool counted = threadIdx.x < R && (!a.counted || (a.counted[b] >> (threadIdx.x % T) & 1));
        lse[threadIdx.x] = counted ? a.lse[(long long)head * R + threadIdx.x] * kLog2e : INFINITY;
    }
    __syncthreads();
    for (int r0 = 0;;) {
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const float x = lse[r0 + i];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x != INFINITY && s[i][e] != -INFINITY) sum[e] += ptx::ex2(s[i][e] - x);
        }
        if ((r0 += AT_ONCE) >= R) break;
        load(r0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = j0 + 256 * e;
        if (j < valid || (j < a.C && a.weights_out != a.weights)) a.weights_out[at + 256 * e] = was[e] + sum[e];
    }
}

// The same for more rows: K is read a second time, the rows in eights.  A block takes 128 slots of one (sequence,
// cached head).  Bound by latency: each warp loads Q and lse again for its 16 slots (4 trees of 64 over 16384 slots of 4 cached
// heads of 256 rows 252-259 us, tensor pipe 11 %, L2 2 %; K alone is 64 MB, 9.5 us).
template <int D>
__global__ void __launch_bounds__(kFewThreads) weights_kernel(CacheAttnArgs a, int blocks)
{
    constexpr int KC = D / 32;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const long long head = blockIdx.x / blocks;
    const int b = (int)(head / a.H), T = a.T, R = a.G * T;
    const int key = (int)(blockIdx.x % blocks) * kBlock + 16 * warp;
    const int length = length_of(a.lengths, b, T, a.C), valid = length + T;
    float sum[2] = {0.f, 0.f};
    if (key < valid) {
        const uint64_t counted = a.counted ? a.counted[b] : ~0ull;
        const uint4 *kp = static_cast<const uint4 *>(a.k) + head * a.C * (D / 8);
        uint4 kr[2][KC];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int j = key + g + 8 * i;
                kr[i][c] = j < valid ? stream16(kp + (long long)j * (D / 8) + 4 * c + q) : make_uint4(0, 0, 0, 0);
            }
        const bool tail = key + 16 > length;
        for (int r0 = 0; r0 < R; r0 += 8) {
            const int r = r0 + g;
            const uint4 *qp = static_cast<const uint4 *>(a.q) + (head * R + r) * (D / 8);
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 qf = r < R ? qp[4 * c + q] : make_uint4(0, 0, 0, 0);
                const uint32_t a0[4] = {kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y};
                const uint32_t a1[4] = {kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w};
                mma16816(s, a0, qf.x, qf.y);
                mma16816(s, a1, qf.z, qf.w);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r0 + 2 * q + e, t = row % T;
                if (row >= R || !(counted >> t & 1)) continue;
                const float lse = a.lse[head * R + row];
                const uint64_t word = tail ? word_of(a.tree, b, T, t) : 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = key + g + 8 * i - length;
                    if (j >= 0 && !(j < T && (word >> j & 1))) continue;
                    sum[i] += ptx::ex2((s[e + 2 * i] * a.scale - lse) * kLog2e);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        const int j = key + g + 8 * i;
        if (q == 0 && j < a.C) {
            const long long at = head * a.C + j;
            if (j < valid) a.weights_out[at] = a.weights[at] + sum[i];
            else if (a.weights_out != a.weights) a.weights_out[at] = a.weights[at];
        }
    }
}

constexpr int kPlanSms = 152;    // the split is a function of the sizes and lengths alone
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Which kernels a call runs, a function of the sizes alone.
enum Kind { kUnit = 1, kFew = 2, kManyWhole = 3, kMany = 4 };
struct Choice {
    Kind kind;
    int rows;        // of a unit
    int ctas;        // kUnit: of a cluster; kFew, kMany: that share the work
    bool few_rows() const { return rows <= 16; }
    bool parts() const { return kind == kFew || kind == kMany; }
};

// Shares of a row's parts in join_many_kernel that has `blocks` blocks without: see launch().
int join_groups(long long blocks)
{
    int groups = 1;
    while (groups < 8 && blocks * groups * 2 <= kJoinBlocks) groups *= 2;
    return groups;
}

long long units_of(int B, int H, int R, int rows) { return (long long)B * H * ((R + rows - 1) / rows); }

// Time in us of CTAs that take up to `steps` steps each, `wave` of them at a time, where a step takes a CTA `step` at
// least and the CTAs on the GPU together `hbm` each.
double waves(long long ctas, long long wave, double steps, double step, double hbm)
{
    auto run = [&](long long active) { return steps * (active * hbm > step ? active * hbm : step) + 2.6; };
    const double t = (double)(ctas / wave) * run(wave) + (ctas % wave ? run(ctas % wave) : 0.0);
    return (ctas > wave ? 0.92 * t : t) - 2.6;
}

// Steps of `slots` each: the mean of a full cache's and of one full to nine tenths (few sequences end at the last slot).
double steps_of(int C, int slots)
{
    const long long c = C, s = slots;
    return 0.5 * (double)((c + s - 1) / s + (c * 9 / 10 + s - 1) / s);
}

// Clusters of 1 to 8 CTAs of unit_kernel that the GPU holds at once (as CUDA's occupancy call says; one CTA an SM at
// d = 128, two at 64).
constexpr short kClusters[2][8] = {{304, 152, 97, 74, 58, 46, 38, 36}, {152, 76, 46, 36, 28, 23, 15, 15}};

// The least estimated time.  The constants (us; a step is 128 slots) were fitted to the times of every choice at 2000
// sizes drawn from 1 to 512 sequences and heads, 1 to 512 rows and 16 to 65536 slots, with lengths that differ by up to
// all of them: what is chosen takes 0.8 % more on average than the best of what the rule below allows at 300 other sizes,
// 1.0 % at 1200 where up to a quarter of the room is free.  (A unit by a cluster against shares and a join: 16 units of
// 1000 and 8000 slots 5.6 and 17.8 us, 7.6 and 16.7; 128 units of 1000 and 16000 12.9 and 160, 20.7 and 161.)  Sequences
// shorter than the cache leave a long one to its cluster or CTA alone, so that it is never given more than 24 steps.
Choice choose(int B, int H, int G, int T, int C, int d)
{
    constexpr int kMostSteps = 24;
    const int R = G * T, slots128 = (C + 127) / 128;
    const bool wide = d == 128;
    const double hbm = wide ? 0.007 : 0.0036;
    Choice best = {kFew, R <= 8 ? 8 : 16, 0};
    const bool eight = best.rows == 8;
    const long long units = units_of(B, H, R, best.rows), wave = wide ? kPlanSms : 2 * kPlanSms;
    best.ctas = (eight ? wide ? FewCfg<128, 1>::BLOCKS : FewCfg<64, 1>::BLOCKS
                       : wide ? FewCfg<128, 2>::BLOCKS : FewCfg<64, 2>::BLOCKS) * kPlanSms;
    double t_best = (eight ? wide ? 9.2 : 13.0 : 12.2) + (double)units * slots128 * hbm + 5.1 * units / wave;
    if (R > 16) {
        const int rows = R <= 128 ? 128 : 256;
        const long long many = units_of(B, H, R, rows);
        // both streams of 128 rows' tiles run at once
        double tile = (rows == 256 ? 2.67 : 0.63) * (wide ? 1.0 : 0.29);
        const double pieces = (double)kPlanSms / many < slots128 ? (double)kPlanSms / many : slots128;
        double t = 10.5 + (double)many * slots128 * (tile / kPlanSms > hbm ? tile / kPlanSms : hbm) + 4.9 * many / kPlanSms +
                   0.14 * pieces / join_groups(many * (rows / 32) * (d / 32));
        if (t < t_best) {
            best = {kMany, rows, kPlanSms};
            t_best = t;
        }
        tile = (rows == 256 ? 1.35 : 0.83) * (wide ? 1.0 : 0.67);
        t = 3.2 + waves(many, kPlanSms, steps_of(C, 128), tile, hbm) + 2.7 * (double)((many + kPlanSms - 1) / kPlanSms);
        if (slots128 <= kMostSteps && t < t_best) {
            best = {kManyWhole, rows, 0};
            t_best = t;
        }
    }
    const double step = wide ? eight ? 0.68 : 0.98 : eight ? 0.6 : 0.71;
    for (int n = 1; n <= 8; ++n) {
        const int steps = (C + 128 * n - 1) / (128 * n);
        const double t =
            5.4 + (n == 1 ? 0.0 : 1.2) + waves(units * n, kClusters[wide][n - 1] * n, steps_of(C, 128 * n), step, hbm);
        if (steps <= kMostSteps && t < t_best) {
            best = {kUnit, R <= 8 ? 8 : 16, n};
            t_best = t;
        }
    }
    return best;
}

// Bytes of the parts' results.
size_t parts_bytes(const Choice &c, int d)
{
    if (!c.parts()) return 0;
    const size_t slots = (size_t)2 * c.ctas * c.rows;
    return up256(slots * d * 4) + up256(slots * 8);
}

// Scores are kept for the accumulated weights where a cached head has few rows in all.
bool keeps_scores(const Choice &c, int R) { return c.few_rows() && R <= 16; }

bool make_kv_maps(KvMaps &maps, const CacheAttnArgs &a)
{
    const long long bh = (long long)a.B * a.H;
    return make_map_3d(&maps.k, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.d, a.C, bh, 64, 16) == CUDA_SUCCESS &&
           make_map_3d(&maps.v, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.d, a.C, bh, 64, 16) == CUDA_SUCCESS;
}

template <int D, int NT>
cudaError_t launch_unit(const CacheAttnArgs &a, int tiles, int ctas, float *kept, cudaStream_t stream)
{
    static std::atomic<bool> set[64];
    constexpr int bytes = UnitCfg<D, NT>::SMEM;
    KvMaps maps;
    if (!make_kv_maps(maps, a)) return cudaErrorInvalidValue;
    const cudaError_t e = raise_smem(reinterpret_cast<const void *>(unit_kernel<D, NT>), bytes, set);
    if (e != cudaSuccess) return e;
    return launch_overlapped(unit_kernel<D, NT>, dim3((unsigned)(a.B * a.H) * tiles * ctas), dim3(32 * kUnitWarps), bytes,
                             (unsigned)ctas, stream, maps, a, tiles, kept);
}

template <int D, int NT>
cudaError_t launch_few(const CacheAttnArgs &a, const Plan &plan, const Parts &parts, int ctas, cudaStream_t stream)
{
    static std::atomic<bool> set[64];
    constexpr int bytes = FewCfg<D, NT>::SMEM;
    KvMaps maps;
    if (!make_kv_maps(maps, a)) return cudaErrorInvalidValue;
    const cudaError_t e = raise_smem(reinterpret_cast<const void *>(few_kernel<D, NT>), bytes, set);
    if (e != cudaSuccess) return e;
    return launch_overlapped(few_kernel<D, NT>, dim3((unsigned)ctas), dim3(kFewThreads), bytes, 1, stream, maps, a, plan,
                             parts);
}

template <int D, int MODE>
cudaError_t launch_many(const CacheAttnArgs &a, const Plan &plan, const Parts &parts, int ctas, cudaStream_t stream)
{
    using C = ManyCfg<D, MODE>;
    ManyMaps maps;
    const long long bh = (long long)a.B * a.H;
    if (make_map_3d(&maps.q, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, a.G * a.T, bh, 64, 128) != CUDA_SUCCESS ||
        make_map_3d(&maps.k, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, a.C, bh, 64, kManyTile) != CUDA_SUCCESS ||
        make_map_3d(&maps.v, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, a.C, bh, 64, kManyTile) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static std::atomic<bool> set[64];
    const cudaError_t e = raise_smem(reinterpret_cast<const void *>(many_kernel<D, MODE>), C::SMEM, set);
    if (e != cudaSuccess) return e;
    return launch_overlapped(many_kernel<D, MODE>, dim3((unsigned)ctas), dim3(C::THREADS), C::SMEM, 1, stream, maps, a,
                             plan, parts);
}

template <int D>
cudaError_t launch(const CacheAttnArgs &a, cudaStream_t stream)
{
    const int R = a.G * a.T;
    const Choice c = choose(a.B, a.H, a.G, a.T, a.C, D);
    const Plan plan = {a.H, (R + c.rows - 1) / c.rows, a.T, a.C, c.few_rows() ? kBlock : kManyTile, c.kind == kManyWhole,
                       c.few_rows() ? 1 : 2};
    const unsigned heads = (unsigned)a.B * (unsigned)a.H;
    char *ws = static_cast<char *>(a.workspace);
    Parts parts = {};
    if (c.parts()) {
        parts.o = reinterpret_cast<float *>(ws);
        parts.ml = reinterpret_cast<float2 *>(ws + up256((size_t)2 * c.ctas * c.rows * D * 4));
    }
    const bool kept = a.weights && keeps_scores(c, R);
    if (kept) parts.scores = reinterpret_cast<float *>(ws + parts_bytes(c, D));
    cudaError_t e;
    if (c.kind == kUnit)
        e = c.rows == 8 ? launch_unit<D, 1>(a, plan.tiles, c.ctas, parts.scores, stream)
                        : launch_unit<D, 2>(a, plan.tiles, c.ctas, parts.scores, stream);
    else if (c.kind == kFew)
        e = c.rows == 8 ? launch_few<D, 1>(a, plan, parts, c.ctas, stream) : launch_few<D, 2>(a, plan, parts, c.ctas, stream);
    else
        e = c.rows == 128 ? launch_many<D, 1>(a, plan, parts, c.kind == kMany ? c.ctas : (int)(heads * plan.tiles), stream)
                          : launch_many<D, 2>(a, plan, parts, c.kind == kMany ? c.ctas : (int)(heads * plan.tiles), stream);
    if (e != cudaSuccess) return e;
    if (c.kind == kFew)
        e = launch_overlapped(join_kernel<D>, dim3(heads * R), dim3(32 * kJoinWarps), 0, 1, stream, a, plan, c.rows, c.ctas,
                              parts);
    if (c.kind == kMany)
    {
        // About as many blocks as the GPU holds at once: more go over the columns one after another (128 units of 256
        // rows 90 -> 79 us), fewer share the parts of a row (one unit of 32000 slots 47 -> 20 us, two of 16000 33 -> 19).
        const unsigned blocks = heads * plan.tiles * (c.rows / 32) * (D / 32);
        const int groups = join_groups(blocks);
        int sweep = 1;
        while (sweep < D / 32 && blocks / sweep > kJoinBlocks) sweep *= 2;
        auto *const kernel = groups == 8   ? join_many_kernel<D, 8>
                             : groups == 4 ? join_many_kernel<D, 4>
                             : groups == 2 ? join_many_kernel<D, 2>
                                           : join_many_kernel<D, 1>;
        e = launch_overlapped(kernel, dim3(blocks / sweep * groups), dim3(256), 0, 1, stream, a, plan, c.rows, c.ctas, parts,
                              sweep);
    }
    if (e != cudaSuccess || !a.weights) return e;
    if (kept) {
        const int blocks = (a.C + kKeptSlots - 1) / kKeptSlots;
        return launch_overlapped(R == 1 ? kept_weights_kernel<1> : kept_weights_kernel<4>, dim3(heads * blocks), dim3(256), 0,
                                 1, stream, a, blocks, (const float *)parts.scores);
    }
    const int blocks = (a.C + kBlock - 1) / kBlock;
    return launch_overlapped(weights_kernel<D>, dim3(heads * blocks), dim3(kFewThreads), 0, 1, stream, a, blocks);
}

}  // namespace

size_t cache_attn_workspace(int B, int H, int G, int T, int C, int d, bool weights)
{
    const Choice c = choose(B, H, G, T, C, d);
    return parts_bytes(c, d) + (weights && keeps_scores(c, G * T) ? up256((size_t)B * H * G * T * C * 4) : 0);
}

void cache_attn_plan(int B, int H, int G, int T, int C, int d, int plan[3])
{
    const Choice c = choose(B, H, G, T, C, d);
    plan[0] = c.kind;
    plan[1] = c.rows;
    plan[2] = c.ctas;
}

cudaError_t launch_cache_attn(const CacheAttnArgs &a, cudaStream_t stream)
{
    return a.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace attn
