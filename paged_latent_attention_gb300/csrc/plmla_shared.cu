// plmla_shared.cu -- gated MLA decode of a batch whose requests share prefixes, on CTA pairs
// of the 5th-generation tensor cores (tcgen05 + TMEM), for sm_103a.
//
//   out[r, j, h] = sigmoid(gate) sum_t w_t c_t,  w = softmax_t(scale q_{r,j,h} . x_t),
//                  t < L_r - (n_q - 1 - j)
//
// The softmax over a history is the merge, by log-sum-exps, of the softmaxes over its
// parts.  The tokens that a group of requests has in common are one part, read once: the
// queries of all members are the rows of one attention problem over them (no causal limit
// falls there).  What each request has of its own is the other part.
//
// Work.  A block is 128 query rows of one part.  plan_kernel lists the parts (groups' prefixes,
// then requests' own tokens); the tiles of 128 tokens of all blocks, in order, are dealt to
// CTA pairs in equal contiguous runs, a block's start counting kStart tiles more.  A pair's
// run within a block is a segment: it leaves a partial output and its log-sum-exp, and
// merge_kernel joins a row's partials in order and applies the gate.  There are no atomics,
// and results depend on the arguments alone.
//
// A pair holds 64 rows in each CTA (cta_group::2, M = 128).  Per tile
//   S = Q K^T      K split by tokens: each CTA loads 64 of them (N = 128)
//   O += P V       V split by columns: each CTA loads its 2 x 128 of 512 (2 x N = 256)
// so every byte that enters an SM serves 128 rows.  TMEM in each CTA: O takes 256 columns (lane =
// row + 64 * half; columns of half h of each 256 in lanes 64 h ..), two score tiles 64 each.
// Measured on this device: such MMAs issue at their full rate (32 and 64 cycles) when their
// operands are warp-uniform and constant but for a base, against 110 cycles each from a
// divergent thread with computed descriptors, so the issuing warp stays converged.
//
// Warps: 0 loads K, 2 loads V (TMA, a ring of four 16 KB items each), 3 Q and K's rope block,
// 1 issues the MMAs of the pair (in the even CTA), K a tile ahead of V, 4-11 softmax and
// epilogue, a thread having a quarter of a row's 128 scores in registers.  The running maximum
// lags: O is only rescaled when a score exceeds it by 2^8 (2^4 for E4M3).  E4M3 pages: queries
// in two E4M3 parts (as in the FP8 decode) and the probabilities in two as well, E4M3 and the
// rest as E5M2 (the MMA takes the types of A and B apart); both parts together take the time that
// bf16 would.  Together they carry 8 bits like bf16 ones down to 2^-6, and steps of 2^-14 and less
// below, so there the reference follows the history down too: once a row's largest in a tile
// falls 2^6 below it, O is scaled up.  A weight is off by 2^-8 of itself, or 2^-12 of the largest of its
// tile.  (Two E4M3 parts under a reference that only rises lose what is below 2^-14 of the row's
// largest weight: a third of the output behind a token that takes 0.62 of the weight.  This
// costs 0.7% of the 4-draft case below, 3% with scores four times as large.)
//
// Measured (over several boxes): 64 requests x 64 heads over 32,768 shared and 300-4,000 own tokens,
// bf16: 194-207 us, the decode kernel 188 of 200, 1.66 PFLOP/s (87% of a library product's burst,
// tensor pipe busy 79% of the time; each SM takes in 139 KB a tile, at 80% of what the L2 gives
// it).  4-draft verification over 48 E4M3 histories, whose prefixes nothing is saved by sharing:
// 144-151 us, the decode 125.  8 answers to 20,011 tokens: 32-36 us, 2 requests of 1,500: 14.6-15.6 us,
// both latency: three launches, a block's start, a partial's way out and back.
// Against the plain decode, which reads a prefix once per request: 64 requests of 66,048 + 2,000
// tokens 360 us, not 684.
//
// Every mbarrier wait is bounded (the odd CTA's for the last commit from when its other warps are
// through); one that gives up sets the status word, and cluster barriers keep both CTAs until
// neither can touch the other.
#include <math.h>

#include <atomic>

#include "plmla_ptx.cuh"
#include "plmla_quantize.cuh"

namespace plmla {
namespace {

constexpr int kShThreads = 384;
constexpr int kShSlots = 4, kShSlot = 16384;    // of the K ring, and of the V ring
constexpr int kShRows = 128;                    // query rows of a block
constexpr int kStart = 5;                       // a block's start, in tiles (3: 6% slower, 6: 1%)
constexpr int kShPlanThreads = 1024;
constexpr int kKept = 64;                       // log-sum-exps of a row that the merge keeps
constexpr int kColS = 256;                      // TMEM column of the first score tile
constexpr int kNever = 0x7FFFFFFF;
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kLn2 = 0.69314718055994531f;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

// Positions and blocks, of prefixes and of requests' own parts, summed together.
struct PlanSum {
    int64_t cost[2];
    int blocks[2];
};
__device__ __forceinline__ PlanSum operator+(const PlanSum &a, const PlanSum &b)
{
    return {{a.cost[0] + b.cost[0], a.cost[1] + b.cost[1]},
            {a.blocks[0] + b.blocks[0], a.blocks[1] + b.blocks[1]}};
}
__device__ __forceinline__ PlanSum scan_warp(PlanSum x)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        PlanSum y;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            y.cost[i] = __shfl_up_sync(0xffffffffu, x.cost[i], o);
            y.blocks[i] = __shfl_up_sync(0xffffffffu, x.blocks[i], o);
        }
        if ((threadIdx.x & 31) >= o)
            x = x + y;
    }
    return x;
}

// Parts 0 .. G - 1 are the groups' prefixes, G .. G + R - 1 the requests' own tokens.  The blocks
// behind the first split E4M3's queries meanwhile, a warp a row.
__global__ void __launch_bounds__(kShPlanThreads)
shared_plan_kernel(const SharedArgs a, const PlanBuffers queries)
{
    __shared__ PlanSum warp_sum[32];
    __shared__ int start[kMaxReqs + 1], least[kMaxReqs], eff[kMaxReqs];
    __shared__ int64_t base[kMaxReqs];          // of the groups' prefixes, for the requests
    __shared__ int block0[kMaxReqs], blocks[kMaxReqs];
    // the decode, and the merge behind it, may start once all work before this call is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x > 0) {
        const int row = ((int)blockIdx.x - 1) * (int)(blockDim.x / 32) + ((int)threadIdx.x >> 5);
        if (row < queries.q_rows)
            quantize_row(queries, row);
        return;
    }
    const int t = threadIdx.x, R = a.num_reqs, G = a.num_groups;
    const int64_t cap = min(a.table_cols * kPageTokens, (int64_t)kNever);
    bool bad = false;
    for (int g = t; g <= G; g += blockDim.x)
        start[g] = a.group_starts[g];
    int len = 0, common = 0;
    if (t < G) {
        common = a.shared_lens[t];
        least[t] = kNever;
    }
    if (t < R) {
        len = max(a.seq_lens[t], 0);
        if (len > cap) {
            len = (int)cap;
            if (a.status != nullptr)
                atomicExch(a.status, kStatusAppendPage);
        }
    }
    __syncthreads();
    for (int g = t; g <= G; g += blockDim.x)
        bad |= (g == 0 && start[0] != 0) || (g == G && start[G] != R) ||
               (g < G && start[g] > start[g + 1]);
    // groups that are no partition of the requests: nothing is shared
    bad = __syncthreads_or(bad) != 0;
    if (bad && t == 0 && a.status != nullptr)
        atomicExch(a.status, kStatusGroups);
    int group = 0;
    if (t < R && !bad) {
        int hi = G - 1;                         // the last group that starts at or before t
        while (group < hi) {
            const int mid = (group + hi + 1) / 2;
            if (start[mid] <= t)
                group = mid;
            else
                hi = mid - 1;
        }
        atomicMin(&least[group], len - (a.n_q - 1));
    }
    __syncthreads();
    SharedPart part = {};
    if (t < G) {
        const int members = bad ? 0 : start[t + 1] - start[t];
        int64_t tiles = members > 1 ? max(0, min(common, least[t])) / kTile : 0;
        // worth it where it saves more tiles than its blocks' starts cost
        const int64_t blocks = ((int64_t)members * a.rows + kShRows - 1) / kShRows;
        const int64_t alone = (int64_t)members * ((a.rows + kShRows - 1) / kShRows);
        if (tiles * (alone - blocks) <= kStart * blocks)
            tiles = 0;
        part.tiles = (int)tiles;
        part.blocks = tiles > 0 ? (int)blocks : 0;
        part.req = bad ? 0 : start[t];
        part.len = (int)tiles * kTile;
        part.vis = kNever;
        part.row0 = part.req * a.rows;
        part.rows = members * a.rows;
        eff[t] = part.len;
    }
    __syncthreads();
    SharedPart mine = {};
    if (t < R) {
        mine.tok0 = bad ? 0 : eff[group];
        mine.tiles = len > mine.tok0 ? (len - mine.tok0 - 1) / kTile + 1 : 0;
        mine.blocks = mine.tiles > 0 ? (a.rows + kShRows - 1) / kShRows : 0;
        mine.req = t;
        mine.len = len;
        mine.vis = len - (a.n_q - 1);
        mine.row0 = t * a.rows;
        mine.rows = a.rows;
    }
    const PlanSum own = {{(int64_t)part.blocks * (part.tiles + kStart),
                          (int64_t)mine.blocks * (mine.tiles + kStart)},
                         {part.blocks, mine.blocks}};
    const PlanSum to_here = scan_warp(own);
    const int lane = t & 31, warp = t >> 5;
    if (lane == 31)
        warp_sum[warp] = to_here;
    __syncthreads();
    PlanSum all = lane < (int)blockDim.x / 32 ? warp_sum[lane] : PlanSum{};
    all = scan_warp(all);
    PlanSum before = {}, total;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int from = max(warp - 1, 0);
        before.cost[i] = __shfl_sync(0xffffffffu, all.cost[i], from);
        before.blocks[i] = __shfl_sync(0xffffffffu, all.blocks[i], from);
        before.cost[i] = warp == 0 ? 0 : before.cost[i];
        before.blocks[i] = warp == 0 ? 0 : before.blocks[i];
        total.cost[i] = __shfl_sync(0xffffffffu, all.cost[i], 31);
        total.blocks[i] = __shfl_sync(0xffffffffu, all.blocks[i], 31);
        before.cost[i] += to_here.cost[i] - own.cost[i];
        before.blocks[i] += to_here.blocks[i] - own.blocks[i];
    }
    part.base = before.cost[0];
    part.block0 = before.blocks[0];
    mine.base = total.cost[0] + before.cost[1];
    mine.block0 = total.blocks[0] + before.blocks[1];
    if (t < G) {
        a.parts[t] = part;
        base[t] = part.base;
        block0[t] = part.block0;
        blocks[t] = part.blocks;
    }
    if (t < R)
        a.parts[G + t] = mine;
    __syncthreads();
    if (t < R) {
        SharedSource from = {};
        if (!bad && blocks[group] > 0)
            from = {{base[group], 0}, {eff[group] / kTile, 0}, {block0[group], 0},
                    {start[group] * a.rows, 0}};
        from.base[1] = mine.base;
        from.tiles[1] = mine.tiles;
        from.block0[1] = mine.block0;
        from.row0[1] = mine.row0;
        a.sources[t] = from;
    }
    if (t == 0)
        *a.total = total.cost[0] + total.cost[1];
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------

struct ShBars {
    uint64_t k_full[kShSlots], k_empty[kShSlots], v_full[kShSlots], v_empty[kShSlots];
    uint64_t rope_full, rope_empty, q_full, q_empty;
    uint64_t zeros[2];                          // by the half of the V ring (E4M3)
    uint64_t tail;
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, pv_done, o_free, drain;
};

struct ShMisc {
    ShBars bars;
    uint32_t tmem;
    int abort, status, first, done;             // warps that are through with their run
    SharedPart part;                            // the first
    float quarter[2][256];                      // exchanged between the quarters of a row
};

template <bool F8>
struct ShFmt {
    static constexpr int k_items = F8 ? 2 : 4;  // of two blocks by 64 tokens
    static constexpr int v_items = F8 ? 2 : 4;
    static constexpr int rope_bytes = F8 ? 4096 : 8192;
    static constexpr int q_part = F8 ? 64 * kRow : 128 * kRow;     // bytes of a query part
    static constexpr int parts = F8 ? 2 : 1;
};

constexpr int kShQ = 64 * 2 * kRow;             // bytes of the queries: 64 rows
constexpr int kShP = 16384;
constexpr int kShRope = 8192;
constexpr int kShRing = kShSlots * kShSlot;
constexpr int kShSmem = kShQ + kShP + 2 * kShRing + kShRope + (int)sizeof(ShMisc);
static_assert(kShSmem <= 232448, "shared memory");

__device__ __forceinline__ uint32_t bar_of(const uint64_t &b) { return smem_u32(&b); }

// A pair's run of tiles, segment by segment; every role walks it alike.
struct ShWalk {
    const SharedPart *parts;
    int64_t pos, end;
    int e, blk;
    SharedPart part;
    int t0, t1;                                 // tiles of the segment
    __device__ void begin(const SharedPart *p, const SharedPart &at_from, int first, int64_t from,
                          int64_t to)
    {
        parts = p;
        pos = from;
        end = to;
        e = first;
        part = at_from;
        blk = pos < end ? (int)((pos - part.base) / (part.tiles + kStart)) : 0;
    }
    __device__ bool next()
    {
        while (pos < end) {
            while (blk >= part.blocks) {
                part = parts[++e];
                blk = 0;
            }
            const int64_t at = part.base + (int64_t)blk * (part.tiles + kStart);
            const int64_t stop = min(end, at + part.tiles + kStart);
            t0 = max(0, (int)(pos - at) - kStart);
            t1 = (int)(stop - at) - kStart;
            slot_block = part.block0 + blk;
            row0 = blk * kShRows;
            pos = stop;
            if (stop == at + part.tiles + kStart)
                ++blk;
            if (t1 > t0)
                return true;
        }
        return false;
    }
    int slot_block, row0;
};

// Pairs with work: each has a position at least, so that every pair between the first and the
// last of a block has a segment of it.
__device__ __forceinline__ int64_t busy_pairs(int64_t total, int pairs)
{
    return total < pairs ? max(total, (int64_t)1) : pairs;
}

// All threads of the pair, without the memory ordering of cluster_sync, whose release waits for
// every store of the CTA.
__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.b32 %0, 1, 0, e;\n\t}"
                 : "=r"(r));
    return r;
}

// The pair's MMA by the elected lane of a converged warp.
template <bool F8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate, uint32_t elected)
{
    if constexpr (F8)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected));
    else
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected));
}

__device__ __forceinline__ void pair_commit(uint32_t bar, uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3), "r"(elected)
        : "memory");
}

// Arrive on a barrier of either CTA, releasing to this CTA: what the softmax warps hand over
// (the probabilities, behind a proxy fence; TMEM) is used by their own SM's tensor core.
__device__ __forceinline__ void arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Expect bytes on one of the even CTA's barriers, and loads that complete there, by the lane
// of a converged warp with `go` set (in a divergent branch every operand costs a move to
// the uniform registers: some 200 cycles a load).
__device__ __forceinline__ void expect_if(uint32_t bar, uint32_t bytes, uint32_t go)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(go)
        : "memory");
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap *map, int c1, int c2, int c3,
                                        uint32_t bar, uint64_t policy, uint32_t go)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %7, 0;\n\t"
        "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {0, %2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy),
        "r"(go)
        : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                        uint32_t bar, uint64_t policy, uint32_t go)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %7, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy),
        "r"(go)
        : "memory");
}

__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// 16 bytes of V: what is not finite becomes 0.
template <bool F8>
__device__ __forceinline__ void finite_16(uint32_t addr)
{
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a mask of the elements whose exponent (bf16), or all of them but the sign (E4M3), is ones
        const uint32_t bad = F8 ? __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                : __vcmpeq2(w[i] & 0x7F807F80u, 0x7F807F80u);
        any |= bad;
        w[i] &= ~bad;
    }
    if (any != 0)
        st_shared_16(addr, w[0], w[1], w[2], w[3]);
}

// The end of the tokens that every row of the part sees.
__device__ __forceinline__ int tokens_to_all(const SharedPart &part) { return min(part.len, part.vis); }

struct ShMaps {
    CUtensorMap k, v, rope, qn, qr;
};

// Waits through the whole run: while the CTA's other warps go on (their waits are bounded), and
// then as wait_drain.
__device__ __noinline__ void wait_last(uint32_t bar, volatile int *abort_flag, volatile int *done,
                                       int others, int32_t *status)
{
    unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, 0)) {
        const unsigned long long now = global_ns();
        if (!*abort_flag && *done < others) {
            t0 = now;
        } else if (now - t0 > kDrainLimitNs) {
            atomicCAS(status, 0, 15);
            return;
        }
    }
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// The page of a part's column, 0 (reported) where the table has none of the pool.
__device__ __forceinline__ int page_at(const SharedArgs &a, int req, int col, int32_t *status)
{
    const int page = a.page_table[(int64_t)req * a.table_ld + col];
    if (page >= 0 && (int64_t)page < a.num_pages)
        return page;
    atomicExch(status, kStatusAppendPage);
    return 0;
}

template <bool F8>
__global__ void __launch_bounds__(kShThreads, 1)
shared_decode_kernel(const __grid_constant__ ShMaps maps, const SharedArgs a)
{
    using F = ShFmt<F8>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t s_q = smem_u32(smem), s_p = s_q + kShQ, s_k = s_p + kShP, s_v = s_k + kShRing;
    const uint32_t s_rope = s_v + kShRing;
    ShMisc &m = *reinterpret_cast<ShMisc *>(smem + kShQ + kShP + 2 * kShRing + kShRope);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    if ((s_q & 1023u) != 0u) {         // cannot be with no static shared memory
        if (threadIdx.x == 0 && a.status != nullptr)
            atomicExch(a.status, 12);
        return;
    }
    if (threadIdx.x >= 64 && threadIdx.x < 64 + sizeof(ShMaps) / sizeof(CUtensorMap))
        asm volatile("prefetch.tensormap [%0];" ::"l"(
            reinterpret_cast<uint64_t>(&maps.k + (threadIdx.x - 64))) : "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kShSlots; ++i) {
            mbar_init(bar_of(m.bars.k_full[i]), 1);           // the even CTA expects for both
            mbar_init(bar_of(m.bars.k_empty[i]), 1);
            mbar_init(bar_of(m.bars.v_full[i]), 1);
            mbar_init(bar_of(m.bars.v_empty[i]), 1);
        }
        mbar_init(bar_of(m.bars.tail), 1);
        mbar_init(bar_of(m.bars.rope_full), 1);
        mbar_init(bar_of(m.bars.rope_empty), 1);
        mbar_init(bar_of(m.bars.q_full), 1);
        mbar_init(bar_of(m.bars.q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_of(m.bars.zeros[i]), 2);            // both CTAs wrote them
            mbar_init(bar_of(m.bars.s_full[i]), 1);
            mbar_init(bar_of(m.bars.s_free[i]), 16);          // the pair's softmax warps
        }
        mbar_init(bar_of(m.bars.p_full), 16);
        mbar_init(bar_of(m.bars.pv_done), 1);
        mbar_init(bar_of(m.bars.o_free), 16);
        mbar_init(bar_of(m.bars.drain), 1);
        m.abort = 0;
        m.status = 0;
        m.first = 0;
        m.done = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&m.tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    const uint32_t rank = cluster_rank();
    const int pair = (int)blockIdx.x >> 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");        // the plan (and split queries)
    const int num_parts = a.num_groups + a.num_reqs;
    SharedPart own = {};
    if ((int)threadIdx.x < num_parts)
        own = a.parts[threadIdx.x];
    const int64_t total = *a.total;
    const int64_t pairs = busy_pairs(total, (int)gridDim.x >> 1);
    const int64_t from = pair < pairs ? total * pair / pairs : total;
    const int64_t to = pair < pairs ? total * (pair + 1) / pairs : total;
    {
        // the part that holds the run's first position: the last one that starts there or before
        int mine = (int)threadIdx.x < num_parts && own.base <= from ? (int)threadIdx.x : 0;
        for (int e = threadIdx.x + kShThreads; e < num_parts; e += kShThreads)
            if (a.parts[e].base <= from)
                mine = e;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (mine != 0)
            atomicMax(&m.first, mine);
        __syncthreads();
        // (another read of it from L2 would be on the way to the first loads)
        if (m.first == (int)threadIdx.x)
            m.part = own;
        else if (threadIdx.x == 0 && m.first >= kShThreads)
            m.part = a.parts[m.first];
        __threadfence_block();                  // (the barrier below orders nothing by itself)
    }
    pair_sync();                                // the pair's barriers are initialised (and fenced)
    const uint32_t tmem = __shfl_sync(0xffffffffu, m.tmem, 0);
    volatile int *abort_flag = &m.abort;
    int32_t *status = &m.status;
    auto lead = [&](const uint64_t &b) { return map_rank(bar_of(b), 0); };
    ShWalk walk;
    walk.begin(a.parts, m.part, m.first, from, to);

    if (warp == 0) {
        // ------------------------------------------------------------ K loads
        const uint64_t keep = l2_policy_evict_last();
        const uint32_t el = elect_one(), el0 = rank == 0 ? el : 0;
        const uint32_t full = lead(m.bars.k_full[0]), empty = bar_of(m.bars.k_empty[0]);
        int64_t g = 0;
        bool ok = true;
        while (ok && walk.next()) {
            int col = -1, page = 0;
#pragma unroll 1
            for (int t = walk.t0; t < walk.t1 && ok; ++t, ++g) {
                const int tok = walk.part.tok0 + t * kTile;
                if (tok / kPageTokens != col) {
                    col = tok / kPageTokens;
                    page = page_at(a, walk.part.req, col, status);
                }
                const int own = tok % kPageTokens + 64 * (int)rank;
                const int half = F8 ? 2 * (int)(g & 1) : 0;
                const uint32_t phase = (uint32_t)(F8 ? g >> 1 : g) & 1u;
#pragma unroll
                for (int i = 0; i < F::k_items; ++i) {
                    const uint32_t at = 8 * (half + i);
                    ok &= wait_bounded(empty + at, phase ^ 1, abort_flag, status, 2);
                    expect_if(full + at, 2 * kShSlot, ok ? el0 : 0);
                    load_4d(s_k + (half + i) * kShSlot, &maps.k, own, 2 * i, page, full + at, keep,
                            ok ? el : 0);
                }
                ok = all_ok(ok);
            }
        }
        // both CTAs' copies complete on the even CTA's barriers: it waits for the last ones
        if (rank == 0 && lane == 0) {
            const int64_t items = g * F::k_items;
            for (int64_t it = items > kShSlots ? items - kShSlots : 0; it < items; ++it)
                wait_drain(bar_of(m.bars.k_full[it % kShSlots]), (uint32_t)(it / kShSlots) & 1u);
        }
    } else if (warp == 3) {
        // --------------------------------------- Q, and the rope block of K
        const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
        const uint32_t el = elect_one(), el0 = rank == 0 ? el : 0;
        const uint32_t rope_full = lead(m.bars.rope_full), q_full = lead(m.bars.q_full);
        int64_t g = 0;
        int loads = 0;
        bool ok = true;
        while (ok && walk.next()) {
            if (loads > 0)
                ok = all_ok(wait_bounded(bar_of(m.bars.q_empty), (loads - 1) & 1, abort_flag, status,
                                         1));
            if (!ok)
                break;
            expect_if(q_full, 2 * kShQ, el0);
            const int row = walk.part.row0 + walk.row0 + 64 * (int)rank;
#pragma unroll
            for (int p = 0; p < F::parts; ++p) {
                const uint32_t dst = s_q + p * F::q_part;
                const int at = p * a.num_reqs * a.rows + row;
                load_3d(dst, &maps.qn, 0, at, 0, q_full, keep, el);
                load_3d(dst + F::q_part - F::rope_bytes, &maps.qr, F8 ? kLatent : 0, at, 0, q_full,
                        keep, el);
            }
            ++loads;
            // other pairs read a prefix too
            const uint64_t use = walk.part.vis == kNever ? keep : once;
            int col = -1, page = 0;
#pragma unroll 1
            for (int t = walk.t0; t < walk.t1 && ok; ++t, ++g) {
                const int tok = walk.part.tok0 + t * kTile;
                if (tok / kPageTokens != col) {
                    col = tok / kPageTokens;
                    page = page_at(a, walk.part.req, col, status);
                }
                if (g > 0)
                    ok = all_ok(wait_bounded(bar_of(m.bars.rope_empty), (uint32_t)(g - 1) & 1u,
                                             abort_flag, status, 3));
                expect_if(rope_full, 2 * F::rope_bytes, ok ? el0 : 0);
                load_3d(s_rope, &maps.rope, kLatent, tok % kPageTokens + 64 * (int)rank, page,
                        rope_full, use, ok ? el : 0);
            }
        }
        if (rank == 0 && lane == 0) {
            if (loads > 0)
                wait_drain(bar_of(m.bars.q_full), (loads - 1) & 1);
            if (g > 0)
                wait_drain(bar_of(m.bars.rope_full), (uint32_t)(g - 1) & 1u);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ V loads
        const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
        const uint32_t el = elect_one(), el0 = rank == 0 ? el : 0;
        const uint32_t full = lead(m.bars.v_full[0]), empty = bar_of(m.bars.v_empty[0]);
        const uint32_t own_tail = map_rank(bar_of(m.bars.tail), rank);
        int64_t g = 0;
        uint32_t tails = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const uint64_t use = walk.part.vis == kNever ? keep : once;
            int col = -1, page = 0;
#pragma unroll 1
            for (int t = walk.t0; t < walk.t1 && ok; ++t, ++g) {
                const int tok = walk.part.tok0 + t * kTile;
                if (tok / kPageTokens != col) {
                    col = tok / kPageTokens;
                    page = page_at(a, walk.part.req, col, status);
                }
                const int in_page = tok % kPageTokens, valid = walk.part.len - tok;
                const int seen = tokens_to_all(walk.part) - tok;
                const int half = F8 ? 2 * (int)(g & 1) : 0;
                const uint32_t phase = (uint32_t)(F8 ? g >> 1 : g) & 1u;
                // item i: bf16 (256 columns i / 2, 64 tokens i % 2); E4M3 (256 columns i)
                if (seen >= kTile) {
#pragma unroll
                    for (int i = 0; i < F::v_items; ++i) {
                        const uint32_t at = 8 * (half + i);
                        const int block = F8 ? 2 * i + (int)rank : 4 * (i >> 1) + 2 * (int)rank;
                        ok &= wait_bounded(empty + at, phase ^ 1, abort_flag, status, 2);
                        expect_if(full + at, 2 * kShSlot, ok ? el0 : 0);
                        load_4d(s_v + (half + i) * kShSlot, &maps.v, in_page + (F8 ? 0 : 64 * (i & 1)),
                                block, page, full + at, use, ok ? el : 0);
                    }
                    ok = all_ok(ok);
                    continue;
                }
                // A history's last tiles.  Rows past the history hold stale data, those of
                // drafts are not seen by all of its queries, and a weight of 0 times NaN is NaN.
                // The tile is loaded on a barrier of this CTA's own; before the MMAs hear of it,
                // rows past the history become zeros, and so does what is not finite in a
                // draft's row (the queries that see it have it in their scores).
                for (int i = 0; i < F::v_items; ++i)
                    ok &= wait_bounded(empty + 8 * (half + i), phase ^ 1, abort_flag, status, 2);
                ok = all_ok(ok);
                if (!ok)
                    break;
                expect_if(bar_of(m.bars.tail), F::v_items * kShSlot, el);
#pragma unroll
                for (int i = 0; i < F::v_items; ++i)
                    load_4d(s_v + (half + i) * kShSlot, &maps.v, in_page + (F8 ? 0 : 64 * (i & 1)),
                            F8 ? 2 * i + (int)rank : 4 * (i >> 1) + 2 * (int)rank, page, own_tail,
                            use, el);
                ok = all_ok(wait_bounded(bar_of(m.bars.tail), tails & 1u, abort_flag, status, 13));
                ++tails;
                constexpr int kCols = F8 ? 1 : 2;             // 128-byte blocks of an item
                constexpr int t_num = F8 ? 128 : 64, pitch = t_num * 128;
                for (int i = 0; i < F::v_items; ++i) {
                    const int n = min(t_num, max(0, valid - (F8 ? 0 : 64 * (i & 1))));
                    const int m = min(n, max(0, seen - (F8 ? 0 : 64 * (i & 1))));
                    for (int b = 0; b < kCols; ++b) {
                        const uint32_t block = s_v + (half + i) * kShSlot + b * pitch;
#pragma unroll 4
                        for (int x = m * 128 + 16 * lane; x < n * 128; x += 512)
                            finite_16<F8>(block + x);
                        for (int x = n * 128 + 16 * lane; x < pitch; x += 512)
                            st_shared_16(block + x, 0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(lead(m.bars.zeros[half >> 1]));
                if (rank == 0 && lane == 0)
                    for (int i = 0; i < F::v_items; ++i)
                        mbar_arrive(bar_of(m.bars.v_full[half + i]));
            }
        }
        if (rank == 0 && lane == 0) {
            const int64_t items = g * F::v_items;
            for (int64_t it = items > kShSlots ? items - kShSlots : 0; it < items; ++it)
                wait_drain(bar_of(m.bars.v_full[it % kShSlots]), (uint32_t)(it / kShSlots) & 1u);
        }
    } else if (warp == 1 && rank == 0) {
        // -------------------------------------------------------- MMA issue
        // K runs a tile ahead of V.  A wait that gives up is noticed at the tile's end: MMAs on
        // what had not arrived stay within the pair's memory, and nothing is stored.
        const uint32_t el = elect_one();
        constexpr uint32_t id_s = idesc_for<F8>(128, 128, false, false);
        constexpr uint32_t id_o = idesc_for<F8>(128, 256, false, true);
        constexpr uint32_t id_o_lo = F8 ? idesc_e5m2_e4m3(128, 256, false, true) : id_o;
        const uint64_t dq0 = sdesc(s_q, 16, 1024, kSw128);
        const uint64_t dq_rope = sdesc(s_q + F::q_part - F::rope_bytes, 16, F8 ? 512 : 1024,
                                       F8 ? kSw64 : kSw128);
        const uint64_t dk_rope = sdesc(s_rope, 16, F8 ? 512 : 1024, F8 ? kSw64 : kSw128);
        const uint64_t dk0 = sdesc(s_k, 16, 1024, kSw128);
        // V: columns contiguous; two 64-column blocks 8 KB apart (bf16), 8-token groups 1 KB
        const uint64_t dv0 = sdesc(s_v, 8192, 1024, kSw128);
        const uint64_t dp0 = sdesc(s_p, 16, 1024, kSw128);
        constexpr uint64_t kPart = F::q_part >> 4;
        ShWalk vw = walk;
        bool more = walk.next(), v_any = vw.next(), ok = true, any = v_any;
        int kt = walk.t0, vt = vw.t0, loads = 0;
        uint32_t tails = 0;                     // phases of the zeros
        int64_t g = 0, v = 0, segs = 0;         // tiles scored, tiles multiplied, segments done
        auto wait = [&](uint32_t bar, uint32_t parity, int code) {
            ok &= wait_bounded(bar, parity, abort_flag, status, code);
            tc_fence_after();
        };
        while (v_any) {
            if (more) {
                if (kt == walk.t0) {
                    wait(bar_of(m.bars.q_full), loads & 1, 4);
                    ++loads;
                }
                const int buf = (int)(g & 1);
                if (g >= 2)
                    wait(bar_of(m.bars.s_free[buf]), (uint32_t)((g - 2) >> 1) & 1u, 5);
                const uint32_t d = tmem + kColS + 64 * buf;
                const uint32_t phase = (uint32_t)(F8 ? g >> 1 : g) & 1u;
                const int half = F8 ? 2 * buf : 0;
#pragma unroll
                for (int i = 0; i < F::k_items; ++i) {
                    if (i == F::k_items / 2) {
                        wait(bar_of(m.bars.rope_full), (uint32_t)g & 1u, 6);
                        constexpr int kSteps = F8 ? 2 : 4;
#pragma unroll
                        for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
                            for (int p = 0; p < F::parts; ++p)
                                pair_mma<F8>(d, dq_rope + p * kPart + 2 * kk, dk_rope + 2 * kk,
                                             id_s, 1, el);
                        pair_commit(bar_of(m.bars.rope_empty), el);
                    }
                    wait(bar_of(m.bars.k_full[0]) + 8 * (half + i), phase, 7);
                    const uint64_t dk = dk0 + (uint64_t)((half + i) * (kShSlot >> 4));
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int p = 0; p < F::parts; ++p)
                            pair_mma<F8>(d, dq0 + p * kPart + (2 * i + kk / 4) * 512 + 2 * (kk % 4),
                                         dk + (kk / 4) * 512 + 2 * (kk % 4), id_s,
                                         (i | kk | p) != 0, el);
                    pair_commit(bar_of(m.bars.k_empty[0]) + 8 * (half + i), el);
                }
                pair_commit(bar_of(m.bars.s_full[buf]), el);
                ++g;
                if (++kt == walk.t1) {
                    pair_commit(bar_of(m.bars.q_empty), el);
                    more = walk.next();
                    kt = walk.t0;
                }
                if (!all_ok(ok))
                    break;
                if (g == 1 && more)
                    continue;
            }
            // the segment before must have left O
            if (vt == vw.t0 && segs > 0)
                wait(bar_of(m.bars.o_free), (uint32_t)(segs - 1) & 1u, 8);
            const int half = F8 ? 2 * (int)(v & 1) : 0;
            if (tokens_to_all(vw.part) - (vw.part.tok0 + vt * kTile) < kTile) {
                wait(bar_of(m.bars.zeros[half >> 1]), tails >> (half >> 1) & 1u, 12);
                tails ^= 1u << (half >> 1);
            }
            wait(bar_of(m.bars.p_full), (uint32_t)v & 1u, 9);
            const uint32_t carry = vt != vw.t0 ? 1 : 0;
            const uint32_t phase = (uint32_t)(F8 ? v >> 1 : v) & 1u;
#pragma unroll
            for (int i = 0; i < F::v_items; ++i) {
                wait(bar_of(m.bars.v_full[0]) + 8 * (half + i), phase, 10);
                const uint64_t dv = dv0 + (uint64_t)((half + i) * (kShSlot >> 4));
                const int h = F8 ? i : i >> 1;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int p = 0; p < F::parts; ++p) {
                        // bf16: 16 tokens a step, P in blocks of 64; E4M3: 32, hi and lo blocks
                        const uint64_t dp = F8 ? dp0 + p * 512 + 2 * kk
                                               : dp0 + (i & 1) * 512 + 2 * kk;
                        const uint32_t acc =
                            (F8 ? (kk | p) != 0 : (kk | (i & 1)) != 0) ? 1u : carry;
                        pair_mma<F8>(tmem + 128 * h, dp, dv + (F8 ? 256 : 128) * kk,
                                     p == 0 ? id_o : id_o_lo, acc, el);
                    }
                pair_commit(bar_of(m.bars.v_empty[0]) + 8 * (half + i), el);
            }
            pair_commit(bar_of(m.bars.pv_done), el);
            ++v;
            if (++vt == vw.t1) {
                ++segs;
                v_any = vw.next();
                vt = vw.t0;
            }
            if (!all_ok(ok))
                break;
        }
        if (any) {
            pair_commit(bar_of(m.bars.drain), el);
            if (lane == 0)
                wait_drain(bar_of(m.bars.drain), 0);
        }
    } else if (warp == 1 && lane == 0) {
        // the even CTA's commits arrive here too: the last of them comes after the others
        if (walk.next())
            wait_last(bar_of(m.bars.drain), abort_flag, &m.done, kShThreads / 32 - 1, status);
    } else if (warp >= 4) {
        // -------------------------------------------------- softmax, epilogue
        // Thread (warp group, quad, lane): row 32 (quad % 2) + lane of this CTA, and of a tile the 32
        // tokens from 64 (quad / 2) + 32 group on: a quarter of the row.  A wait that gives up
        // clears `ok`: the loops run on without waiting or storing, so that every thread still
        // meets the barriers.
        const int quad = warp & 3, row = 32 * (quad & 1) + lane, side = quad >> 1;
        const int group = (warp - 4) >> 2, tid = 32 * quad + lane + 128 * group;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        constexpr float kLag = F8 ? 4.f : 8.f, kUp = F8 ? 4.f : 0.f;
        constexpr float kFall = 6.f, kMost = 40.f;            // (E4M3)
        constexpr int kChunks = F8 ? 2 : 4;     // 16-byte chunks of P (of each part)
        const uint32_t p_row = s_p + row * 128 + (F8 ? 0 : side * 8192);
        bool ok = true;
        int64_t g = 0;
        int exchange = 0;
        auto wait = [&](const uint64_t &b, uint32_t parity, int code) {
            ok = all_ok(ok && wait_bounded(bar_of(b), parity, abort_flag, status, code));
            tc_fence_after();
        };
        auto arrive = [&](const uint64_t &b) {
            __syncwarp();
            if (lane == 0)
                arrive_pair(lead(b));
        };
        while (walk.next()) {
            const SharedPart &part = walk.part;
            const int in_part = walk.row0 + 64 * (int)rank + row;
            const bool real = in_part < part.rows;
            // tokens that the row sees
            int limit = part.len;
            if (part.vis != kNever)
                limit = min(part.len, part.vis + in_part / a.heads);
            float f = a.scale_log2;
            if constexpr (F8)
                f = real ? ldexpf(f * a.kv_scale, a.qexp[part.row0 + in_part]) : 1.f;
            // in units of log2, of all tokens; of this thread's tokens
            float high = -INFINITY, top_most = -INFINITY, sum = 0.f;
            for (int t = walk.t0; t < walk.t1; ++t, ++g, ++exchange) {
                const int buf = (int)(g & 1);
                wait(m.bars.s_full[buf], (uint32_t)(g >> 1) & 1u, 11);
                float x[32];
                {
                    uint32_t r[2][16];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tmem_ld16(lanes + kColS + 64 * buf + 32 * group + 16 * i, r[i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __uint_as_float(r[i / 16][i % 16]);
                }
                tc_fence_before();
                arrive(m.bars.s_free[buf]);
                const int seen = limit - (part.tok0 + t * kTile + 64 * side + 32 * group);
                if (seen < 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = i < seen ? x[i] : -INFINITY;
                }
                float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int i = 4; i < 32; ++i)
                    top[i % 4] = fmaxf(top[i % 4], x[i]);
                float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                float(&quarter)[256] = m.quarter[exchange & 1];
                quarter[tid] = best;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                best = fmaxf(fmaxf(best, quarter[tid ^ 64]),
                             fmaxf(quarter[tid ^ 128], quarter[tid ^ 192])) * f;
                float shrink = 1.f;
                if (t == walk.t0) {
                    high = best;
                } else if (best > high + kLag || (F8 && best < high - kFall && best > -INFINITY)) {
                    // (kMost octaves below the largest a weight does not count any more)
                    const float next = F8 ? fmaxf(best, top_most - kMost) : best;
                    shrink = fast_exp2(high - next);          // 0 where nothing was seen before
                    high = next;
                    sum *= shrink;
                }
                top_most = fmaxf(top_most, best);
                const float ref = high == -INFINITY ? 0.f : high - kUp;
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    x[i] = fast_exp2(fmaf(x[i], f, -ref));
                    add[i % 4] += x[i];
                }
                sum += (add[0] + add[1]) + (add[2] + add[3]);
                uint32_t hi[4 * kChunks], lo[F8 ? 4 * kChunks : 1];
                if constexpr (F8) {
#pragma unroll
                    for (int w = 0; w < 8; ++w) {
                        // hi: four significant bits, rounded; lo: the rest, in three
                        const uint16_t h0 = e4m3x2(x[4 * w], x[4 * w + 1]);
                        const uint16_t h1 = e4m3x2(x[4 * w + 2], x[4 * w + 3]);
                        const float2 f0 = e4m3x2_to_float2(h0), f1 = e4m3x2_to_float2(h1);
                        hi[w] = (uint32_t)h0 | (uint32_t)h1 << 16;
                        lo[w] = (uint32_t)e5m2x2(x[4 * w] - f0.x, x[4 * w + 1] - f0.y) |
                                (uint32_t)e5m2x2(x[4 * w + 2] - f1.x, x[4 * w + 3] - f1.y) << 16;
                    }
                } else {
                    lo[0] = 0;
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * w], x[2 * w + 1]);
                        hi[w] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                }
                // P is free, and O at rest, once the product of the tile before is done
                if (g > 0)
                    wait(m.bars.pv_done, (uint32_t)(g - 1) & 1u, 14);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int chunk = (F8 ? 4 * side : 0) + kChunks * group + c;
                    const uint32_t at = p_row + ((chunk ^ (row & 7)) << 4);
                    st_shared_16(at, hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                    if constexpr (F8)
                        st_shared_16(at + 8192, lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                }
                if (__any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                    for (int c = 128 * group; c < 128 * group + 128; c += 16) {
                        uint32_t r[16];
                        tmem_ld16(lanes + c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            r[i] = __float_as_uint(__uint_as_float(r[i]) * shrink);
                        tmem_st16(lanes + c, r);
                    }
                    tmem_wait_st();
                }
                fence_proxy_async();
                tc_fence_before();
                arrive(m.bars.p_full);
            }
            // the segment's partial
            float(&quarter)[256] = m.quarter[exchange++ & 1];
            quarter[tid] = sum;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            // (in one order, so that all four agree)
            const int q0 = tid & 63;
            sum = (quarter[q0] + quarter[q0 + 64]) + (quarter[q0 + 128] + quarter[q0 + 192]);
            wait(m.bars.pv_done, (uint32_t)(g - 1) & 1u, 15);
            const int64_t slot = (int64_t)walk.slot_block + pair;
            const bool store = real && ok && !*abort_flag;
            float scale = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;    // NaN stays
            if constexpr (F8)
                scale *= a.kv_scale;
            // lane by lane, so that a store covers 512 bytes
            float4 *out = reinterpret_cast<float4 *>(a.o_part) +
                          ((slot * 2 + (int)rank) * 4 + quad) * 64 * 32 + lane;
            uint32_t r[2][16];                  // the next columns are read while these are stored
            tmem_ld16(lanes + 128 * group, r[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 128 * group + 16 * j;
                tmem_wait_ld();
                if (j < 7)
                    tmem_ld16(lanes + c + 16, r[(j + 1) & 1]);
                const uint32_t(&x)[16] = r[j & 1];
                if (store)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[(c / 4 + i) * 32] = make_float4(
                            __uint_as_float(x[4 * i]) * scale, __uint_as_float(x[4 * i + 1]) * scale,
                            __uint_as_float(x[4 * i + 2]) * scale,
                            __uint_as_float(x[4 * i + 3]) * scale);
            }
            tc_fence_before();
            arrive(m.bars.o_free);
            if (store && side == 0 && group == 0)
                a.lse_part[slot * kShRows + 64 * (int)rank + row] =
                    sum == 0.f ? -INFINITY : (high - kUp + log2f(sum)) * kLn2;
        }
    }

    if (warp != 1 && lane == 0)
        atomicAdd(&m.done, 1);
    tc_fence_before();
    __syncthreads();
    // A pair leaves together: no copy or arrival of one CTA is on its way to the other, and
    // each has waited for its own copy of the last commit.
    pair_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
    if (threadIdx.x == 0 && m.status != 0 && a.status != nullptr)
        atomicExch(a.status, m.status);
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------

// The sigmoid times 2^8; the merge of many rows is bound by instructions, which the exact
// division and exponential were half of.  Within 2^-20 of itself for gates above -16, 2^-17 down to
// -92.8 (the exponent's rounding), 0 below: the quotient takes divisors up to 2^126, which the
// factor brings to where a bf16 product with at most 1 ends.
constexpr float kGateScale = 256.f;
__device__ __forceinline__ float gate_of(float x)
{
    return __fdividef(1.f, 1.f / kGateScale + fast_exp2(fmaf(-x, (float)kLog2e, -8.f)));
}

// A block takes 32 rows by 8 C columns: a warp C of the columns of every PARTS'th partial, a lane
// a row, as the partials lie ([slot, CTA, TMEM quadrant, four columns, lane]), and the block
// writes its outputs in whole pieces of rows.  A row's partials are those of the group's
// prefix, then those of the request's own tokens, in the order of their tokens.  Many rows are
// bound by the reads and take 16 columns a warp; with few, each of many partials, latency
// counts, and two warps share them (512 rows of 20 partials: 3 us less), two blocks an SM (0.7 us
// less than with one; the form for many rows is slower with any minimum: 1-13%).
template <int C, int PARTS>
__global__ void __launch_bounds__(256 * PARTS, PARTS == 1 ? 0 : 2)
shared_merge_kernel(const SharedArgs a, const int pairs)
{
    constexpr int kThreads = 256 * PARTS, kWarps = kThreads / 32, kBlocks = kLatent / (8 * C);
    constexpr int kOut = 32 * 2 * C / kThreads;               // groups of 4 columns of a thread
    __shared__ float tile[PARTS][32][8 * C + 1], sums[PARTS][32];
    __shared__ float lses[kKept][32], highs[kWarps][32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp >> 3;
    const int64_t rows = (int64_t)a.num_reqs * a.rows, row0 = (int64_t)(blockIdx.x / kBlocks) * 32;
    const int row = (int)min(row0 + lane, rows - 1), req = row / a.rows;  // (2^25 rows at most)
    const int col0 = (int)(blockIdx.x % kBlocks) * 8 * C, col = col0 + C * (warp & 7);
    uint2 gate[kOut];
#pragma unroll
    for (int q = 0; q < kOut; ++q) {
        const int u = threadIdx.x + q * kThreads;
        gate[q] = make_uint2(0u, 0u);
        if (row0 + u / (2 * C) < rows)
            gate[q] = *reinterpret_cast<const uint2 *>(a.gate + (row0 + u / (2 * C)) * kLatent +
                                                       col0 + 4 * (u % (2 * C)));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the row's partials: of the prefix (0) and of its own tokens (1)
    const int64_t total = *a.total, busy = busy_pairs(total, pairs);
    const SharedSource from = a.sources[req];
    // the pair that has position x: (the last p with p total / busy, rounded down, <= x)
    auto pair_of = [&](int64_t x) -> int {
        return total < 1 << 24 ? (int)(((uint32_t)(x + 1) * (uint32_t)busy - 1) / (uint32_t)total)
                               : (int)(((x + 1) * busy - 1) / total);
    };
    int n[2], at[2];
    int64_t first[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int in_part = row - from.row0[i], blk = in_part / kShRows;
        // positions of the block's tiles
        const int64_t v0 = from.base[i] + (int64_t)blk * (from.tiles[i] + kStart) + kStart;
        n[i] = at[i] = 0;
        first[i] = 0;
        if (from.tiles[i] > 0) {
            const int p0 = pair_of(v0);
            n[i] = pair_of(v0 + from.tiles[i] - 1) - p0 + 1;
            first[i] = (int64_t)from.block0[i] + blk + p0;
            at[i] = in_part % kShRows;
        }
    }
    // their log-sum-exps, each by one of the warps
    const int all = n[0] + n[1];
    float high = -INFINITY;
    auto lse_at = [&](int k) -> float {
        const int64_t slot = k < n[0] ? first[0] + k : first[1] + k - n[0];
        return __ldcg(a.lse_part + slot * kShRows + (k < n[0] ? at[0] : at[1]));
    };
    for (int k = warp; k < all; k += kWarps) {
        const float l = lse_at(k);
        if (k < kKept)
            lses[k][lane] = l;
        high = fmaxf(high, l);
    }
    highs[warp][lane] = high;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        high = fmaxf(high, highs[w][lane]);
    const float ref = high == -INFINITY ? 0.f : high;
    float acc[C] = {}, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // CTA, quadrant (rows, side of 128 columns), four columns, lane
        const int quad = (at[i] >> 5 & 1) + 2 * (col >> 7 & 1);
        const float4 *src = reinterpret_cast<const float4 *>(a.o_part) +
                            (((first[i] * 2 + (at[i] >> 6)) * 4 + quad) * 64 +
                             (col >> 8) * 32 + (col & 127) / 4) * 32 + (at[i] & 31);
        const int before = i == 0 ? 0 : n[0], kept = min(n[i], kKept - min(before, kKept));
        auto take = [&](int k, float l) {
            float4 x[C / 4];
#pragma unroll
            for (int j = 0; j < C / 4; ++j)
                x[j] = __ldcg(src + (int64_t)k * kShRows * kLatent / 4 + 32 * j);
            const float w = fast_exp2((l - ref) * (float)kLog2e);
            sum += w;
#pragma unroll
            for (int j = 0; j < C / 4; ++j) {
                if (w == 0.f)                   // not seen by the row: may hold 0 times NaN
                    x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                acc[4 * j] = fmaf(w, x[j].x, acc[4 * j]);
                acc[4 * j + 1] = fmaf(w, x[j].y, acc[4 * j + 1]);
                acc[4 * j + 2] = fmaf(w, x[j].z, acc[4 * j + 2]);
                acc[4 * j + 3] = fmaf(w, x[j].w, acc[4 * j + 3]);
            }
        };
#pragma unroll (64 / C)
        for (int k = part; k < kept; k += PARTS)
            take(k, lses[before + k][lane]);
        for (int k = kept + (kept + part) % PARTS; k < n[i]; k += PARTS)
            take(k, lse_at(before + k));
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
        tile[part][lane][C * (warp & 7) + j] = acc[j];
    if ((warp & 7) == 0)
        sums[part][lane] = sum;
    __syncthreads();
    if (warp == 0 && col0 == 0 && row0 + lane < rows && a.lse != nullptr) {
        sum = PARTS == 2 ? sums[0][lane] + sums[PARTS - 1][lane] : sums[0][lane];
        a.lse[row] = sum == 0.f ? -INFINITY : high + logf(sum);
    }
#pragma unroll
    for (int q = 0; q < kOut; ++q) {
        const int u = threadIdx.x + q * kThreads, i = u / (2 * C), c = 4 * (u % (2 * C));
        if (row0 + i >= rows)
            continue;
        float s = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            s += sums[p][i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] += tile[p][i][c + j];
        }
        const float inv = s == 0.f ? 0.f : 1.f / (s * kGateScale);
        const float2 g0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&gate[q].x));
        const float2 g1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&gate[q].y));
        const __nv_bfloat162 o0 = __floats2bfloat162_rn(v[0] * inv * gate_of(g0.x),
                                                        v[1] * inv * gate_of(g0.y));
        const __nv_bfloat162 o1 = __floats2bfloat162_rn(v[2] * inv * gate_of(g1.x),
                                                        v[3] * inv * gate_of(g1.y));
        *reinterpret_cast<uint2 *>(a.out + (row0 + i) * kLatent + col0 + c) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&o0), *reinterpret_cast<const uint32_t *>(&o1));
    }
}

template <bool F8>
cudaError_t launch_decode(const SharedArgs &a, int sms, cudaStream_t stream)
{
    const CUtensorMapDataType dt = F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t es = F8 ? 1 : 2, wide = F8 ? 128 : 64;
    const cuuint64_t blocks = F8 ? 4 : 9, rows = (cuuint64_t)a.num_reqs * a.rows;
    ShMaps m;
    // (column in a 128-byte block, token, block, page)
    const cuuint64_t dims[4] = {wide, (cuuint64_t)kPageTokens, blocks, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {kRow * es, 128, (cuuint64_t)a.page_stride * es};
    const cuuint32_t w32 = (cuuint32_t)wide;
    const cuuint32_t k_box[4] = {w32, 64, 2, 1};
    const cuuint32_t v_box[4] = {w32, 128, 1, 1};
    bool ok = make_map(&m.k, dt, a.slab, 4, dims, strides, k_box);
    m.v = m.k;
    if (F8)
        ok = ok && make_map(&m.v, dt, a.slab, 4, dims, strides, v_box);
    // the 64 rope columns: 128-byte rows (bf16), or 64-byte ones with their swizzle
    const cuuint64_t r_dims[3] = {(cuuint64_t)kRow, (cuuint64_t)kPageTokens, (cuuint64_t)a.num_pages};
    const cuuint64_t r_str[2] = {kRow * es, (cuuint64_t)a.page_stride * es};
    const cuuint32_t r_box[3] = {64, 64, 1};
    const CUtensorMapSwizzle r_sw = F8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    ok = ok && make_map(&m.rope, dt, a.slab, 3, r_dims, r_str, r_box, r_sw);
    if (F8) {
        // [hi rows | lo rows] of 576 bytes: (column in a block, row, block)
        const cuuint64_t n_dims[3] = {128, 2 * rows, 4}, n_str[2] = {kRow, 128};
        const cuuint64_t o_dims[3] = {kRow, 2 * rows, 1}, o_str[2] = {kRow, kRow};
        const cuuint32_t n_box[3] = {128, 64, 4}, o_box[3] = {64, 64, 1};
        ok = ok && make_map(&m.qn, dt, a.q8, 3, n_dims, n_str, n_box) &&
             make_map(&m.qr, dt, a.q8, 3, o_dims, o_str, o_box, r_sw);
    } else {
        const cuuint64_t n_dims[3] = {64, rows, 8}, n_str[2] = {kLatent * 2, 128};
        const cuuint64_t o_dims[3] = {kRope, rows, 1}, o_str[2] = {kRope * 2, kRope * 2};
        const cuuint32_t n_box[3] = {64, 64, 8}, o_box[3] = {64, 64, 1};
        ok = ok && make_map(&m.qn, dt, a.q_nope, 3, n_dims, n_str, n_box) &&
             make_map(&m.qr, dt, a.q_rope, 3, o_dims, o_str, o_box);
    }
    if (!ok)
        return cudaErrorInvalidValue;
    // once per device: the attribute stays with the function
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit == 0 || (set.load(std::memory_order_relaxed) & bit) == 0) {
        err = cudaFuncSetAttribute(shared_decode_kernel<F8>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kShSmem);
        if (err != cudaSuccess)
            return err;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
    cfg.blockDim = dim3(kShThreads);
    cfg.dynamicSmemBytes = (size_t)kShSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SharedArgs b = a;
    // the accumulator's truncation is given back (see plmla_mass.cu): 4 units of 2^-23 for a
    // chain of 36 bf16 MMAs, 1 for E4M3's
    b.scale_log2 = (float)((double)a.scale * kLog2e * (1.0 + (F8 ? 1.0 : 4.0) * 0x1p-23));
    err = cudaLaunchKernelEx(&cfg, shared_decode_kernel<F8>, m, b);
    if (err != cudaSuccess)
        return err;
    // (blocks of the form for few rows: an SM holds two)
    const unsigned groups = (unsigned)((rows + 31) / 32);
    const bool few = groups * 8 <= 2u * (unsigned)sms;
    cudaLaunchConfig_t mc = {};
    mc.gridDim = dim3(groups * (few ? 8 : 4));
    mc.blockDim = dim3(few ? 512 : 256);
    mc.stream = stream;
    mc.attrs = attr + 1;
    mc.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&mc, shared_merge_kernel<8, 2>, b, sms / 2)
               : cudaLaunchKernelEx(&mc, shared_merge_kernel<16, 1>, b, sms / 2);
}

}  // namespace

int64_t shared_slots(int num_reqs, int rows, int num_groups, int sms)
{
    const int64_t total = (int64_t)num_reqs * rows;
    return total / kShRows + num_groups + (int64_t)num_reqs * ((rows + kShRows - 1) / kShRows) +
           sms / 2;
}

cudaError_t launch_shared(const SharedArgs &a, int sms, cudaStream_t stream)
{
    const int most = a.num_reqs > a.num_groups ? a.num_reqs : a.num_groups;
    PlanBuffers queries = {};
    int threads = (most + 31) / 32 * 32, blocks = 1;
    if (a.q8 != nullptr) {
        queries.q_nope = a.q_nope;
        queries.q_rope = a.q_rope;
        queries.q8 = a.q8;
        queries.qexp = a.qexp;
        queries.q_rows = a.num_reqs * a.rows;
        threads = threads < 256 ? 256 : threads;
        blocks += (queries.q_rows + threads / 32 - 1) / (threads / 32);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, shared_plan_kernel, a, queries);
    if (err != cudaSuccess)
        return err;
    return a.q8 != nullptr ? launch_decode<true>(a, sms, stream)
                           : launch_decode<false>(a, sms, stream);
}

}  // namespace plmla
