// plmla_mass.cu -- accumulated attention weight of every cached token, on the
// 5th-generation tensor cores (tcgen05 + TMEM) with TMA page loads, for sm_103a.
//
//   mass[r, t] <- decay mass[r, t] + sum_{rows (j, h): t < L_r - (n_q - 1 - j)}
//                                    exp(scale q_{r,j,h} . x_t - lse_{r,j,h})
//
// With the decode's lse in hand the weights need no running maximum: one pass
// recomputes each score and sums its exponential, and token t's sum depends on
// token t's row alone.  So the transposed form of the decode fits again,
//   S^T[t, row] = K_tile[t, 0:576] . Q[row, 0:576]   (M = 128 tokens),
// with a token per TMEM lane: a thread sums its lane's columns in fp32, with no
// exchange between threads, and rows of a page past the history (stale data,
// NaN) stay in their own lanes, which are not stored.
//
// Work.  Tiles of 128 tokens (always inside one page), numbered through the
// requests, are dealt to persistent workers (a CTA, or a pair of CTAs with a tile
// each) in equal contiguous runs; the CTA that has a tile writes its tokens, so
// there are no atomics and the result does not depend on timing.  The form goes by
// the query rows per request (n_q * heads):
//   up to 128 rows  one CTA; Q of the request is resident (rows x 1152 B) and the
//                   tiles stream through a ring of 16 KB column blocks: each KV
//                   byte is read once and bounds the kernel (E4M3 in pairs with a query
//                   part in each CTA streamed 14% slower: 135 us against 118 us for 32
//                   histories of 30,000 tokens at 128 rows);
//   up to 256       a CTA pair (cta_group::2, M = 256 tokens): Q is resident in
//                   halves, one in each CTA, the tiles stream;
//   more            a CTA pair; its two tiles are resident and the query rows
//                   stream past them from L2 in chunks of 256, half into each CTA:
//                   the tensor cores bound the kernel.  The next tiles are
//                   prefetched into L2 meanwhile.
// In a pair every SM fetches only half of the query rows that its tensor cores
// multiply, and each operand byte in shared memory serves twice the products: with
// one CTA and N = 128 shared memory and L2 bounded the kernel at 40% of the bf16
// peak.  E4M3 pages take the two-part query of the FP8 decode: the hi and the lo
// part multiply the same tile into one accumulator.
//
// Warp roles (320 threads): warp 0 = producer, warp 1 = MMA issuer (of the pair's
// even CTA) and TMEM owner, warps 2..9 = two groups of four that take the (tile,
// row chunk) units in turn.  In a pair both producers' copies complete on the even
// CTA's barriers, and MMA commits release slots and publish accumulators in both.
// Every mbarrier wait is bounded as in the decode; a wait that gives up stops the
// CTA's stores and sets the status word, and cluster barriers keep both CTAs of a
// pair until neither can touch the other.
#include <math.h>

#include "plmla_ptx.cuh"

namespace plmla {
namespace {

constexpr int kMassThreads = 320;
constexpr int kMassSlot = kTile * 128;          // ring slot: 128 rows of 128 bytes
constexpr int kMassMaxSlots = 12;
constexpr int kMassChunk = 128;                 // query rows of one MMA per CTA
constexpr int kMassCols = 512;                  // TMEM columns: two buffers of 256
constexpr int kMassSmem = 232448;
constexpr double kLog2e = 1.4426950408889634074;

struct MassBars {
    uint64_t full[kMassMaxSlots], empty[kMassMaxSlots];   // ring
    uint64_t k_full[9], k_empty[9];                       // resident tile, per column block
    uint64_t q_full, q_empty;                             // resident queries
    uint64_t s_full[2], s_free[2];                        // accumulators
    uint64_t drain;
};

// Small on purpose: with bf16 pages it leaves room for a fifth ring slot beside 147
// KB of resident operand.
template <bool F8>
struct MassMisc {
    MassBars bars;
    uint32_t tmem;
    int abort, status;
    int first_req, first_step;          // this worker's first request, and its first step
    alignas(16) float neg_lse[2][2 * kMassChunk];             // [group] -lse log2 e of the rows
    alignas(16) float factor[F8 ? 2 : 1][F8 ? 2 * kMassChunk : 4];  // scale log2 e kv_scale 2^e
    float part[kTile];                  // second group's sums of a tile
};

// Column blocks of one 576-wide row: 9 of 64 bf16, or 5 of 128 E4M3 bytes (the
// last one half empty), and the 32-byte K steps in each.
template <bool F8>
struct MassFmt {
    static constexpr int blocks = F8 ? 5 : 9;
    static constexpr int step = F8 ? 128 : 64;
    static constexpr int parts = F8 ? 2 : 1;                  // query parts (hi, lo)
    static constexpr int tile_bytes = blocks * kMassSlot;
    // the order of the products: bf16 takes the rope block in the middle (see kMassShort)
    __device__ static int block(int i)
    {
        return F8 || i < blocks / 2 ? i : i == blocks / 2 ? blocks - 1 : i - 1;
    }
    __device__ static int mmas(int block) { return F8 && block == 4 ? 2 : 4; }
};

__device__ __forceinline__ uint32_t bar_of(const uint64_t &b) { return smem_u32(&b); }

// Position in the request-major order of steps: step g of the whole is step g -
// first of request r.
struct StepWalk {
    const int32_t *lens;
    int64_t cap;                        // tokens that a row of mass and of pages hold
    int span, r, first, end;
    __device__ int steps(int r) const
    {
        const int64_t L = lens[r];
        return L <= 0 ? 0 : (int)((min(L, cap) + span - 1) / span);
    }
    __device__ void begin(int r0, int f)
    {
        r = r0;
        first = f;
        end = f + steps(r0);
    }
    __device__ int local(int g)
    {
        while (g >= end) {
            first = end;
            end += steps(++r);
        }
        return g - first;
    }
};

// Columns that a thread reads from TMEM at a time: two batches of SETS sets fit its
// registers.
template <int SETS>
constexpr int kMassBatch = SETS == 4 ? 8 : 16;

template <int W>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[W])
{
    if constexpr (W == 16)
        tmem_ld16(taddr, r);
    else
        tmem_ld8(taddr, r);
}

// Adds the weights of W columns (scores in SETS column sets) of this thread's token to
// sum; MASKED: of the columns from `first` on.
template <bool F8, int SETS, bool MASKED, int W>
__device__ __forceinline__ void add_weights(const uint32_t (&v)[SETS][W], const float4 *neg,
                                            const float4 *fac, float scale_log2, int first,
                                            float (&sum)[4])
{
#pragma unroll
    for (int e = 0; e < W / 4; ++e) {
        const float4 l4 = neg[e];
        const float l[4] = {l4.x, l4.y, l4.z, l4.w};
        float f[4] = {scale_log2, scale_log2, scale_log2, scale_log2};
        if constexpr (F8) {
            const float4 f4 = fac[e];
            f[0] = f4.x, f[1] = f4.y, f[2] = f4.z, f[3] = f4.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float score = __uint_as_float(v[0][4 * e + j]);
            if constexpr (SETS == 2)
                score += __uint_as_float(v[1][4 * e + j]);
            if constexpr (SETS == 4)
                score = (score + __uint_as_float(v[1][4 * e + j])) +
                        (__uint_as_float(v[2][4 * e + j]) + __uint_as_float(v[3][4 * e + j]));
            const float w = fast_exp2(fmaf(score, f[j], l[j]));
            sum[j] += !MASKED || 4 * e + j >= first ? w : 0.f;
        }
    }
}

// The weights of `cols` columns (a multiple of 16) from TMEM address `at`, each further
// set `half` columns on: a batch at a time, the next on its way while the last is summed.
template <bool F8, int SETS, bool MASKED>
__device__ __forceinline__ void sum_columns(uint32_t at, int half, int cols, const float4 *neg,
                                            const float4 *fac, float scale_log2, int first,
                                            float (&sum)[4])
{
    constexpr int W = kMassBatch<SETS>;
    uint32_t x[SETS][W], y[SETS][W];
    auto fetch = [&](int c, uint32_t(&v)[SETS][W]) {
#pragma unroll
        for (int i = 0; i < SETS; ++i)
            tmem_ld_cols<W>(at + i * half + c, v[i]);
    };
    auto add = [&](int c, const uint32_t(&v)[SETS][W]) {
        add_weights<F8, SETS, MASKED, W>(v, neg + c / 4, fac + (F8 ? c / 4 : 0), scale_log2,
                                         first - c, sum);
    };
    fetch(0, x);
#pragma unroll 1
    for (int c = 0; c < cols; c += 2 * W) {
        tmem_wait_ld();
        if (c + W < cols)
            fetch(c + W, y);
        add(c, x);
        if (c + W < cols) {
            tmem_wait_ld();
            if (c + 2 * W < cols)
                fetch(c + 2 * W, x);
            add(c + W, y);
        }
    }
}

// The tensor core's fp32 accumulator truncates: every MMA of a chain takes part of a unit
// in the last place off the partial sum, always towards zero.  Where the partial sums grow
// evenly to the score, the score ends up smaller by a share of itself, kMassShort of 2^-23
// (found where the error against 64 bits is least; N(0, 1) rows, rows of unlike sizes and
// rows with a common direction agree), and the epilogue's scale gives it back.  bf16: 4
// for a chain of 36 MMAs, 2 of 18, 1 of 9; weights off by 1.5e-6 -> 1.4e-7 (2-norm; 32
// queries of 64 heads), 8.5e-7 -> 2.8e-7 (128 rows), 5.6e-7 -> 2.2e-7 (64 rows), as in
// fp32 arithmetic.  The rope block in the middle lets scores that come from the rope part
// alone grow to half of the chain too: 2.8e-7 with it, 1.4e-6 with it at the end.  E4M3
// products have few bits and mostly add up exactly: 1 for the 36 MMAs of a pair (5.3e-7 ->
// 1.2e-7), 0 for a part's 18.  A score that comes whole from the first MMAs or the last is
// off by about kMassShort of 2^-23, on either side, instead of by up to twice that.
template <bool F8, int CG, int SETS>
constexpr double kMassShort = F8 ? (CG == 2 ? 1.0 : 0.0) : 4.0 / SETS;

// CG = CTAs of a worker (1, or a pair); QRES = queries resident, tiles streaming.
// half = query rows per CTA of one MMA (N / CG) when QRES.
template <bool F8, int CG, bool QRES, int SETS>
__global__ void __launch_bounds__(kMassThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_qn,
            const __grid_constant__ CUtensorMap tm_qr, const MassArgs a, const int half,
            const int slots)
{
    using F = MassFmt<F8>;
    constexpr int kSpan = kTile * CG;                         // tokens of a worker's step
    constexpr int kWidth = kMassChunk * CG;                   // query rows of a chunk, at most
    // One CTA keeps SETS column sets that the epilogue adds: the scores of the query's
    // hi and lo part (E4M3; one MMA of N = 2 rows), or of every SETS'th column block
    // (bf16), whose shorter chains of MMAs lose less to the accumulator's truncation
    // (see kMassShort), at no cost in time.
    constexpr int kParts = F8 && CG == 2 ? 2 : 1;             // MMAs per K step, one a query part
    constexpr int kBufCols = kMassCols / 2;
    constexpr int kBufs = 2;
    static_assert(CG == 1 || SETS == 1, "column sets");

    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t s_res = smem_u32(smem);                    // resident operand
    const uint32_t res_bytes = QRES ? (uint32_t)half * 2 * kRow : (uint32_t)F::tile_bytes;
    const uint32_t s_ring = s_res + res_bytes;
    MassMisc<F8> &m =
        *reinterpret_cast<MassMisc<F8> *>(smem + res_bytes + slots * kMassSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((s_res & 1023u) != 0u) {       // cannot be with no static shared memory
        if (threadIdx.x == 0 && a.status != nullptr)
            atomicExch(a.status, 12);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(bar_of(m.bars.full[i]), 1);
            mbar_init(bar_of(m.bars.empty[i]), 1);
        }
        for (int i = 0; i < 9; ++i) {
            mbar_init(bar_of(m.bars.k_full[i]), 1);
            mbar_init(bar_of(m.bars.k_empty[i]), 1);
        }
        mbar_init(bar_of(m.bars.q_full), 1);
        mbar_init(bar_of(m.bars.q_empty), 1);
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(bar_of(m.bars.s_full[i]), 1);
            mbar_init(bar_of(m.bars.s_free[i]), 4 * CG);      // one arrival per warp of a group
        }
        mbar_init(bar_of(m.bars.drain), 1);
        m.abort = 0;
        m.status = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&m.tmem)),
                         "r"(kMassCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&m.tmem)),
                         "r"(kMassCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
    }
    const int rank = CG == 2 ? (int)cluster_rank() : 0;
    const int workers = (int)gridDim.x / CG, worker = (int)blockIdx.x / CG;
    StepWalk walk = {a.seq_lens, min(a.mass_cols, a.table_cols * kPageTokens), kSpan, 0, 0, 0};
    int g0, g1;                         // this worker's steps
    {
        // steps per request (four a thread), prefix-summed; the thread in whose
        // requests the worker's first step falls notes where.  32 bits hold the sums:
        // every token has a float of mass.
        int *warp_sum = reinterpret_cast<int *>(m.part);
        int own[4], sum = 0, bad = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * (int)threadIdx.x + e;
            own[e] = r < a.num_reqs ? walk.steps(r) : 0;
            if (r < a.num_reqs && a.seq_lens[r] > walk.cap && blockIdx.x == 0)
                bad = a.seq_lens[r] > a.table_cols * kPageTokens ? kStatusAppendPage
                                                                 : kStatusMassLength;
            sum += own[e];
        }
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            warp_sum[warp] = x;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (bad != 0)
            m.status = bad;
        x -= sum;
        int total = 0;
        for (int w = 0; w < kMassThreads / 32; ++w) {
            x += w < warp ? warp_sum[w] : 0;
            total += warp_sum[w];
        }
        g0 = total / workers * worker + min(worker, total % workers);
        g1 = g0 + total / workers + (worker < total % workers ? 1 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (x <= g0 && g0 < x + own[e]) {
                m.first_req = 4 * (int)threadIdx.x + e;
                m.first_step = x;
            }
            x += own[e];
        }
        __syncthreads();
        if (g0 < g1)
            walk.begin(m.first_req, m.first_step);
    }
    if constexpr (F8)
        asm volatile("griddepcontrol.wait;" ::: "memory");    // the split queries
    if constexpr (CG == 2)
        cluster_sync();                 // the pair's barriers are initialised
    const uint32_t tmem = m.tmem;
    const int chunks = QRES ? 1 : (a.rows + kWidth - 1) / kWidth;
    // query rows of chunk c per CTA: a pair's N is a multiple of 32 (the rows past the
    // request's are multiplied and not used)
    auto chunk_half = [&](int c) {
        if constexpr (QRES)
            return half;
        return min(kMassChunk, (a.rows - c * kWidth + 31) / 32 * 16);
    };
    // the even CTA's copy of a barrier, where the pair's copies complete
    auto lead = [&](const uint64_t &b) { return CG == 2 ? map_rank(bar_of(b), 0) : bar_of(b); };
    auto commit = [&](const uint64_t &b) {
        if constexpr (CG == 2)
            mma_commit_pair(bar_of(b));
        else
            mma_commit(bar_of(b));
    };
    volatile int *abort_flag = &m.abort;
    int32_t *status = &m.status;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        const uint64_t once = l2_policy_evict_first();
        int slot = 0, issued = 0, q_loads = 0, cur = -1;
        uint32_t phase = 0;
        bool ok = true;
        auto expect = [&](const uint64_t &b, uint32_t bytes) {
            if (rank == 0)
                mbar_arrive_expect_tx(bar_of(b), CG * bytes);
        };
        auto load_q = [&](uint32_t dst, const CUtensorMap *map, int col, int row, uint32_t bar) {
            if constexpr (CG == 2)
                tma_load_2d_pair(dst, map, col, row, bar);
            else
                tma_load_2d(dst, map, col, row, bar);
        };
        auto load_k = [&](uint32_t dst, int col, int tok, int page, uint32_t bar) {
            if constexpr (CG == 2)
                tma_load_3d_pair(dst, &tm_k, col, tok, page, bar, once);
            else
                tma_load_3d_hint(dst, &tm_k, col, tok, page, bar, once);
        };
        auto ring_slot = [&](uint32_t bytes) -> bool {
            if (!wait_bounded(bar_of(m.bars.empty[slot]), phase ^ 1, abort_flag, status, 2))
                return false;
            expect(m.bars.full[slot], bytes);
            return true;
        };
        // page and first row of this CTA's tile of step i of request r
        auto tile_at = [&](int r, int i, int *tok) -> int {
            const int64_t t = (int64_t)i * kSpan + rank * kTile;
            *tok = (int)(t % kPageTokens);
            int page = t / kPageTokens < a.table_cols
                           ? a.page_table[(int64_t)r * a.table_ld + t / kPageTokens] : 0;
            if (page < 0 || (int64_t)page >= a.num_pages)
                page = 0;                                     // reported and not stored below
            return page;
        };
        auto ring_next = [&]() {
            ++issued;
            if (++slot == slots) {
                slot = 0;
                phase ^= 1;
            }
        };
        int64_t n = 0, k_loads = 0;         // tiles so far, blocks of resident tiles issued
        for (int g = g0; g < g1 && ok; ++g, ++n) {
            const int i = walk.local(g);
            const int r = walk.r;
            int tok;
            const int page = tile_at(r, i, &tok);
            // the next step's tile comes to L2 while this one is resident
            if (!QRES && g + 1 < g1) {
                StepWalk ahead = walk;
                const int next = ahead.local(g + 1);
                int tok1;
                const int page1 = tile_at(ahead.r, next, &tok1);
#pragma unroll 1
                for (int k = 0; k < F::blocks; ++k)
                    tma_prefetch_3d(&tm_k, F::step * k, tok1, page1);
            }
            if constexpr (QRES) {
                if (r != cur) {
                    if (q_loads > 0 && !wait_bounded(bar_of(m.bars.q_empty), (q_loads - 1) & 1,
                                                     abort_flag, status, 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = lead(m.bars.q_full);
                    expect(m.bars.q_full, (uint32_t)half * 2 * kRow);
                    // E4M3: a pair keeps each part whole, one CTA the parts' rows of a
                    // column block together (the rope block's rows are 64 bytes)
                    constexpr bool stacked = F8 && CG == 1;
                    for (int p = 0; p < F::parts; ++p) {
                        const uint32_t dst = s_res + (stacked ? 0 : p * half * kRow);
                        const uint32_t pitch = half * 128 * (stacked ? 2 : 1);
                        const int at = (p * a.num_reqs + r) * a.rows + rank * half;
                        for (int k = 0; k < F::blocks - 1; ++k)
                            load_q(dst + k * pitch + (stacked ? p * half * 128 : 0), &tm_qn,
                                   F::step * k, at, bar);
                        load_q(dst + (F::blocks - 1) * pitch + (stacked ? p * half * 64 : 0), &tm_qr,
                               F8 ? kLatent : 0, at, bar);
                    }
                    ++q_loads;
                    cur = r;
                }
#pragma unroll 1
                for (int i = 0; i < F::blocks; ++i) {
                    const int k = F::block(i);
                    if (!ring_slot(kMassSlot)) {
                        ok = false;
                        break;
                    }
                    load_k(s_ring + slot * kMassSlot, F::step * k, tok, page,
                           lead(m.bars.full[slot]));
                    ring_next();
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < chunks && ok; ++c) {
                    const int row = c * kWidth + rank * chunk_half(c);
#pragma unroll 1
                    for (int i = 0; i < F::blocks && ok; ++i) {
                        const int k = F::block(i);
                        if (c == 0) {
                            if (n > 0 && !wait_bounded(bar_of(m.bars.k_empty[k]), (n - 1) & 1,
                                                       abort_flag, status, 3)) {
                                ok = false;
                                break;
                            }
                            expect(m.bars.k_full[k], kMassSlot);
                            load_k(s_res + k * kMassSlot, F::step * k, tok, page,
                                   lead(m.bars.k_full[k]));
                            ++k_loads;
                        }
                        for (int p = 0; p < F::parts; ++p) {
                            const bool rope = k == F::blocks - 1;
                            if (!ring_slot(F8 && rope ? kMassSlot / 2 : kMassSlot)) {
                                ok = false;
                                break;
                            }
                            load_q(s_ring + slot * kMassSlot, rope ? &tm_qr : &tm_qn,
                                   rope ? (F8 ? kLatent : 0) : F::step * k,
                                   (p * a.num_reqs + r) * a.rows + row, lead(m.bars.full[slot]));
                            ring_next();
                        }
                    }
                }
            }
        }
        // every issued copy lands before the CTA can exit (in a pair the even CTA waits
        // for both, and the odd one for it, at the cluster barrier below)
        if (q_loads > 0 && rank == 0)
            wait_drain(bar_of(m.bars.q_full), (q_loads - 1) & 1);
        for (int it = issued > slots ? issued - slots : 0; it < issued && rank == 0; ++it)
            wait_drain(bar_of(m.bars.full[it % slots]), (uint32_t)(it / slots) & 1u);
        for (int64_t it = k_loads > F::blocks ? k_loads - F::blocks : 0;
             it < k_loads && rank == 0; ++it)
            wait_drain(bar_of(m.bars.k_full[F::block((int)(it % F::blocks))]),
                       (uint32_t)(it / F::blocks) & 1u);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---------------------------------------------------------- MMA issuer
        int slot = 0, q_loads = 0, cur = -1;
        uint32_t phase = 0;
        int64_t u = 0, n = 0;                                 // units and tiles so far
        bool ok = true, issued = false;
        for (int g = g0; g < g1 && ok; ++g, ++n) {
            walk.local(g);
            const int r = walk.r;
            if constexpr (QRES) {
                if (r != cur) {
                    if (!wait_bounded(bar_of(m.bars.q_full), q_loads & 1, abort_flag, status, 4)) {
                        ok = false;
                        break;
                    }
                    ++q_loads;
                    cur = r;
                }
            }
#pragma unroll 1
            for (int c = 0; c < chunks && ok; ++c, ++u) {
                const int buf = (int)(u % kBufs);
                if (u >= kBufs && !wait_bounded(bar_of(m.bars.s_free[buf]),
                                                (uint32_t)(u / kBufs - 1) & 1u, abort_flag, status,
                                                5)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t idesc = idesc_for<F8>(
                    128 * CG, (F8 && CG == 1 ? 2 : CG) * chunk_half(c), false, false);
                const uint32_t d = tmem + kBufCols * buf;
                // unrolled: with the blocks' order and offsets worked out between the MMAs
                // the window of 32 queries took 361 us instead of 329
#pragma unroll
                for (int i = 0; i < F::blocks && ok; ++i) {
                    const int k = F::block(i);
                    const bool rope = k == F::blocks - 1;
                    if (QRES || c == 0) {
                        if (!wait_bounded(QRES ? bar_of(m.bars.full[slot]) : bar_of(m.bars.k_full[k]),
                                          QRES ? phase : (uint32_t)(n & 1), abort_flag, status, 6)) {
                            ok = false;
                            break;
                        }
                    }
#pragma unroll 1
                    for (int p = 0; p < kParts; ++p) {
                        uint32_t s_k, s_q;
                        if constexpr (QRES) {
                            s_k = s_ring + slot * kMassSlot;
                            s_q = s_res + p * half * kRow + k * half * 128 * (F8 && CG == 1 ? 2 : 1);
                        } else {
                            if (!wait_bounded(bar_of(m.bars.full[slot]), phase, abort_flag, status,
                                              7)) {
                                ok = false;
                                break;
                            }
                            s_k = s_res + k * kMassSlot;
                            s_q = s_ring + slot * kMassSlot;
                        }
                        tc_fence_after();
                        const uint64_t da = sdesc(s_k, 16, 1024, kSw128);
                        const uint64_t db = F8 && rope ? sdesc(s_q, 16, 512, kSw64)
                                                       : sdesc(s_q, 16, 1024, kSw128);
                        const int mmas = F::mmas(k);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (kk < mmas) {
                                if constexpr (CG == 2)
                                    mma_pair<F8>(d, da + 2 * kk, db + 2 * kk, idesc,
                                                 (i | p | kk) != 0);
                                else if constexpr (F8)
                                    mma_e4m3(d, da + 2 * kk, db + 2 * kk, idesc, (i | kk) != 0);
                                else
                                    mma_bf16(d + i % SETS * half, da + 2 * kk, db + 2 * kk, idesc,
                                             (i / SETS | kk) != 0);
                            }
                        issued = true;
                        if (!QRES || p == kParts - 1) {
                            commit(m.bars.empty[slot]);
                            if (++slot == slots) {
                                slot = 0;
                                phase ^= 1;
                            }
                        }
                    }
                    if (!QRES && ok && c == chunks - 1)
                        commit(m.bars.k_empty[k]);
                }
                if (!ok)
                    break;
                commit(m.bars.s_full[buf]);
            }
            if constexpr (QRES) {
                if (ok && g + 1 >= walk.end)                  // the request's last step
                    commit(m.bars.q_empty);
            }
        }
        if (issued) {
            commit(m.bars.drain);
            wait_drain(bar_of(m.bars.drain), 0);
        }
    } else if (CG == 2 && warp == 1 && lane == 0) {
        // the even CTA's commits arrive here too: the last of them comes after the others
        if (g0 < g1)
            wait_drain(bar_of(m.bars.drain), 0);
    } else if (warp >= 2) {
        // ------------------------------------------------------------ weights
        // A wait that gives up clears `ok`: the loops run on without waiting or
        // storing, so that every thread still meets the group barriers.
        const int group = (warp - 2) >> 2, quad = warp & 3;
        const int tok = 32 * quad + lane, me = ((warp - 2) & 3) * 32 + lane;
        const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16);
        int64_t u = 0;
        int cur = -1, L = 0;
        bool ok = true;
        const float scale_log2 = a.scale_log2;
        for (int g = g0; g < g1; ++g) {
            const int i = walk.local(g);
            const int r = walk.r;
            if (r != cur)
                L = a.seq_lens[r];
            const int64_t t0 = (int64_t)i * kSpan + rank * kTile, t = t0 + tok;
            // the owner of the tile's sums: the unit's group, or the first group
            const bool mine = QRES ? (u & 1) == group : group == 0;
            // (the pair's second tile may lie past the history)
            const bool inside = t0 < L && t0 / kPageTokens < a.table_cols;
            const int page =
                inside ? a.page_table[(int64_t)r * a.table_ld + t0 / kPageTokens] : 0;
            const bool page_ok = page >= 0 && (int64_t)page < a.num_pages;
            if (!page_ok && mine && me == 0)
                atomicExch(status, kStatusAppendPage);
            const bool store = mine && inside && page_ok && t < L && t < a.mass_cols;
            float *out = a.mass + (int64_t)r * a.mass_ld + t;
            const float old = store && a.decay != 0.f ? a.decay * *out : 0.f;
            // every row of the request sees the whole tile
            const bool visible = t0 + kTile <= (int64_t)L - (a.n_q - 1);
            // the token's first query row: draft j sees it from L - (n_q - 1 - j) > t on
            const int first_row =
                t < L ? max(0, (int)(t - L) + a.n_q) * a.heads : 0x7FFFFFFF;
            float acc = 0.f;
            for (int c = 0; c < chunks; ++c, ++u) {
                if ((u & 1) != group)
                    continue;
                const int cols = QRES ? a.rows : min(kWidth, a.rows - c * kWidth);
                const int row0 = c * kWidth;
                if (!QRES || r != cur) {
                    // stage the unit's rows, once the group has done with the last ones
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                    for (int e = me; e < cols; e += kTile) {
                        const int64_t at = (int64_t)r * a.rows + row0 + e;
                        const float lse = a.lse[at];
                        // a row without weights (lse -inf) adds nothing: 2^-inf
                        m.neg_lse[group][e] = isinf(lse) ? -INFINITY : -lse * (float)kLog2e;
                        if constexpr (F8)
                            m.factor[group][e] = ldexpf(scale_log2 * a.kv_scale, a.qexp[at]);
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                    cur = r;
                }
                const int buf = (int)(u % kBufs);
                if (ok && !wait_bounded(bar_of(m.bars.s_full[buf]), (uint32_t)(u / kBufs) & 1u,
                                        abort_flag, status, 8))
                    ok = false;
                tc_fence_after();
                const float4 *neg = reinterpret_cast<const float4 *>(m.neg_lse[group]);
                const float4 *fac = reinterpret_cast<const float4 *>(m.factor[F8 ? group : 0]);
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t at = taddr + kBufCols * buf;
                if (visible)
                    sum_columns<F8, SETS, false>(at, half, cols, neg, fac, scale_log2, 0, sum);
                else
                    sum_columns<F8, SETS, true>(at, half, cols, neg, fac, scale_log2,
                                                 first_row - row0, sum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_cluster(lead(m.bars.s_free[buf]));
                    else
                        mbar_arrive(bar_of(m.bars.s_free[buf]));
                }
                acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            if constexpr (!QRES) {
                if (group == 1)
                    m.part[tok] = acc;
                asm volatile("bar.sync 3, 256;" ::: "memory");
                if (group == 0)
                    acc += m.part[tok];
                asm volatile("bar.sync 3, 256;" ::: "memory");
            }
            if (store && ok && !*abort_flag)
                *out = old + acc;
        }
    }

    tc_fence_before();
    __syncthreads();
    // A pair leaves together: no copy or arrival of one CTA is on its way to the other,
    // and each has waited for its own copy of the last commit.  (Every wait above is
    // bounded, so all threads get here.)
    if constexpr (CG == 2)
        cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kMassCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kMassCols));
    }
    if (threadIdx.x == 0 && m.status != 0 && a.status != nullptr)
        atomicExch(a.status, m.status);
}

template <bool F8, int CG, bool QRES, int SETS>
cudaError_t launch_mass_form(const MassArgs &a, int sms, cudaStream_t stream)
{
    const CUtensorMapDataType dt = F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t es = F8 ? 1 : 2;
    const cuuint64_t rows = (cuuint64_t)a.num_reqs * a.rows;
    // rows of one query box: a pair splits N, a multiple of 32, in halves
    const int half = !QRES ? kMassChunk : CG == 1 ? a.rows : (a.rows + 31) / 32 * 16;
    const cuuint32_t q_rows = (cuuint32_t)half;
    CUtensorMap k, qn, qr;
    const cuuint64_t k_dims[3] = {(cuuint64_t)kRow, (cuuint64_t)kPageTokens, (cuuint64_t)a.num_pages};
    const cuuint64_t k_strides[2] = {(cuuint64_t)kRow * es, (cuuint64_t)a.page_stride * es};
    const cuuint32_t k_box[3] = {(cuuint32_t)MassFmt<F8>::step, (cuuint32_t)kTile, 1};
    bool ok = make_map(&k, dt, a.slab, 3, k_dims, k_strides, k_box);
    if (F8) {
        // [hi rows | lo rows] of 576 bytes: 128-byte boxes of the latent, a 64-byte
        // box (64-byte swizzle) of the rope part
        const cuuint64_t dims[2] = {(cuuint64_t)kRow, 2 * rows}, strides[1] = {(cuuint64_t)kRow};
        const cuuint32_t box[2] = {128, q_rows}, rope_box[2] = {64, q_rows};
        ok = ok && make_map(&qn, dt, a.q8, 2, dims, strides, box) &&
             make_map(&qr, dt, a.q8, 2, dims, strides, rope_box, CU_TENSOR_MAP_SWIZZLE_64B);
    } else {
        const cuuint64_t n_dims[2] = {(cuuint64_t)kLatent, rows}, n_str[1] = {(cuuint64_t)kLatent * 2};
        const cuuint64_t r_dims[2] = {(cuuint64_t)kRope, rows}, r_str[1] = {(cuuint64_t)kRope * 2};
        const cuuint32_t box[2] = {64, q_rows};
        ok = ok && make_map(&qn, dt, a.q_nope, 2, n_dims, n_str, box) &&
             make_map(&qr, dt, a.q_rope, 2, r_dims, r_str, box);
    }
    if (!ok)
        return cudaErrorInvalidValue;
    const int res = QRES ? half * 2 * kRow : MassFmt<F8>::tile_bytes;
    int slots = (kMassSmem - res - (int)sizeof(MassMisc<F8>)) / kMassSlot;
    slots = slots < kMassMaxSlots ? slots : kMassMaxSlots;
    const int smem = res + slots * kMassSlot + (int)sizeof(MassMisc<F8>);
    cudaError_t err = cudaFuncSetAttribute(mass_kernel<F8, CG, QRES, SETS>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kMassSmem);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / CG * CG));
    cfg.blockDim = dim3(kMassThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // E4M3 pages: CTAs start as those of the query split end, and wait for the whole split
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = F8 ? 2 : 1;
    MassArgs b = a;
    b.scale_log2 = (float)((double)a.scale * kLog2e * (1.0 + kMassShort<F8, CG, SETS> * 0x1p-23));
    return cudaLaunchKernelEx(&cfg, mass_kernel<F8, CG, QRES, SETS>, k, qn, qr, b, half, slots);
}

template <bool F8>
cudaError_t launch_mass_typed(const MassArgs &a, int sms, cudaStream_t stream)
{
    if (!F8 && a.rows <= kMassChunk / 2)
        return launch_mass_form<F8, 1, true, F8 ? 2 : 4>(a, sms, stream);
    if (a.rows <= kMassChunk)
        return launch_mass_form<F8, 1, true, 2>(a, sms, stream);
    return a.rows <= 2 * kMassChunk ? launch_mass_form<F8, 2, true, 1>(a, sms, stream)
                                    : launch_mass_form<F8, 2, false, 1>(a, sms, stream);
}

}  // namespace

cudaError_t launch_mass(const MassArgs &a, int sms, cudaStream_t stream)
{
    return a.q8 != nullptr ? launch_mass_typed<true>(a, sms, stream)
                           : launch_mass_typed<false>(a, sms, stream);
}

}  // namespace plmla
