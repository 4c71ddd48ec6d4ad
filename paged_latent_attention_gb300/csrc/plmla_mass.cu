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
// requests, are dealt to one persistent CTA per SM in equal contiguous runs; the
// CTA that has a tile writes its tokens, so there are no atomics and the result
// does not depend on timing.  Which operand stays in shared memory goes by the
// query rows per request (n_q * heads):
//   up to 128 rows  Q of the request is resident (rows x 1152 B) and the tiles
//                   stream through a ring of 16 KB column blocks: each KV byte is
//                   read once and bounds the kernel;
//   more            the tile is resident and the query rows stream past it from L2
//                   in chunks of 128: the tensor cores bound the kernel.
// Both cases issue the same MMAs (M = 128, N <= 128 rows, fp32 accumulators in
// four TMEM buffers of 128 columns).  E4M3 pages take the two-part query of the
// FP8 decode: the hi and the lo part multiply the same tile into one accumulator.
//
// Warp roles (320 threads): warp 0 = producer, warp 1 = MMA issuer and TMEM
// owner, warps 2..9 = two groups of four that take the (tile, row chunk) units in
// turn.  Every mbarrier wait is bounded as in the decode; a wait that gives up
// stops the CTA's stores and sets the status word.
#include <math.h>

#include "plmla_ptx.cuh"

namespace plmla {
namespace {

constexpr int kMassThreads = 320;
constexpr int kMassSlot = kTile * 128;          // ring slot: 128 rows of 128 bytes
constexpr int kMassMaxSlots = 12;
constexpr int kMassChunk = 128;                 // query rows of one MMA and one TMEM buffer
constexpr int kMassBufs = 4;
constexpr int kMassSmem = 232448;
constexpr double kLog2e = 1.4426950408889634074;

struct MassBars {
    uint64_t full[kMassMaxSlots], empty[kMassMaxSlots];   // ring
    uint64_t k_full[9], k_empty[9];                       // resident tile, per column block
    uint64_t q_full, q_empty;                             // resident queries
    uint64_t s_full[kMassBufs], s_free[kMassBufs];        // accumulators
    uint64_t drain;
};

struct MassMisc {
    MassBars bars;
    uint32_t tmem;
    int abort, status;
    alignas(16) float neg_lse[2][2][kMassChunk];    // [group][buffer] -lse log2 e of the unit's rows
    float factor[2][2][kMassChunk];     // E4M3: scale log2 e kv_scale 2^e of the row
    int limit[2][2][kMassChunk];        // tokens the row sees
    float part[2][kTile];               // second group's sums of a tile
    int64_t warp_sum[kMassThreads / 32];
    int64_t start[kMaxReqs + 1];        // first tile of each request
};

// Column blocks of one 576-wide row: 9 of 64 bf16, or 5 of 128 E4M3 bytes (the
// last one half empty), and the 32-byte K steps in each.
template <bool F8>
struct MassFmt {
    static constexpr int blocks = F8 ? 5 : 9;
    static constexpr int step = F8 ? 128 : 64;
    static constexpr int parts = F8 ? 2 : 1;                  // query parts (hi, lo)
    static constexpr int tile_bytes = blocks * kMassSlot;
    __device__ static int mmas(int block) { return F8 && block == 4 ? 2 : 4; }
};

__device__ __forceinline__ uint32_t bar_of(const uint64_t &b) { return smem_u32(&b); }

// Position in the request-major tile order.
struct TileWalk {
    const int64_t *start;
    int r;
    __device__ int64_t local(int64_t g)          // tile g's index within its request r
    {
        while (g >= start[r + 1])
            ++r;
        return g - start[r];
    }
};

template <bool F8, bool QRES>
__global__ void __launch_bounds__(kMassThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_qn,
            const __grid_constant__ CUtensorMap tm_qr, const MassArgs a, const int slots)
{
    using F = MassFmt<F8>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t s_res = smem_u32(smem);                    // resident operand
    const uint32_t res_bytes = QRES ? (uint32_t)a.rows * 2 * kRow : (uint32_t)F::tile_bytes;
    const uint32_t s_ring = s_res + res_bytes;
    MassMisc &m = *reinterpret_cast<MassMisc *>(smem + res_bytes + slots * kMassSlot);
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
        for (int i = 0; i < kMassBufs; ++i) {
            mbar_init(bar_of(m.bars.s_full[i]), 1);
            mbar_init(bar_of(m.bars.s_free[i]), 4);           // one arrival per warp of a group
        }
        mbar_init(bar_of(m.bars.drain), 1);
        m.abort = 0;
        m.status = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&m.tmem)),
                     "r"(kMassBufs * kMassChunk));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // tiles per request, prefix-summed; four requests a thread
    {
        const int64_t cap = min(a.mass_cols, a.table_ld * kPageTokens);
        int64_t own[4], sum = 0;
        int bad = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * (int)threadIdx.x + e;
            const int64_t L = r < a.num_reqs ? (int64_t)a.seq_lens[r] : 0;
            if (L > cap && blockIdx.x == 0)
                bad = L > a.table_ld * kPageTokens ? kStatusAppendPage : kStatusMassLength;
            own[e] = L <= 0 ? 0 : (min(L, cap) + kTile - 1) / kTile;
            sum += own[e];
        }
        int64_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            m.warp_sum[warp] = x;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (bad != 0)
            m.status = bad;
        x -= sum;
        for (int w = 0; w < warp; ++w)
            x += m.warp_sum[w];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * (int)threadIdx.x + e;
            if (r <= a.num_reqs)
                m.start[r] = x;
            x += own[e];
        }
        __syncthreads();
    }
    const uint32_t tmem = m.tmem;
    const int64_t total = m.start[a.num_reqs];
    const int64_t g0 = total / gridDim.x * blockIdx.x + min((int64_t)blockIdx.x, total % gridDim.x);
    const int64_t g1 = g0 + total / gridDim.x + (blockIdx.x < total % gridDim.x ? 1 : 0);
    TileWalk walk = {m.start, 0};
    const int chunks = QRES ? 1 : (a.rows + kMassChunk - 1) / kMassChunk;
    volatile int *abort_flag = &m.abort;
    int32_t *status = &m.status;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        const uint64_t once = l2_policy_evict_first();
        int slot = 0, issued = 0, q_loads = 0, cur = -1;
        uint32_t phase = 0;
        bool ok = true;
        auto ring_slot = [&](uint32_t bytes) -> bool {
            if (!wait_bounded(bar_of(m.bars.empty[slot]), phase ^ 1, abort_flag, status, 2))
                return false;
            mbar_arrive_expect_tx(bar_of(m.bars.full[slot]), bytes);
            return true;
        };
        auto ring_next = [&]() {
            ++issued;
            if (++slot == slots) {
                slot = 0;
                phase ^= 1;
            }
        };
        int64_t n = 0, k_loads = 0;         // tiles so far, blocks of resident tiles issued
        for (int64_t g = g0; g < g1 && ok; ++g, ++n) {
            const int64_t i = walk.local(g);
            const int r = walk.r;
            int page = a.page_table[(int64_t)r * a.table_ld + i * kTile / kPageTokens];
            if (page < 0 || (int64_t)page >= a.num_pages)
                page = 0;                                     // reported and not stored below
            const int tok = (int)(i * kTile % kPageTokens);
            if constexpr (QRES) {
                if (r != cur) {
                    if (q_loads > 0 && !wait_bounded(bar_of(m.bars.q_empty), (q_loads - 1) & 1,
                                                     abort_flag, status, 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = bar_of(m.bars.q_full);
                    const int row = r * a.rows;
                    mbar_arrive_expect_tx(bar, (uint32_t)a.rows * 2 * kRow);
                    for (int p = 0; p < F::parts; ++p) {
                        const uint32_t dst = s_res + p * a.rows * kRow;
                        const int at = row + p * a.num_reqs * a.rows;
                        for (int k = 0; k < F::blocks - 1; ++k)
                            tma_load_2d(dst + k * a.rows * 128, &tm_qn, F::step * k, at, bar);
                        tma_load_2d(dst + (F::blocks - 1) * a.rows * 128, &tm_qr,
                                    F8 ? kLatent : 0, at, bar);
                    }
                    ++q_loads;
                    cur = r;
                }
#pragma unroll 1
                for (int k = 0; k < F::blocks; ++k) {
                    if (!ring_slot(kMassSlot)) {
                        ok = false;
                        break;
                    }
                    tma_load_3d_hint(s_ring + slot * kMassSlot, &tm_k, F::step * k, tok, page,
                                     bar_of(m.bars.full[slot]), once);
                    ring_next();
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < chunks && ok; ++c) {
#pragma unroll 1
                    for (int k = 0; k < F::blocks && ok; ++k) {
                        if (c == 0) {
                            const uint32_t bar = bar_of(m.bars.k_full[k]);
                            if (n > 0 && !wait_bounded(bar_of(m.bars.k_empty[k]), (n - 1) & 1,
                                                       abort_flag, status, 3)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(bar, kMassSlot);
                            tma_load_3d_hint(s_res + k * kMassSlot, &tm_k, F::step * k, tok, page,
                                             bar, once);
                            ++k_loads;
                        }
                        for (int p = 0; p < F::parts; ++p) {
                            const bool rope = k == F::blocks - 1;
                            if (!ring_slot(F8 && rope ? kMassSlot / 2 : kMassSlot)) {
                                ok = false;
                                break;
                            }
                            const int at = r * a.rows + c * kMassChunk + p * a.num_reqs * a.rows;
                            tma_load_2d(s_ring + slot * kMassSlot, rope ? &tm_qr : &tm_qn,
                                        rope ? (F8 ? kLatent : 0) : F::step * k, at,
                                        bar_of(m.bars.full[slot]));
                            ring_next();
                        }
                    }
                }
            }
        }
        // every issued copy lands before the CTA can exit
        if (q_loads > 0)
            wait_drain(bar_of(m.bars.q_full), (q_loads - 1) & 1);
        for (int it = issued > slots ? issued - slots : 0; it < issued; ++it)
            wait_drain(bar_of(m.bars.full[it % slots]), (uint32_t)(it / slots) & 1u);
        for (int64_t it = k_loads > F::blocks ? k_loads - F::blocks : 0; it < k_loads; ++it)
            wait_drain(bar_of(m.bars.k_full[it % F::blocks]), (uint32_t)(it / F::blocks) & 1u);
    } else if (warp == 1 && lane == 0) {
        // ---------------------------------------------------------- MMA issuer
        int slot = 0, q_loads = 0, cur = -1;
        uint32_t phase = 0;
        int64_t u = 0, n = 0;                                 // units and tiles so far
        bool ok = true, issued = false;
        for (int64_t g = g0; g < g1 && ok; ++g, ++n) {
            const int64_t i = walk.local(g);
            const int r = walk.r;
            (void)i;
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
                const int buf = (int)(u % kMassBufs);
                if (u >= kMassBufs && !wait_bounded(bar_of(m.bars.s_free[buf]),
                                                    (uint32_t)(u / kMassBufs - 1) & 1u, abort_flag,
                                                    status, 5)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int cols = QRES ? a.rows : min(kMassChunk, a.rows - c * kMassChunk);
                const uint32_t idesc = idesc_for<F8>(128, cols, false, false);
                const uint32_t d = tmem + kMassChunk * buf;
#pragma unroll 1
                for (int k = 0; k < F::blocks && ok; ++k) {
                    const bool rope = k == F::blocks - 1;
                    if (QRES || c == 0) {
                        if (!wait_bounded(QRES ? bar_of(m.bars.full[slot]) : bar_of(m.bars.k_full[k]),
                                          QRES ? phase : (uint32_t)(n & 1), abort_flag, status, 6)) {
                            ok = false;
                            break;
                        }
                    }
#pragma unroll 1
                    for (int p = 0; p < F::parts; ++p) {
                        uint32_t s_k, s_q;
                        if constexpr (QRES) {
                            s_k = s_ring + slot * kMassSlot;
                            s_q = s_res + p * a.rows * kRow + k * a.rows * 128;
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
                            if (kk < mmas)
                                mma<F8>(d, da + 2 * kk, db + 2 * kk, idesc, (k | p | kk) != 0);
                        issued = true;
                        if (!QRES || p == F::parts - 1) {
                            mma_commit(bar_of(m.bars.empty[slot]));
                            if (++slot == slots) {
                                slot = 0;
                                phase ^= 1;
                            }
                        }
                    }
                    if (!QRES && ok && c == chunks - 1)
                        mma_commit(bar_of(m.bars.k_empty[k]));
                }
                if (!ok)
                    break;
                mma_commit(bar_of(m.bars.s_full[buf]));
            }
            if constexpr (QRES) {
                if (ok && g + 1 >= m.start[r + 1])            // the request's last tile
                    mma_commit(bar_of(m.bars.q_empty));
            }
        }
        if (issued) {
            mma_commit(bar_of(m.bars.drain));
            wait_drain(bar_of(m.bars.drain), 0);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ weights
        // A wait that gives up clears `ok`: the loops run on without waiting or
        // storing, so that every thread still meets the group barriers.
        const int group = (warp - 2) >> 2, quad = warp & 3;
        const int tok = 32 * quad + lane, me = ((warp - 2) & 3) * 32 + lane;
        const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16);
        int64_t u = 0, n = 0;
        int staged = 0, cur = -1, L = 0;
        bool ok = true;
        const float scale_log2 = a.scale_log2;
        for (int64_t g = g0; g < g1; ++g, ++n) {
            const int64_t i = walk.local(g);
            const int r = walk.r;
            if (r != cur)
                L = a.seq_lens[r];
            const int64_t t = i * kTile + tok;
            // the owner of the tile's sums: the unit's group, or the first group
            const bool mine = QRES ? (u & 1) == group : group == 0;
            const int page = a.page_table[(int64_t)r * a.table_ld + i * kTile / kPageTokens];
            const bool page_ok = page >= 0 && (int64_t)page < a.num_pages;
            if (!page_ok && mine && me == 0)
                atomicExch(status, kStatusAppendPage);
            const bool store = mine && page_ok && t < L && t < a.mass_cols;
            float *out = a.mass + (int64_t)r * a.mass_ld + t;
            const float old = store && a.decay != 0.f ? a.decay * *out : 0.f;
            // every row of the request sees the whole tile
            const bool visible = (i + 1) * kTile <= (int64_t)L - (a.n_q - 1);
            float acc = 0.f;
            for (int c = 0; c < chunks; ++c, ++u) {
                if ((u & 1) != group)
                    continue;
                const int cols = QRES ? a.rows : min(kMassChunk, a.rows - c * kMassChunk);
                if (!QRES || r != cur) {
                    // stage the unit's rows; the other buffer may still be read
                    ++staged;
                    const int b = staged & 1;
                    if (me < cols) {
                        const int row = c * kMassChunk + me;
                        const int64_t at = (int64_t)r * a.rows + row;
                        const float lse = a.lse[at];
                        // a row without weights (lse -inf) adds nothing: 2^-inf
                        m.neg_lse[group][b][me] =
                            isinf(lse) ? -INFINITY : -lse * (float)kLog2e;
                        m.limit[group][b][me] = L - (a.n_q - 1 - row / a.heads);
                        if constexpr (F8)
                            m.factor[group][b][me] = ldexpf(scale_log2 * a.kv_scale, a.qexp[at]);
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                    cur = r;
                }
                const int buf = (int)(u % kMassBufs);
                if (ok && !wait_bounded(bar_of(m.bars.s_full[buf]), (uint32_t)(u / kMassBufs) & 1u,
                                        abort_flag, status, 8))
                    ok = false;
                tc_fence_after();
                const float4 *neg = reinterpret_cast<const float4 *>(m.neg_lse[group][staged & 1]);
                const float4 *fac = reinterpret_cast<const float4 *>(m.factor[group][staged & 1]);
                const int4 *lim = reinterpret_cast<const int4 *>(m.limit[group][staged & 1]);
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t x[16];
                    tmem_ld16(taddr + kMassChunk * buf + c0, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 l4 = neg[c0 / 4 + e];
                        float f[4] = {scale_log2, scale_log2, scale_log2, scale_log2};
                        if constexpr (F8) {
                            const float4 f4 = fac[c0 / 4 + e];
                            f[0] = f4.x, f[1] = f4.y, f[2] = f4.z, f[3] = f4.w;
                        }
                        float w[4];
                        w[0] = fast_exp2(fmaf(__uint_as_float(x[4 * e]), f[0], l4.x));
                        w[1] = fast_exp2(fmaf(__uint_as_float(x[4 * e + 1]), f[1], l4.y));
                        w[2] = fast_exp2(fmaf(__uint_as_float(x[4 * e + 2]), f[2], l4.z));
                        w[3] = fast_exp2(fmaf(__uint_as_float(x[4 * e + 3]), f[3], l4.w));
                        if (!visible) {
                            const int4 v = lim[c0 / 4 + e];
                            w[0] = t < v.x ? w[0] : 0.f;
                            w[1] = t < v.y ? w[1] : 0.f;
                            w[2] = t < v.z ? w[2] : 0.f;
                            w[3] = t < v.w ? w[3] : 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sum[j] += w[j];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_of(m.bars.s_free[buf]));
                acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            if constexpr (!QRES) {
                if (group == 1)
                    m.part[n & 1][tok] = acc;
                asm volatile("bar.sync 3, 256;" ::: "memory");
                if (group == 0)
                    acc += m.part[n & 1][tok];
            }
            if (store && ok && !*abort_flag)
                *out = old + acc;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kMassBufs * kMassChunk));
    }
    if (threadIdx.x == 0 && m.status != 0 && a.status != nullptr)
        atomicExch(a.status, m.status);
}

template <bool F8, bool QRES>
cudaError_t launch_mass_mode(const MassArgs &a, int sms, cudaStream_t stream)
{
    const CUtensorMapDataType dt = F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t es = F8 ? 1 : 2;
    const cuuint64_t rows = (cuuint64_t)a.num_reqs * a.rows;
    const cuuint32_t q_rows = QRES ? (cuuint32_t)a.rows : (cuuint32_t)kMassChunk;
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
    const int res = QRES ? a.rows * 2 * kRow : MassFmt<F8>::tile_bytes;
    int slots = (kMassSmem - res - (int)sizeof(MassMisc)) / kMassSlot;
    slots = slots < kMassMaxSlots ? slots : kMassMaxSlots;
    const int smem = res + slots * kMassSlot + (int)sizeof(MassMisc);
    cudaError_t err = cudaFuncSetAttribute(mass_kernel<F8, QRES>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kMassSmem);
    if (err != cudaSuccess)
        return err;
    mass_kernel<F8, QRES><<<sms, kMassThreads, smem, stream>>>(k, qn, qr, a, slots);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mass(const MassArgs &a, int sms, cudaStream_t stream)
{
    const bool resident = a.rows <= kMassChunk;
    if (a.q8 != nullptr)
        return resident ? launch_mass_mode<true, true>(a, sms, stream)
                        : launch_mass_mode<true, false>(a, sms, stream);
    return resident ? launch_mass_mode<false, true>(a, sms, stream)
                    : launch_mass_mode<false, false>(a, sms, stream);
}

}  // namespace plmla
