// plmla_evict.cu -- holding a cache to a budget: which tokens of each history
// stay (the heaviest by accumulated attention weight, after the scheme of Zhang
// et al., "H2O: Heavy-Hitter Oracle", 2023), and the copy of their rows into
// fresh pages.
#include <cooperative_groups.h>

#include "plmla_internal.cuh"

namespace plmla {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
//
// Of request r's L tokens the first `sink`, the last `recent` and, of those
// between, the k = keep - sink - recent heaviest stay; equal weights go to the
// lower index.  A weight maps to a 32-bit key in the same order (NaN below all,
// -0 = +0), and the k-th largest key T is found by radix selection: histograms
// of 11, 11 and 10 bits, each over the keys that match the digits found so far.
// Every key above T stays, and the first of those equal to T until k is reached.
//
// One thread-block cluster per request: each CTA holds a contiguous slice of the
// candidates, the histograms meet through distributed shared memory, and a CTA's
// output offset is the sum of the counts before it (which its histograms give),
// so the indices come out in ascending order without a sort.  The first
// kSelCache keys of a slice stay in shared memory after their first read.
//
// Weights are read four at a time (aligned groups; the ends of a slice element by
// element).  The first histogram of a large CTA has four copies, interleaved so that
// they lie in different banks: its digit is the sign, the exponent and two bits, and
// weights crowd into a few of those bins.

constexpr int kSelThreads = 1024;             // of a CTA; rows of at most kSelSmall weights
constexpr int kSelSmall = 4096, kSelSmallThreads = 256;   // take smaller ones, several an SM
constexpr int kSelBins = 2048;
constexpr int kSelCoarse = kSelBins / 64;     // sums of 64 bins
constexpr int kSelBatch = 4;                  // groups of four that a thread has in flight
constexpr int kSelCache = 38912;              // keys of a slice kept in shared memory
constexpr int kSelChunk = 8192;               // groups of four written out at a time
constexpr int kSelMaxCluster = 16;

struct SelectArgs {
    const float *mass;
    int64_t mass_ld, mass_cols;
    const int32_t *seq_lens;
    int keep, sink, recent;
    int32_t *kept;
    int64_t kept_ld;
    int32_t *kept_lens;
    int cache_groups;              // groups that the dynamic shared memory holds
};

template <int NT>
struct SelectSmem {
    static constexpr int copies = NT >= kSelThreads ? 4 : 1;   // of hist[0]
    // (arrays read in vectors are aligned for them)
    alignas(16) uint32_t hist[3][kSelBins];    // this CTA's, one per digit, read by the whole cluster
    alignas(16) uint32_t copied[copies > 1 ? kSelBins * copies : 4];
    uint32_t coarse[3][kSelCoarse];// sums of 64 bins each, read by the whole cluster
    uint32_t warp_sum[2][32];
    uint32_t counts[2];            // this CTA's keys above T and equal to T, read by the cluster
    uint32_t peer[kSelMaxCluster * 32];            // coarse sums, from every CTA
    alignas(16) uint32_t peer_bins[kSelMaxCluster * 64];   // 64 bins, from every CTA
    uint32_t seg[kSelChunk / 32];  // counts, then offsets, of 32 groups (above | equal << 16)
    unsigned char flags[kSelChunk];// per group: which of its four stay (above | equal << 4)
};

// Order-preserving key: larger weight, larger key; NaN 0, -0 as +0 (-0 + 0 = +0).
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return w == w ? key : 0u;
}

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    return x;
}

// Exclusive prefix sum over the block's threads, and the total.  One barrier; the
// caller alternates between two `warp_sum` arrays.
template <int NT>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sum, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t x = warp_inclusive(v, lane);
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    const uint32_t w = warp_inclusive(lane < NT / 32 ? warp_sum[lane] : 0u, lane);
    *total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0u) + x - v;
}

template <int NT>
__global__ void __launch_bounds__(NT) select_kernel(const SelectArgs a)
{
    extern __shared__ uint4 cache[];
    using Smem = SelectSmem<NT>;
    __shared__ Smem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int r = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t L64 = a.seq_lens[r];
    {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int b = tid; b < 3 * kSelBins / 4; b += NT)
            reinterpret_cast<uint4 *>(sm.hist)[b] = zero;
        for (int b = tid; b < kSelBins * Smem::copies / 4 && Smem::copies > 1; b += NT)
            reinterpret_cast<uint4 *>(sm.copied)[b] = zero;
    }
    const int L = (int)(L64 < 0 ? 0 : (L64 > a.mass_cols ? a.mass_cols : L64));
    const float *mass = a.mass + (int64_t)r * a.mass_ld;
    int32_t *kept = a.kept + (int64_t)r * a.kept_ld;
    if (L <= a.keep) {             // everything stays
        for (int i = me * NT + tid; i < L; i += C * NT)
            kept[i] = i;
        if (me == 0 && tid == 0)
            a.kept_lens[r] = L;
        return;                    // the whole cluster takes this branch
    }
    const int hi = L - a.recent;
    const uint32_t k = (uint32_t)(a.keep - a.sink - a.recent);
    for (int i = me * NT + tid; i < a.sink + a.recent; i += C * NT) {
        if (i < a.sink)
            kept[i] = i;
        else
            kept[a.keep - a.recent + (i - a.sink)] = hi + (i - a.sink);
    }
    if (me == 0 && tid == 0)
        a.kept_lens[r] = a.keep;
    if (k == 0)
        return;

    // candidates [sink, hi) in groups of four aligned weights: group g holds
    // tokens 4 g - skew .. 4 g - skew + 3
    const uint32_t skew = (uint32_t)(reinterpret_cast<uintptr_t>(mass) / 4) & 3u;
    const uint32_t v0 = (uint32_t)a.sink + skew, v1 = (uint32_t)hi + skew;
    const uint32_t first = v0 / 4, groups = (v1 + 3) / 4 - first;
    const uint32_t per = (groups + C - 1) / C;
    const uint32_t g0 = first + min(groups, me * per), g1 = first + min(groups, (me + 1) * per);
    // which of group g's elements are candidates: all but in the outermost groups
    const uint32_t last = first + groups - 1;
    const uint32_t first_bits = 0xFu & (0xFu << (v0 - 4 * first));
    const uint32_t last_bits = 0xFu >> (4 * last + 4 - v1);
    auto valid = [&](uint32_t g) -> uint32_t {
        return (g == first ? first_bits : 0xFu) & (g == last ? last_bits : 0xFu);
    };
    auto fetch = [&](uint32_t g) -> uint4 {
        const float *p = mass + ((int64_t)4 * g - skew);
        const uint32_t bits = valid(g);
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (bits == 0xFu) {
            w = *reinterpret_cast<const float4 *>(p);
        } else {
            if (bits & 1u) w.x = p[0];
            if (bits & 2u) w.y = p[1];
            if (bits & 4u) w.z = p[2];
            if (bits & 8u) w.w = p[3];
        }
        return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
    };
    const uint32_t cached = (uint32_t)a.cache_groups;
    auto keys = [&](uint32_t g) -> uint4 { return g - g0 < cached ? cache[g - g0] : fetch(g); };
    // f(g, keys of group g) over this thread's groups of [lo, hi), the loads of
    // kSelBatch groups in flight together
    auto batched = [&](uint32_t lo, uint32_t hi, auto load, auto f) {
        for (uint32_t g = lo + tid; g < hi; g += kSelBatch * NT) {
            uint4 q[kSelBatch];
#pragma unroll
            for (int j = 0; j < kSelBatch; ++j)
                if (g + j * NT < hi)
                    q[j] = load(g + j * NT);
#pragma unroll
            for (int j = 0; j < kSelBatch; ++j)
                if (g + j * NT < hi)
                    f(g + j * NT, q[j]);
        }
    };

    // first digit, filling the cache
    __syncthreads();
    {
        uint32_t *hist = Smem::copies > 1 ? sm.copied + lane % Smem::copies : sm.hist[0];
        batched(g0, g1, fetch, [&](uint32_t g, const uint4 &q) {
            const uint32_t bits = valid(g);
            if (g - g0 < cached)
                cache[g - g0] = q;
            if (bits & 1u) atomicAdd(&hist[(q.x >> 21) * Smem::copies], 1u);
            if (bits & 2u) atomicAdd(&hist[(q.y >> 21) * Smem::copies], 1u);
            if (bits & 4u) atomicAdd(&hist[(q.z >> 21) * Smem::copies], 1u);
            if (bits & 8u) atomicAdd(&hist[(q.w >> 21) * Smem::copies], 1u);
        });
        if constexpr (Smem::copies > 1) {
            __syncthreads();
            for (int b = tid; b < kSelBins; b += NT) {
                const uint4 c = *reinterpret_cast<const uint4 *>(&sm.copied[b * Smem::copies]);
                sm.hist[0][b] = (c.x + c.y) + (c.z + c.w);
            }
        }
    }
    uint32_t prefix = 0, rank = k;             // the rank'th largest among the matching keys
    uint32_t above_T = 0;                      // this thread's share of the CTA's keys above T
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *hist = sm.hist[pass];
        if (pass > 0) {
            // keys that match the digits found: those from `least` on, `width` of them
            const uint32_t least = prefix << (shift + bits), width = 1u << (shift + bits);
            batched(g0, g1, keys, [&](uint32_t g, const uint4 &q) {
                const uint32_t x[4] = {q.x - least, q.y - least, q.z - least, q.w - least};
                if (min(min(x[0], x[1]), min(x[2], x[3])) >= width)
                    return;
                const uint32_t v = valid(g);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (x[e] < width && (v >> e & 1u))
                        atomicAdd(&hist[x[e] >> shift], 1u);
            });
        }
        // Which bin holds the rank'th largest: first among the 32 sums of 64 bins,
        // then among that sum's 64 bins.  In a cluster thread t brings a peer's value
        // to shared memory; every warp then finds the same answer for itself.
        __syncthreads();
        uint2 own[kSelCoarse / (NT / 32)];              // bins 2 lane, + 1 of a warp's sums
#pragma unroll
        for (int j = 0; j < kSelCoarse / (NT / 32); ++j) {
            const int w = warp + j * (NT / 32);
            own[j] = *reinterpret_cast<const uint2 *>(hist + 64 * w + 2 * lane);
            const uint32_t part = __reduce_add_sync(0xffffffffu, own[j].x + own[j].y);
            if (lane == 0)
                sm.coarse[pass][w] = part;
        }
        const uint32_t *sums = sm.coarse[pass], *fine = hist;
        if (C > 1) {
            cluster.sync();
            if (tid < 32 * C)
                sm.peer[tid] = *cluster.map_shared_rank(&sm.coarse[pass][lane], warp);
            sums = sm.peer;
        }
        __syncthreads();
        uint32_t n = 0;
        for (int c = 0; c < C; ++c)
            n += sums[32 * c + 31 - lane];              // from the top
        uint32_t below = warp_inclusive(n, lane);
        const int at = __ffs(__ballot_sync(0xffffffffu, rank <= below)) - 1;
        rank -= __shfl_sync(0xffffffffu, below - n, at);
        const int base = 64 * (31 - at);
        fine += base;
        if (C > 1) {
            if (tid < 64 * C)
                sm.peer_bins[tid] = *cluster.map_shared_rank(hist + base + (tid & 63), tid >> 6);
            __syncthreads();
            fine = sm.peer_bins;
        }
        uint32_t n1 = 0, n0 = 0;                        // the lane's upper and lower bin
        for (int c = 0; c < C; ++c) {
            const uint2 v = *reinterpret_cast<const uint2 *>(fine + 64 * c + 62 - 2 * lane);
            n0 += v.x;
            n1 += v.y;
        }
        below = warp_inclusive(n0 + n1, lane);
        const int pair = __ffs(__ballot_sync(0xffffffffu, rank <= below)) - 1;
        rank -= __shfl_sync(0xffffffffu, below - n0 - n1, pair);
        n1 = __shfl_sync(0xffffffffu, n1, pair);
        uint32_t bin = (uint32_t)(base + 63 - 2 * pair);
        if (rank > n1) {
            rank -= n1;
            --bin;
        }
        prefix = (prefix << bits) | bin;
#pragma unroll
        for (int j = 0; j < kSelCoarse / (NT / 32); ++j) {
            const uint32_t b = 64u * (warp + j * (NT / 32)) + 2u * lane;
            above_T += (b + 1u > bin ? own[j].y : 0u) + (b > bin ? own[j].x : 0u);
        }
    }
    const uint32_t T = prefix;
    {
        uint32_t total;
        block_scan<NT>(above_T, sm.warp_sum[1], &total);
        if (tid == 0) {
            sm.counts[0] = total;
            sm.counts[1] = sm.hist[2][T & 1023u];
        }
    }
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();
    // keys above T all stay, and the first `rank` of those equal to T: all, some or
    // none of this CTA's.  Unless it is some, one comparison tells who stays.
    uint32_t gt_before = 0, eq_before = 0;
    for (int c = 0; c < me; ++c) {
        gt_before += *cluster.map_shared_rank(&sm.counts[0], c);
        eq_before += *cluster.map_shared_rank(&sm.counts[1], c);
    }
    const uint32_t eq_own = sm.counts[1];
    const bool some = rank > eq_before && rank < eq_before + eq_own;
    const uint32_t least = rank > eq_before ? T : T + 1;
    if (!some) {
        // output offset of the first to stay: those before it, above and equal
        gt_before += min(eq_before, rank);
        eq_before = 0;
    }
    for (uint32_t c0 = g0; c0 < g1; c0 += kSelChunk) {
        const uint32_t c1 = min(g1, c0 + kSelChunk), segs = (c1 - c0 + 31) / 32;
        // whole warps run, so that every segment's counts are summed by 32 lanes
        auto load = [&](uint32_t i) { return c0 + i < c1 ? keys(c0 + i) : make_uint4(0, 0, 0, 0); };
        batched(0, segs * 32, load, [&](uint32_t i, const uint4 &q) {
            uint32_t f = 0;
            if (c0 + i < c1) {
                if (!some)
                    f = (q.x >= least ? 1u : 0u) | (q.y >= least ? 2u : 0u) |
                        (q.z >= least ? 4u : 0u) | (q.w >= least ? 8u : 0u);
                else
                    f = (q.x > T ? 1u : 0u) | (q.y > T ? 2u : 0u) | (q.z > T ? 4u : 0u) |
                        (q.w > T ? 8u : 0u) | (q.x == T ? 16u : 0u) | (q.y == T ? 32u : 0u) |
                        (q.z == T ? 64u : 0u) | (q.w == T ? 128u : 0u);
                const uint32_t v = valid(c0 + i);
                f &= v | (v << 4);
            }
            sm.flags[i] = (unsigned char)f;
            const uint32_t n = __popc(f & 0xFu) | ((uint32_t)__popc(f >> 4) << 16);
            const uint32_t s = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0)
                sm.seg[i / 32] = s;
        });
        __syncthreads();
        uint32_t total;
        const uint32_t off =
            block_scan<NT>(tid < (int)segs ? sm.seg[tid] : 0u, sm.warp_sum[0], &total);
        if (tid < (int)segs)
            sm.seg[tid] = off;
        __syncthreads();
        for (uint32_t i = tid; i < segs * 32; i += NT) {
            const uint32_t f = sm.flags[i];
            const uint32_t n = __popc(f & 0xFu) | ((uint32_t)__popc(f >> 4) << 16);
            const uint32_t at = sm.seg[i / 32] + warp_inclusive(n, lane) - n;
            uint32_t gb = gt_before + (at & 0xFFFFu), eb = eq_before + (at >> 16);
            if (f == 0)
                continue;
            if (!some) {
                int32_t *to = kept + a.sink + gb;
                const int32_t t = (int32_t)(4 * (c0 + i) - skew);
                if (f & 1u) *to++ = t;
                if (f & 2u) *to++ = t + 1;
                if (f & 4u) *to++ = t + 2;
                if (f & 8u) *to++ = t + 3;
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool gt = (f >> e) & 1u, eq = (f >> (4 + e)) & 1u;
                if (gt || (eq && eb < rank))
                    kept[a.sink + gb + min(eb, rank)] = (int32_t)(4 * (c0 + i) + e - skew);
                gb += gt;
                eb += eq;
            }
        }
        gt_before += total & 0xFFFFu;
        eq_before += total >> 16;
        __syncthreads();
    }
    if (C > 1)
        cluster.sync();            // no CTA leaves while its counts may still be read
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------
//
// Kept row i of request r (token kept[r, i], read through the old page table) is
// copied to row i of the new one, for every layer, and its accumulated weight to
// mass_out[r, i].  Pure data movement: each row is read and written once.  A warp
// takes as many rows as make 288 16-byte vectors (4 rows of bf16 pages, 8 of E4M3
// pages): 9 vectors a lane, all in flight before the first store.

constexpr int kCompactThreads = 256;
constexpr int kCompactVecs = 9;

struct CompactArgs {
    void *slab[kCompactLayers];
    int64_t num_pages, page_bytes;
    const int32_t *table;
    int64_t table_ld;
    const int32_t *seq_lens;
    const int32_t *out_table;
    int64_t out_ld;
    const int32_t *kept;
    int64_t kept_ld;
    const int32_t *kept_lens;
    int keep;
    const float *mass;
    int64_t mass_ld, mass_cols;
    float *mass_out;
    int64_t mass_out_ld;
    int32_t *status;
};

template <bool F8>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactArgs a)
{
    constexpr int row_vecs = F8 ? 36 : 72;                       // 16-byte vectors per row
    constexpr int rows = 32 * kCompactVecs / row_vecs;           // rows per warp: 4 or 8
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y;
    const int i0 = (blockIdx.x * (kCompactThreads / 32) + (threadIdx.x >> 5)) * rows;
    const int n = min(a.keep, a.kept_lens[r]);
    if (i0 >= n)
        return;
    unsigned char *slab = static_cast<unsigned char *>(a.slab[blockIdx.z]);
    int64_t src = -1, dst = -1;                                  // lane i: row i0 + i
    if (lane < rows && i0 + lane < n) {
        const int i = i0 + lane;
        const int t = a.kept[(int64_t)r * a.kept_ld + i];
        int from = -1, to = -1;
        if (t >= 0 && t < a.seq_lens[r] && t / kPageTokens < a.table_ld &&
            i / kPageTokens < a.out_ld) {
            from = a.table[(int64_t)r * a.table_ld + t / kPageTokens];
            to = a.out_table[(int64_t)r * a.out_ld + i / kPageTokens];
        }
        if (from < 0 || to < 0 || (int64_t)from >= a.num_pages || (int64_t)to >= a.num_pages) {
            if (a.status != nullptr)
                atomicExch(a.status, kStatusAppendPage);
        } else {
            constexpr int row_bytes = F8 ? kRow : 2 * kRow;
            src = (int64_t)from * a.page_bytes + (int64_t)(t % kPageTokens) * row_bytes;
            dst = (int64_t)to * a.page_bytes + (int64_t)(i % kPageTokens) * row_bytes;
            if (a.mass != nullptr && blockIdx.z == 0 && t < a.mass_cols)
                a.mass_out[(int64_t)r * a.mass_out_ld + i] = a.mass[(int64_t)r * a.mass_ld + t];
        }
    }
    uint4 v[kCompactVecs];
#pragma unroll
    for (int j = 0; j < kCompactVecs; ++j) {
        const int u = lane + 32 * j, row = u / row_vecs;
        const int64_t s = __shfl_sync(0xffffffffu, src, row);
        if (s >= 0)
            v[j] = *reinterpret_cast<const uint4 *>(slab + s + 16 * (u % row_vecs));
    }
#pragma unroll
    for (int j = 0; j < kCompactVecs; ++j) {
        const int u = lane + 32 * j, row = u / row_vecs;
        const int64_t d = __shfl_sync(0xffffffffu, dst, row);
        if (d >= 0)
            *reinterpret_cast<uint4 *>(slab + d + 16 * (u % row_vecs)) = v[j];
    }
}

// Clusters of 2^log CTAs that the device holds at once (0: none, or it cannot say).
int select_max_clusters(int log)
{
    static int cached[64][5] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    if (cached[dev][log] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1u << log);
        cfg.blockDim = dim3(kSelThreads);
        cfg.dynamicSmemBytes = 4 * kSelCache;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << log;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, select_kernel<kSelThreads>, &cfg) != cudaSuccess) {
            cudaGetLastError();    // such clusters are not offered: take smaller ones
            n = 0;
        }
        cached[dev][log] = n + 1;
    }
    return cached[dev][log] - 1;
}

}  // namespace

cudaError_t launch_select(const float *mass, int64_t mass_ld, int64_t mass_cols,
                          const int32_t *seq_lens, int num_reqs, int keep, int sink, int recent,
                          int32_t *kept, int64_t kept_ld, int32_t *kept_lens,
                          cudaStream_t stream)
{
    // Rows of at most kSelSmall weights: one small CTA each.  Longer ones: the widest
    // cluster that leaves a CTA 4096 weights and has room for every request at once.
    const bool small = mass_cols <= kSelSmall;
    const void *kernel = small ? reinterpret_cast<const void *>(select_kernel<kSelSmallThreads>)
                               : reinterpret_cast<const void *>(select_kernel<kSelThreads>);
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)(4 * kSelCache));
    if (err == cudaSuccess && !small)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess)
        return err;
    // (More clusters than the device holds at once take turns: 16 histories of 100,000
    // tokens took 32 us in clusters of 8, against 20 us in clusters of 4.)
    int log = small ? 0 : 4;
    while (log > 0 && (mass_cols < ((int64_t)4096 << log) || num_reqs > select_max_clusters(log)))
        --log;
    const int cluster = 1 << log;
    // a slice of the longest history, up to kSelCache weights
    const int64_t groups = (mass_cols + 3) / 4 + 1, slice = (groups + cluster - 1) / cluster;
    const int cache_groups = (int)(slice < kSelCache / 4 ? slice : kSelCache / 4);
    SelectArgs a = {mass, mass_ld, mass_cols, seq_lens, keep, sink, recent, kept, kept_ld,
                    kept_lens, cache_groups};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_reqs * cluster));
    cfg.blockDim = dim3(small ? kSelSmallThreads : kSelThreads);
    cfg.dynamicSmemBytes = sizeof(uint4) * (size_t)cache_groups;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[1] = {&a};
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_compact(int num_layers, void *const *slabs, bool fp8, int64_t num_pages,
                           int64_t page_bytes, const int32_t *table, int64_t table_ld,
                           const int32_t *seq_lens, const int32_t *out_table, int64_t out_ld,
                           const int32_t *kept, int64_t kept_ld, const int32_t *kept_lens,
                           int num_reqs, int keep, const float *mass, int64_t mass_ld,
                           int64_t mass_cols, float *mass_out, int64_t mass_out_ld, int32_t *status,
                           cudaStream_t stream)
{
    const int per_block = kCompactThreads / 32 * (32 * kCompactVecs / (fp8 ? 36 : 72));
    for (int l0 = 0; l0 < num_layers; l0 += kCompactLayers) {
        const int n = num_layers - l0 < kCompactLayers ? num_layers - l0 : kCompactLayers;
        CompactArgs a = {};
        for (int l = 0; l < n; ++l)
            a.slab[l] = slabs[l0 + l];
        a.num_pages = num_pages;
        a.page_bytes = page_bytes;
        a.table = table;
        a.table_ld = table_ld;
        a.seq_lens = seq_lens;
        a.out_table = out_table;
        a.out_ld = out_ld;
        a.kept = kept;
        a.kept_ld = kept_ld;
        a.kept_lens = kept_lens;
        a.keep = keep;
        a.mass = l0 == 0 ? mass : nullptr;      // carried once
        a.mass_ld = mass_ld;
        a.mass_cols = mass_cols;
        a.mass_out = mass_out;
        a.mass_out_ld = mass_out_ld;
        a.status = status;
        const dim3 grid((unsigned)((keep + per_block - 1) / per_block), (unsigned)num_reqs,
                        (unsigned)n);
        if (fp8)
            compact_kernel<true><<<grid, kCompactThreads, 0, stream>>>(a);
        else
            compact_kernel<false><<<grid, kCompactThreads, 0, stream>>>(a);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace plmla
