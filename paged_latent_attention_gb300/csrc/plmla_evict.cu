// plmla_evict.cu -- holding a cache to a budget: which tokens of each history
// stay (the heaviest by accumulated attention weight, after the scheme of Zhang
// et al., "H2O: Heavy-Hitter Oracle", 2023), and the copy of their rows into
// fresh pages.
#include <cooperative_groups.h>

#include <atomic>

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
// kSelCache weights of a slice stay in shared memory after their first read.
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
constexpr int kSelCache = 38912;              // weights of a slice kept in shared memory
constexpr int kSelChunk = 8192;               // groups of four written out at a time
constexpr int kSelMaxCluster = 16;
constexpr int kSelLong = 28672;               // weights of a slice from which parts pay,
constexpr int kSelPartThreads = 512;          // in CTAs of which two passes' fit an SM

struct SelectArgs {
    const float *mass;
    int64_t mass_ld, mass_cols;
    const int32_t *seq_lens;
    int keep, sink, recent;
    int32_t *kept;
    int64_t kept_ld;
    int32_t *kept_lens;
    int32_t *status;               // may be null
    int cache_groups;              // groups that the dynamic shared memory holds
};

template <int NT>
struct SelectSmem {
    static constexpr int copies = NT > kSelSmallThreads ? 4 : 1;   // of hist[0]
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

__device__ __forceinline__ uint4 weight_keys(const float4 &w)
{
    return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
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

// One request's candidates and the slice of them that part `me` of `parts` takes.
// Candidates [sink, hi) lie in groups of four aligned weights: group g holds tokens
// 4 g - skew .. 4 g - skew + 3.
struct Slice {
    const float *mass;
    uint32_t skew, first, last, first_bits, last_bits;
    uint32_t g0, g1;                   // this part's groups

    __device__ Slice(const float *row, int sink, int hi, uint32_t me, uint32_t parts) : mass(row)
    {
        skew = (uint32_t)(reinterpret_cast<uintptr_t>(mass) / 4) & 3u;
        const uint32_t v0 = (uint32_t)sink + skew, v1 = (uint32_t)hi + skew;
        first = v0 / 4;
        const uint32_t groups = (v1 + 3) / 4 - first, per = (groups + parts - 1) / parts;
        last = first + groups - 1;
        first_bits = 0xFu & (0xFu << (v0 - 4 * first));
        last_bits = 0xFu >> (4 * last + 4 - v1);
        g0 = first + min(groups, me * per);
        g1 = first + min(groups, (me + 1) * per);
    }
    // which of group g's elements are candidates: all but in the outermost groups
    __device__ uint32_t valid(uint32_t g) const
    {
        return (g == first ? first_bits : 0xFu) & (g == last ? last_bits : 0xFu);
    }
    // Group g's weights where all four are candidates, else zeros, which whoever uses
    // them replaces by edge(g): one predicated load, so that several go out together
    // (with both cases here each load waited for the one before).
    __device__ float4 fetch(uint32_t g) const
    {
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid(g) == 0xFu)
            w = *reinterpret_cast<const float4 *>(mass + ((int64_t)4 * g - skew));
        return w;
    }
    __device__ float4 edge(uint32_t g) const
    {
        const float *p = mass + ((int64_t)4 * g - skew);
        const uint32_t bits = valid(g);
        return make_float4(bits & 1u ? p[0] : 0.f, bits & 2u ? p[1] : 0.f, bits & 4u ? p[2] : 0.f,
                           bits & 8u ? p[3] : 0.f);
    }
    __device__ int32_t token(uint32_t g) const { return (int32_t)(4 * g - skew); }
};

// Where the keys of a slice are: groups before `split` in shared memory.
struct Source {
    const uint4 *cache;
    uint32_t split;
};

// The weights of groups at + i + j NT, i = this thread's first, for j < kSelBatch.
template <int NT>
__device__ __forceinline__ void load_batch(const Slice &s, uint32_t g, float4 (&w)[kSelBatch])
{
#pragma unroll
    for (int j = 0; j < kSelBatch; ++j)
        w[j] = s.fetch(min(g + j * NT, s.last));
}

// f(i, keys of group at + i) for this thread's i of [0, n).  The groups lie on one side
// of src.split.  Loads go out kSelBatch together; where the threads are few enough for
// the registers (kSelPartThreads) the next batch goes out before the last is used, and
// the first may have been loaded by the caller (`ready`).  WARPS: whole warps run, with
// other groups' keys for i >= n.
template <int NT, bool WARPS, typename F>
__device__ __forceinline__ void batched(const Slice &s, const Source &src, uint32_t at, uint32_t n,
                                        F f, const float4 (*ready)[kSelBatch] = nullptr)
{
    constexpr bool ahead = NT == kSelPartThreads;
    const uint32_t end = WARPS ? (n + 31) / 32 * 32 : n;
    if (at + n <= src.split) {
        const uint4 *p = src.cache + (at - s.g0);
#pragma unroll 2
        for (uint32_t i = threadIdx.x; i < end; i += NT)
            f(i, p[WARPS ? min(i, n - 1) : i]);
        return;
    }
    float4 w[kSelBatch];
    if (ready != nullptr) {
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j)
            w[j] = (*ready)[j];
    } else if (ahead) {
        load_batch<NT>(s, at + threadIdx.x, w);
    }
    for (uint32_t i = threadIdx.x; i < end; i += kSelBatch * NT) {
        float4 next[kSelBatch];
        if constexpr (ahead)
            load_batch<NT>(s, at + i + kSelBatch * NT, next);
        else
            load_batch<NT>(s, at + i, w);
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j)
            if (i + j * NT < end) {
                const uint32_t g = min(at + i + j * NT, s.last);
                if (s.valid(g) != 0xFu)
                    w[j] = s.edge(g);
                f(i + j * NT, weight_keys(w[j]));
            }
        if constexpr (ahead) {
#pragma unroll
            for (int j = 0; j < kSelBatch; ++j)
                w[j] = next[j];
        }
    }
}

// What a request keeps without a choice, written by its parts together: everything
// if it fits, else the first `sink` and the last `recent` tokens.  Whether there is
// a choice left to make, and among which tokens.
template <int NT>
__device__ __forceinline__ bool select_forced(const SelectArgs &a, int r, int me, int parts, int L,
                                              bool write)
{
    int32_t *kept = a.kept + (int64_t)r * a.kept_ld;
    const int tid = threadIdx.x;
    if (write && me == 0 && tid == 0) {
        a.kept_lens[r] = min(L, a.keep);
        if (a.seq_lens[r] > L && a.status != nullptr)
            atomicExch(a.status, kStatusMassLength);
    }
    if (L <= a.keep) {
        for (uint32_t i = me * NT + tid; i < (uint32_t)L && write; i += parts * NT)
            kept[i] = (int32_t)i;
        return false;
    }
    const uint32_t sink = a.sink, ends = sink + a.recent;
    for (uint32_t i = me * NT + tid; i < ends && write; i += parts * NT)
        kept[i < sink ? i : a.keep - ends + i] = (int32_t)(i < sink ? i : L - ends + i);
    return a.keep > a.sink + a.recent;
}

__device__ __forceinline__ int select_length(const SelectArgs &a, int r)
{
    const int64_t L = a.seq_lens[r];
    return (int)(L < 0 ? 0 : (L > a.mass_cols ? a.mass_cols : L));
}

// The first digit's histogram of a slice (zeroed before); keep(i, keys) sees each group.
template <int NT, typename Keep>
__device__ __forceinline__ void count_first(SelectSmem<NT> &sm, const Slice &s, Keep keep,
                                            const float4 (*ready)[kSelBatch] = nullptr)
{
    constexpr int copies = SelectSmem<NT>::copies;
    uint32_t *hist = copies > 1 ? sm.copied + threadIdx.x % copies : sm.hist[0];
    batched<NT, false>(s, Source{nullptr, s.g0}, s.g0, s.g1 - s.g0, [&](uint32_t i, const uint4 &q) {
        const uint32_t bits = s.valid(s.g0 + i);
        keep(i, q);
        if (bits & 1u) atomicAdd(&hist[(q.x >> 21) * copies], 1u);
        if (bits & 2u) atomicAdd(&hist[(q.y >> 21) * copies], 1u);
        if (bits & 4u) atomicAdd(&hist[(q.z >> 21) * copies], 1u);
        if (bits & 8u) atomicAdd(&hist[(q.w >> 21) * copies], 1u);
    }, ready);
    if constexpr (copies > 1) {
        __syncthreads();
        for (int b = threadIdx.x; b < kSelBins; b += NT) {
            const uint4 c = *reinterpret_cast<const uint4 *>(&sm.copied[b * copies]);
            sm.hist[0][b] = (c.x + c.y) + (c.z + c.w);
        }
    }
}

// Digit 1 or 2 (`pass`): its bits, and the histogram of the keys that match `prefix`,
// the digits found before: those from `least` on, `width` of them.
__device__ __forceinline__ int digit_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int pass) { return pass == 2 ? 10 : 11; }

template <int NT>
__device__ __forceinline__ void count_matching(uint32_t *hist, const Slice &s, const Source &src,
                                               int pass, uint32_t prefix,
                                               const float4 (*ready)[kSelBatch] = nullptr)
{
    const int shift = digit_shift(pass), top = shift + digit_bits(pass);
    const uint32_t least = prefix << top, width = 1u << top;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const uint32_t at = side == 0 ? s.g0 : src.split;
        const uint32_t n = (side == 0 ? src.split : s.g1) - at;
        batched<NT, false>(s, src, at, n, [&](uint32_t i, const uint4 &q) {
            const uint32_t x[4] = {q.x - least, q.y - least, q.z - least, q.w - least};
            if (min(min(x[0], x[1]), min(x[2], x[3])) >= width)
                return;
            const uint32_t v = s.valid(at + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x[e] < width && (v >> e & 1u))
                    atomicAdd(&hist[x[e] >> shift], 1u);
        }, ready);
    }
}

// A warp's search, from the top, for the lane in whose count n the rank'th falls;
// rank becomes the rank within it.
__device__ __forceinline__ int find_lane(uint32_t n, int lane, uint32_t *rank)
{
    const uint32_t upto = warp_inclusive(n, lane);
    const int at = __ffs(__ballot_sync(0xffffffffu, *rank <= upto)) - 1;
    *rank -= __shfl_sync(0xffffffffu, upto - n, at);
    return at;
}

// Writes the slice's tokens that stay, in order: keys above T, and those equal to it
// from the eq_before'th on until `rank` of them have been taken.  gt_before: keys
// above T before the slice; eq_own: the slice's keys equal to T.
template <int NT>
__device__ __forceinline__ void write_kept(SelectSmem<NT> &sm, const Slice &s, const Source &src,
                                           int32_t *kept, uint32_t T, uint32_t rank,
                                           uint32_t gt_before, uint32_t eq_before, uint32_t eq_own,
                                           const float4 (*ready)[kSelBatch] = nullptr)
{
    const int tid = threadIdx.x, lane = tid & 31;
    // All, some or none of the slice's equal keys stay.  Unless it is some, one
    // comparison tells who stays.
    const bool some = rank > eq_before && rank < eq_before + eq_own;
    const uint32_t least = rank > eq_before ? T : T + 1;
    if (!some) {
        // output offset of the first to stay: those before it, above and equal
        gt_before += min(eq_before, rank);
        eq_before = 0;
    }
    for (uint32_t c0 = s.g0, c1; c0 < s.g1; c0 = c1) {
        c1 = min(s.g1, c0 + kSelChunk);
        if (c0 < src.split)
            c1 = min(c1, src.split);               // on one side of it
        const uint32_t segs = (c1 - c0 + 31) / 32;
        batched<NT, true>(s, src, c0, c1 - c0, [&](uint32_t i, const uint4 &q) {
            uint32_t f;
            if (!some)
                f = (q.x >= least ? 1u : 0u) | (q.y >= least ? 2u : 0u) |
                    (q.z >= least ? 4u : 0u) | (q.w >= least ? 8u : 0u);
            else
                f = (q.x > T ? 1u : 0u) | (q.y > T ? 2u : 0u) | (q.z > T ? 4u : 0u) |
                    (q.w > T ? 8u : 0u) | (q.x == T ? 16u : 0u) | (q.y == T ? 32u : 0u) |
                    (q.z == T ? 64u : 0u) | (q.w == T ? 128u : 0u);
            const uint32_t v = i < c1 - c0 ? s.valid(c0 + i) : 0u;
            f &= v | (v << 4);
            sm.flags[i] = (unsigned char)f;
            // a warp's lanes hold the groups of one segment
            const uint32_t n = __popc(f & 0xFu) | ((uint32_t)__popc(f >> 4) << 16);
            const uint32_t sum = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0)
                sm.seg[i / 32] = sum;
        }, c0 == s.g0 ? ready : nullptr);
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
            const int32_t t = s.token(c0 + i);
            if (!some) {
                int32_t *to = kept + gb;
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
                    kept[gb + min(eb, rank)] = t + e;
                gb += gt;
                eb += eq;
            }
        }
        gt_before += total & 0xFFFFu;
        eq_before += total >> 16;
        __syncthreads();
    }
}

template <int NT>
__global__ void __launch_bounds__(NT) select_kernel(const SelectArgs a)
{
    extern __shared__ uint4 cache[];
    __shared__ SelectSmem<NT> sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int r = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = select_length(a, r);
    {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int b = tid; b < 3 * kSelBins / 4; b += NT)
            reinterpret_cast<uint4 *>(sm.hist)[b] = zero;
        for (int b = tid; b < (int)(sizeof(sm.copied) / 16); b += NT)
            reinterpret_cast<uint4 *>(sm.copied)[b] = zero;
    }
    if (!select_forced<NT>(a, r, me, C, L, true))
        return;                    // the whole cluster takes this branch
    const Slice s(a.mass + (int64_t)r * a.mass_ld, a.sink, L - a.recent, me, C);
    const uint32_t cached = (uint32_t)a.cache_groups;
    const Source src = {cache, min(s.g1, s.g0 + cached)};
    __syncthreads();
    count_first<NT>(sm, s, [&](uint32_t i, const uint4 &q) {
        if (i < cached)
            cache[i] = q;
    });
    // the rank'th largest among the keys that match `prefix`
    uint32_t prefix = 0, rank = (uint32_t)(a.keep - a.sink - a.recent);
    uint32_t above_T = 0;                      // this thread's share of the CTA's keys above T
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        uint32_t *hist = sm.hist[pass];
        if (pass > 0)
            count_matching<NT>(hist, s, src, pass, prefix);
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
        const int base = 64 * (31 - find_lane(n, lane, &rank));
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
        const int pair = find_lane(n0 + n1, lane, &rank);
        n1 = __shfl_sync(0xffffffffu, n1, pair);
        uint32_t bin = (uint32_t)(base + 63 - 2 * pair);
        if (rank > n1) {
            rank -= n1;
            --bin;
        }
        prefix = (prefix << digit_bits(pass)) | bin;
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
    uint32_t gt_before = 0, eq_before = 0;
    for (int c = 0; c < me; ++c) {
        gt_before += *cluster.map_shared_rank(&sm.counts[0], c);
        eq_before += *cluster.map_shared_rank(&sm.counts[1], c);
    }
    write_kept<NT>(sm, s, src, a.kept + (int64_t)r * a.kept_ld + a.sink, T, rank, gt_before,
                   eq_before, sm.counts[1]);
    if (C > 1)
        cluster.sync();            // no CTA leaves while its counts may still be read
}

// Long rows, few of them: a cluster has 16 SMs at most, so the same search runs as
// four kernels in which every request has `parts` CTAs (one per SM together), whose
// histograms meet in a workspace.  Pass p finds digit p - 1 among the parts'
// histograms (each CTA for itself: 32 sums and 64 bins per part, a few KB from L2),
// counts digit p of its slice, and notes how many keys above the final threshold the
// parts before it have shown so far; the last pass writes.  Each pass reads the slice
// again, from L2, its first loads before the pass ahead of it has finished.
// Measured against the cluster form: one row of a million weights 26 us (45), of four
// millions 41 us (141), four rows of a million 39 us (44), two of 500,000 23 us (26);
// below kSelLong weights a slice the cluster wins (one row of 300,000 22 us, 23 in
// parts).
struct SelectParts {
    int parts;
    uint32_t *hist;                // [request][3][part][kSelBins]
    uint32_t *coarse;              // [request][3][part][kSelCoarse]
    uint32_t *before;              // [request][part] keys above T in the parts before
    uint2 *state;                  // [request][3] prefix and rank once digit p is found
};

template <int PASS>
__global__ void __launch_bounds__(kSelPartThreads, 2) select_part_kernel(const SelectArgs a,
                                                                         const SelectParts p)
{
    constexpr int NT = kSelPartThreads, kWarps = NT / 32;
    __shared__ SelectSmem<NT> sm;
    __shared__ uint4 red[kWarps][32];
    const int r = blockIdx.x / p.parts, me = blockIdx.x % p.parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // The next pass's CTAs take their places beside these and wait for this grid to
    // finish; until then they read only what was there before the first pass.
    if constexpr (PASS < 3)
        asm volatile("griddepcontrol.launch_dependents;");
    const int L = select_length(a, r);
    if (!select_forced<NT>(a, r, me, p.parts, L, PASS == 0)) {
        // (no grid ends before the one ahead of it)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const Slice s(a.mass + (int64_t)r * a.mass_ld, a.sink, L - a.recent, me, p.parts);
    float4 ready[kSelBatch];
    load_batch<NT>(s, s.g0 + tid, ready);
    if constexpr (PASS == 0) {
        for (int b = tid; b < (int)(sizeof(sm.copied) / 16); b += NT)
            reinterpret_cast<uint4 *>(sm.copied)[b] = zero;
    } else if constexpr (PASS < 3) {
        for (int b = tid; b < kSelBins / 4; b += NT)
            reinterpret_cast<uint4 *>(sm.hist[PASS])[b] = zero;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Source src = {nullptr, s.g0};
    uint32_t prefix = 0, rank = (uint32_t)(a.keep - a.sink - a.recent);
    uint32_t gt_before = 0, eq_before = 0, eq_own = 0;
    if constexpr (PASS > 0) {
        constexpr int found = PASS - 1;        // the digit to find
        if constexpr (PASS > 1) {
            const uint2 st = p.state[3 * r + found - 1];
            prefix = st.x;
            rank = st.y;
            gt_before = p.before[(int64_t)r * p.parts + me];
        }
        const uint32_t *coarse = p.coarse + ((int64_t)3 * r + found) * p.parts * kSelCoarse;
        const uint32_t *hist = p.hist + ((int64_t)3 * r + found) * p.parts * kSelBins;
        // warp w sums parts w, w + kWarps, ...: of all parts, and of those before this one
        uint32_t n = 0, b = 0;
        for (int c = warp; c < p.parts; c += kWarps) {
            const uint32_t v = coarse[c * kSelCoarse + lane];
            n += v;
            b += c < me ? v : 0u;
        }
        red[warp][31 - lane] = make_uint4(n, b, 0u, 0u);       // from the top
        __syncthreads();
        n = b = 0;
        for (int w = 0; w < kWarps; ++w) {
            const uint4 v = red[w][lane];
            n += v.x;
            b += v.y;
        }
        const int at = find_lane(n, lane, &rank);
        gt_before += __reduce_add_sync(0xffffffffu, lane < at ? b : 0u);
        const int base = 64 * (31 - at);
        __syncthreads();
        uint4 v = zero;                        // lower and upper bin of all parts; of those before
        for (int c = warp; c < p.parts; c += kWarps) {
            const uint2 x =
                *reinterpret_cast<const uint2 *>(hist + c * kSelBins + base + 62 - 2 * lane);
            v.x += x.x;
            v.y += x.y;
            v.z += c < me ? x.x : 0u;
            v.w += c < me ? x.y : 0u;
        }
        red[warp][lane] = v;
        __syncthreads();
        v = zero;
        for (int w = 0; w < kWarps; ++w) {
            const uint4 x = red[w][lane];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        const int pair = find_lane(v.x + v.y, lane, &rank);
        const uint32_t n1 = __shfl_sync(0xffffffffu, v.y, pair);
        const bool lower = rank > n1;
        gt_before += __reduce_add_sync(0xffffffffu, lane < pair ? v.z + v.w
                                                    : lane == pair && lower ? v.w : 0u);
        eq_before = __shfl_sync(0xffffffffu, lower ? v.z : v.w, pair);
        if (lower)
            rank -= n1;
        const uint32_t bin = (uint32_t)(base + 63 - 2 * pair) - (lower ? 1u : 0u);
        prefix = (prefix << digit_bits(found)) | bin;
        eq_own = hist[me * kSelBins + bin];
        if (PASS < 3 && tid == 0) {
            p.before[(int64_t)r * p.parts + me] = gt_before;
            if (me == 0)
                p.state[3 * r + found] = make_uint2(prefix, rank);
        }
    }
    if constexpr (PASS == 3) {
        write_kept<NT>(sm, s, src, a.kept + (int64_t)r * a.kept_ld + a.sink, prefix, rank,
                       gt_before, eq_before, eq_own, &ready);
    } else {
        __syncthreads();
        if constexpr (PASS == 0)
            count_first<NT>(sm, s, [](uint32_t, const uint4 &) {}, &ready);
        else
            count_matching<NT>(sm.hist[PASS], s, src, PASS, prefix, &ready);
        __syncthreads();
        const int64_t at = ((int64_t)3 * r + PASS) * p.parts + me;
        for (int w = warp; w < kSelCoarse; w += kWarps) {
            const uint2 own = *reinterpret_cast<const uint2 *>(sm.hist[PASS] + 64 * w + 2 * lane);
            reinterpret_cast<uint2 *>(p.hist + at * kSelBins + 64 * w)[lane] = own;
            const uint32_t part = __reduce_add_sync(0xffffffffu, own.x + own.y);
            if (lane == 0)
                p.coarse[at * kSelCoarse + w] = part;
        }
    }
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
    int64_t table_ld, table_cols;
    const int32_t *seq_lens;
    const int32_t *out_table;
    int64_t out_ld, out_cols;
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
    const int64_t start = ((int64_t)blockIdx.x * (kCompactThreads / 32) + (threadIdx.x >> 5)) * rows;
    const int n = min(a.keep, a.kept_lens[r]);
    if (start >= n)
        return;
    const int i0 = (int)start;
    unsigned char *slab = static_cast<unsigned char *>(a.slab[blockIdx.z]);
    int64_t src = -1, dst = -1;                                  // lane i: row i0 + i
    if (lane < rows && i0 + lane < n) {
        const int i = i0 + lane;
        const int t = a.kept[(int64_t)r * a.kept_ld + i];
        int from = -1, to = -1;
        if (t >= 0 && t < a.seq_lens[r] && t / kPageTokens < a.table_cols &&
            i / kPageTokens < a.out_cols) {
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
            if (a.mass != nullptr && blockIdx.z == 0) {
                if (t < a.mass_cols)
                    a.mass_out[(int64_t)r * a.mass_out_ld + i] = a.mass[(int64_t)r * a.mass_ld + t];
                else if (a.status != nullptr)
                    atomicExch(a.status, kStatusMassLength);
            }
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

cudaError_t select_attributes(const void *kernel)
{
    const cudaError_t err = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(4 * kSelCache));
    return err != cudaSuccess
               ? err
               : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// Clusters of 2^log CTAs that the device holds at once (0: none, or it cannot say).
// An answer is kept; a query that failed is made again by the next call.
int select_max_clusters(int log)
{
    static std::atomic<int> cached[64][5];         // the answer + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cached[dev][log].load(std::memory_order_relaxed) - 1;
    if (n < 0) {
        if (select_attributes(reinterpret_cast<const void *>(select_kernel<kSelThreads>)) !=
            cudaSuccess)
            return 0;
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
        if (cudaOccupancyMaxActiveClusters(&n, select_kernel<kSelThreads>, &cfg) != cudaSuccess) {
            cudaGetLastError();    // such clusters are not offered: take smaller ones
            return 0;
        }
        cached[dev][log].store(n + 1, std::memory_order_relaxed);
    }
    return n;
}

// log2 of the CTAs per request.  Rows of at most kSelSmall weights: one small CTA
// each.  Longer ones: the widest cluster that leaves a CTA 4096 weights and has room
// for every request at once.  (More clusters than the device holds take turns: 16
// histories of 100,000 tokens took 32 us in clusters of 8, 21 us in clusters of 4.)
int select_cluster_log(int num_reqs, int64_t mass_cols)
{
    int log = mass_cols <= kSelSmall ? 0 : 4;
    while (log > 0 && (mass_cols < ((int64_t)4096 << log) || num_reqs > select_max_clusters(log)))
        --log;
    return log;
}

}  // namespace

// Parts per request of the form for long rows (0: the cluster form serves as well):
// where a cluster's slices pass kSelLong weights and every request can have at least
// twice the cluster's SMs.
int select_parts(int num_reqs, int64_t mass_cols, int sms)
{
    const int log = select_cluster_log(num_reqs, mass_cols);
    const int parts = sms / num_reqs;
    return mass_cols >> log > kSelLong && parts >= 2 << log ? parts : 0;
}

size_t select_workspace(int num_reqs, int parts)
{
    // per request: state, and per part three histograms, their sums and a count
    return (size_t)num_reqs *
           (3 * sizeof(uint2) + (size_t)parts * sizeof(uint32_t) * (3 * (kSelBins + kSelCoarse) + 1));
}

cudaError_t launch_select(const float *mass, int64_t mass_ld, int64_t mass_cols,
                          const int32_t *seq_lens, int num_reqs, int keep, int sink, int recent,
                          int32_t *kept, int64_t kept_ld, int32_t *kept_lens, int parts,
                          void *workspace, int32_t *status, cudaStream_t stream)
{
    SelectArgs a = {mass, mass_ld, mass_cols, seq_lens, keep, sink, recent, kept, kept_ld,
                    kept_lens, status, 0};
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    if (parts > 0) {
        SelectParts p = {parts};
        p.state = static_cast<uint2 *>(workspace);
        p.hist = reinterpret_cast<uint32_t *>(p.state + 3 * num_reqs);
        p.coarse = p.hist + (size_t)num_reqs * 3 * parts * kSelBins;
        p.before = p.coarse + (size_t)num_reqs * 3 * parts * kSelCoarse;
        // later passes are launched ahead of the end of the one before
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)(num_reqs * parts));
        cfg.blockDim = dim3(kSelPartThreads);
        cudaError_t err = cudaLaunchKernelEx(&cfg, select_part_kernel<0>, a, p);
        cfg.numAttrs = 1;
        if (err == cudaSuccess)
            err = cudaLaunchKernelEx(&cfg, select_part_kernel<1>, a, p);
        if (err == cudaSuccess)
            err = cudaLaunchKernelEx(&cfg, select_part_kernel<2>, a, p);
        return err == cudaSuccess ? cudaLaunchKernelEx(&cfg, select_part_kernel<3>, a, p) : err;
    }
    const bool small = mass_cols <= kSelSmall;
    const void *kernel = small ? reinterpret_cast<const void *>(select_kernel<kSelSmallThreads>)
                               : reinterpret_cast<const void *>(select_kernel<kSelThreads>);
    const cudaError_t err = select_attributes(kernel);
    if (err != cudaSuccess)
        return err;
    const int cluster = 1 << select_cluster_log(num_reqs, mass_cols);
    // a slice of the longest history, up to kSelCache weights
    const int64_t groups = (mass_cols + 3) / 4 + 1, slice = (groups + cluster - 1) / cluster;
    a.cache_groups = (int)(slice < kSelCache / 4 ? slice : kSelCache / 4);
    cfg.gridDim = dim3((unsigned)(num_reqs * cluster));
    cfg.blockDim = dim3(small ? kSelSmallThreads : kSelThreads);
    cfg.dynamicSmemBytes = sizeof(uint4) * (size_t)a.cache_groups;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    void *args[1] = {&a};
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_compact(int num_layers, void *const *slabs, bool fp8, int64_t num_pages,
                           int64_t page_bytes, const int32_t *table, int64_t table_ld,
                           int64_t table_cols, const int32_t *seq_lens, const int32_t *out_table,
                           int64_t out_ld, int64_t out_cols, const int32_t *kept, int64_t kept_ld,
                           const int32_t *kept_lens, int num_reqs, int keep, const float *mass,
                           int64_t mass_ld, int64_t mass_cols, float *mass_out,
                           int64_t mass_out_ld, int32_t *status, cudaStream_t stream)
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
        a.table_cols = table_cols;
        a.seq_lens = seq_lens;
        a.out_table = out_table;
        a.out_ld = out_ld;
        a.out_cols = out_cols;
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
        const dim3 grid((unsigned)(((int64_t)keep + per_block - 1) / per_block), (unsigned)num_reqs,
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
