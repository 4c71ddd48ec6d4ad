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
// output offset is the sum of the counts before it, so the indices come out in
// ascending order without a sort.  A slice that fits is kept in shared memory
// after its first read.

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelCache = 40960;              // keys of a slice kept in shared memory

struct SelectArgs {
    const float *mass;
    int64_t mass_ld, mass_cols;
    const int32_t *seq_lens;
    int keep, sink, recent;
    int32_t *kept;
    int64_t kept_ld;
    int32_t *kept_lens;
};

struct SelectSmem {
    uint32_t hist[kSelBins];       // this CTA's histogram, read by the whole cluster
    uint32_t sum[kSelBins];        // the cluster's
    uint32_t warp_sum[kSelWarps];
    uint32_t counts[2];            // this CTA's keys above T and equal to T, read by the cluster
    uint32_t bin, rank;            // the digit found, and the rank left within it
    uint32_t above[kSelWarps], equal[kSelWarps];
};

// Order-preserving key: larger weight, larger key; NaN 0, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u)
        return 0u;
    if (u == 0x80000000u)
        u = 0u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the block's threads (and the total).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sum, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();               // warp_sum may still be read from the last call
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int i = 0; i < kSelWarps; ++i) {
        const uint32_t s = warp_sum[i];
        before += i < warp ? s : 0u;
        all += s;
    }
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const SelectArgs a)
{
    extern __shared__ uint32_t cache[];
    __shared__ SelectSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int r = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t L64 = a.seq_lens[r];
    const int L = (int)(L64 < 0 ? 0 : (L64 > a.mass_cols ? a.mass_cols : L64));
    const float *mass = a.mass + (int64_t)r * a.mass_ld;
    int32_t *kept = a.kept + (int64_t)r * a.kept_ld;
    if (L <= a.keep) {             // everything stays
        for (int i = me * kSelThreads + tid; i < L; i += C * kSelThreads)
            kept[i] = i;
        if (me == 0 && tid == 0)
            a.kept_lens[r] = L;
        return;                    // the whole cluster takes this branch
    }
    const int lo = a.sink, hi = L - a.recent, n = hi - lo;
    const uint32_t k = (uint32_t)(a.keep - a.sink - a.recent);
    for (int i = me * kSelThreads + tid; i < a.sink + a.recent; i += C * kSelThreads) {
        if (i < a.sink)
            kept[i] = i;
        else
            kept[a.keep - a.recent + (i - a.sink)] = hi + (i - a.sink);
    }
    if (me == 0 && tid == 0)
        a.kept_lens[r] = a.keep;
    if (k == 0)
        return;

    // this CTA's slice of the candidates, a multiple of 32 long but for the last
    const int per = ((n + C - 1) / C + 31) / 32 * 32;
    const int s0 = min(n, me * per), s1 = min(n, s0 + per), len = s1 - s0;
    const float *mine = mass + lo + s0;
    const bool cached = per <= kSelCache;
    for (int i = tid; cached && i < len; i += kSelThreads)
        cache[i] = weight_key(mine[i]);
    auto key = [&](int i) -> uint32_t { return cached ? cache[i] : weight_key(mine[i]); };

    uint32_t prefix = 0, rank = k;             // the rank'th largest among the matching keys
    const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const uint32_t mask = (1u << bits[pass]) - 1u;
        for (int b = tid; b < kSelBins; b += kSelThreads)
            sm.hist[b] = 0;
        __syncthreads();
        for (int i = tid; i < len; i += kSelThreads) {
            const uint32_t u = key(i);
            if (pass == 0 || (u >> (shift[pass] + bits[pass])) == prefix)
                atomicAdd(&sm.hist[(u >> shift[pass]) & mask], 1u);
        }
        cluster.sync();
        for (int b = tid; b < kSelBins; b += kSelThreads) {
            uint32_t s = 0;
            for (int c = 0; c < C; ++c)
                s += *cluster.map_shared_rank(&sm.hist[b], c);
            sm.sum[b] = s;
        }
        __syncthreads();
        // thread t takes bins 2047 - 2t and 2046 - 2t: the scan runs from the top
        const int b1 = kSelBins - 1 - 2 * tid, b0 = b1 - 1;
        const uint32_t v1 = sm.sum[b1], v0 = sm.sum[b0];
        uint32_t total;
        const uint32_t above = block_scan(v1 + v0, sm.warp_sum, &total);
        if (above < rank && rank <= above + v1) {
            sm.bin = (uint32_t)b1;
            sm.rank = rank - above;
        } else if (above + v1 < rank && rank <= above + v1 + v0) {
            sm.bin = (uint32_t)b0;
            sm.rank = rank - above - v1;
        }
        cluster.sync();            // every CTA has read the histograms before they are reused
        prefix = (prefix << bits[pass]) | sm.bin;
        rank = sm.rank;
    }

    // keys above T all stay, and the first `rank` of those equal to T
    const uint32_t T = prefix;
    const int warp_len = ((len + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int w0 = min(len, warp * warp_len), w1 = min(len, w0 + warp_len);
    uint32_t gt = 0, eq = 0;
    for (int i = w0; i < w1; i += 32) {
        const uint32_t u = i + lane < w1 ? key(i + lane) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && u > T));
        eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && u == T));
    }
    if (lane == 0) {
        sm.above[warp] = gt;
        sm.equal[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            g += sm.above[i];
            e += sm.equal[i];
        }
        sm.counts[0] = g;
        sm.counts[1] = e;
    }
    cluster.sync();
    uint32_t gt_before = 0, eq_before = 0;
    for (int c = 0; c < me; ++c) {
        gt_before += *cluster.map_shared_rank(&sm.counts[0], c);
        eq_before += *cluster.map_shared_rank(&sm.counts[1], c);
    }
    for (int i = 0; i < warp; ++i) {
        gt_before += sm.above[i];
        eq_before += sm.equal[i];
    }
    for (int i = w0; i < w1; i += 32) {
        const uint32_t u = i + lane < w1 ? key(i + lane) : 0u;
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t g = __ballot_sync(0xffffffffu, i + lane < w1 && u > T);
        const uint32_t e = __ballot_sync(0xffffffffu, i + lane < w1 && u == T);
        const uint32_t gb = gt_before + __popc(g & below), eb = eq_before + __popc(e & below);
        const bool stay = ((g >> lane) & 1u) || (((e >> lane) & 1u) && eb < rank);
        if (stay)
            kept[a.sink + gb + min(eb, rank)] = lo + s0 + i + lane;
        gt_before += __popc(g);
        eq_before += __popc(e);
    }
    cluster.sync();                // no CTA leaves while its counts may still be read
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

}  // namespace

cudaError_t launch_select(const float *mass, int64_t mass_ld, int64_t mass_cols,
                          const int32_t *seq_lens, int num_reqs, int keep, int sink, int recent, int32_t *kept,
                          int64_t kept_ld, int32_t *kept_lens, int sms, cudaStream_t stream)
{
    const SelectArgs a = {mass, mass_ld, mass_cols, seq_lens, keep, sink, recent, kept, kept_ld, kept_lens};
    // the widest cluster (at most 8) that leaves a CTA 4096 weights and the SMs
    // enough room for every request at once
    int cluster = 8;
    while (cluster > 1 && (mass_cols < (int64_t)4096 * cluster || (int64_t)num_reqs * cluster > sms))
        cluster /= 2;
    const int64_t slice = (mass_cols + cluster - 1) / cluster + 31;
    const size_t smem = sizeof(uint32_t) * (size_t)(slice < kSelCache ? slice : kSelCache);
    cudaError_t err = cudaFuncSetAttribute(
        select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(4 * kSelCache));
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_reqs * cluster));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel, a);
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
