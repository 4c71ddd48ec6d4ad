// plmla_pages.cu -- ownership of cache pages by counts: histories that share pages are
// forked, released, and given room to grow, on the device.
//
//   counts[p] = the table rows (and other holders) that hold page p; 0 = free
//   fork      out[i] <- table[parents[i]]: counts follow, no row of the cache moves
//   free      counts[p] -= 1 for every page of a row; its history becomes empty
//   reserve   room for n new tokens behind every history: free pages in ascending order,
//             and a partly filled last page that others hold too is copied first
//             (in row order; the last of its holders keeps it)
//
// A pool has no other state than its counts: the free pages are found by a scan, which for
// the pools that fit a GPU (160,000 pages of 1.77 MB at most) costs microseconds and keeps
// the result a function of the arguments, whatever was freed in which order.
//
// Fork and free: one block per row, a page per thread; atomics on counts add up to the
// same whole numbers in any order.  A page that an out row already holds in the same place
// stays without touching its count.  Both are latency-bound: three dependent loads and an
// atomic.  A fork into the emptied double of a table and the release of the old rows, so every
// page's count goes up and down: 1,024 rows with 196,306 pages 9.5 us, four rows 4.4; a fork of rows
// that are there already 4.0 and 1.9.
//
// Reserve: one block plans (rows in threads, prefix sums, 16,384 counts a sweep), then a grid
// of blocks copies the planned pages, one contiguous piece per (row, layer), at the copy
// rate of HBM.  The copy is launched programmatically behind the plan.  Eight E4M3 prompts' 64
// continuations in four layers: 35.5-37 us with the fork before it, of which the bytes take 31; two
// rows and one page 9-10 us, latency.
#include "plmla_internal.cuh"

namespace plmla {
namespace {

constexpr int kForkThreads = 128;               // of a row
constexpr int kForkBlock = 1024, kForkCluster = 8;
constexpr int kReserveThreads = 1024;
constexpr int kSweep = 16 * kReserveThreads;    // counts that the block looks at together
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                    // 16-byte vectors of a thread in flight
constexpr int kCopyPiece = kCopyThreads * kCopyVecs;

// (of several codes the largest stays, whichever row comes first)
__device__ __forceinline__ void report(int32_t *status, int32_t code)
{
    if (status != nullptr)
        atomicMax(status, code);
}

__device__ __forceinline__ void hold(int32_t *counts, int64_t num_pages, int page, int32_t *status)
{
    if (page < 0 || page >= num_pages)
        report(status, kStatusAppendPage);
    else
        atomicAdd(counts + page, 1);
}

// A holder of the page finds it counted: what other rows of this launch give up never takes
// the count below the holders that remain.
__device__ __forceinline__ void give_up(int32_t *counts, int64_t num_pages, int page,
                                        int32_t *status)
{
    if (page < 0 || page >= num_pages) {
        report(status, kStatusAppendPage);
    } else if (atomicSub(counts + page, 1) <= 0) {
        atomicAdd(counts + page, 1);
        report(status, kStatusPageCount);
    }
}

__device__ __forceinline__ int pages_of(int len) { return len <= 0 ? 0 : (len - 1) / kPageTokens + 1; }

// All holders are added before any is taken off: otherwise a page that is held without being
// counted would end with a count that depends on which row comes first.  Up to 64 rows
// are a cluster with a barrier between (BOTH), more are two launches, the second of which has
// read its rows when the first ends (4 rows 2.4 us and a launch more for the host, not 1.9;
// in one launch without an order 4 rows took 1.5 us, 1,024 rows 2.4, not 4.0).  A row is the work of 128
// threads; threads without a row or with one that is left as it is go through the barriers.
enum ForkStep { BOTH, HOLD, GIVE };
template <int STEP>
__global__ void __launch_bounds__(kForkBlock) fork_kernel(const ForkArgs a)
{
    if (STEP == HOLD)
        asm volatile("griddepcontrol.launch_dependents;");
    const int t = threadIdx.x % kForkThreads;
    const int i = (int)blockIdx.x * (int)(blockDim.x / kForkThreads) + (int)threadIdx.x / kForkThreads;
    const bool speaks = STEP != GIVE && t == 0;
    bool mine = i < a.out_rows;
    const int parent = mine ? a.parents[i] : -1, held = mine ? a.out_lens[i] : 0;
    int old = pages_of(held), len = 0;
    if (parent >= 0 && parent < a.rows)
        len = a.lens[parent];
    if (held < 0 || len < 0) {
        if (speaks)
            report(a.status, kStatusAppendPosition);
        mine = false;
        old = len = 0;
    }
    if (old > a.out_cols) {
        old = (int)a.out_cols;
        if (speaks)
            report(a.status, kStatusAppendPage);
    }
    if (parent >= a.rows && speaks)
        report(a.status, kStatusParent);
    int pages = pages_of(len);
    if (pages > a.cols || pages > a.out_cols) {
        pages = len = 0;
        if (speaks)
            report(a.status, kStatusAppendPage);
    }
    int32_t *out = a.out_table + (int64_t)i * a.out_ld;
    const int32_t *from = a.table + (int64_t)parent * a.ld;
    const int end = max(old, pages);
    // the first column of a thread, for both steps (most rows have no other)
    int was = t < old ? out[t] : 0, now = t < pages ? from[t] : 0;
    if (STEP != GIVE)
        for (int c = t; c < end; c += kForkThreads) {
            const int w = c == t ? was : c < old ? out[c] : 0;
            const int n = c == t ? now : c < pages ? from[c] : 0;
            if (c < pages && !(c < old && w == n))
                hold(a.counts, a.num_pages, n, a.status);
        }
    if (STEP == HOLD)
        return;
    if (STEP == BOTH)
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    else
        asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int c = t; c < end; c += kForkThreads) {
        if (c > t) {
            was = c < old ? out[c] : 0;
            now = c < pages ? from[c] : 0;
        }
        if (c < old && c < pages && was == now)
            continue;
        if (c < old)
            give_up(a.counts, a.num_pages, was, a.status);
        if (c < pages)
            out[c] = now;
    }
    __syncthreads();                            // every thread has read out_lens
    if (mine && t == 0)
        a.out_lens[i] = len;
}

__global__ void __launch_bounds__(kForkThreads)
free_kernel(const int32_t *table, int64_t ld, int64_t cols, int32_t *lens, int32_t *counts,
            int64_t num_pages, int32_t *status)
{
    const int r = blockIdx.x;
    const int len = lens[r];
    int pages = pages_of(len);
    if (len < 0) {
        if (threadIdx.x == 0)
            report(status, kStatusAppendPosition);
        return;
    }
    if (pages > cols) {
        pages = (int)cols;
        if (threadIdx.x == 0)
            report(status, kStatusAppendPage);
    }
    for (int c = threadIdx.x; c < pages; c += kForkThreads)
        give_up(counts, num_pages, table[(int64_t)r * ld + c], status);
    __syncthreads();
    if (threadIdx.x == 0)
        lens[r] = 0;
}

// Exclusive prefix sum over the block's threads, and the total.
__device__ __forceinline__ int block_scan(int v, int *warp_sum, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();                            // warp_sum of an earlier scan has been read
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    *total = warp_sum[31];
    return x - v + (warp == 0 ? 0 : warp_sum[warp - 1]);
}

// Which of the 16 pages from `first` on are free, a bit each.
__device__ __forceinline__ uint32_t free_bits(const int32_t *counts, int64_t first, int64_t num_pages)
{
    uint32_t bits = 0;
    if (first + 16 <= num_pages && (reinterpret_cast<uintptr_t>(counts) & 15u) == 0) {
        const int4 *p = reinterpret_cast<const int4 *>(counts + first);
        int4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = p[j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bits |= ((v[j].x == 0) | (v[j].y == 0) << 1 | (v[j].z == 0) << 2 | (v[j].w == 0) << 3)
                    << (4 * j);
    } else {
        for (int j = 0; j < 16; ++j)
            if (first + j < num_pages && counts[first + j] == 0)
                bits |= 1u << j;
    }
    return bits;
}

__global__ void __launch_bounds__(kReserveThreads) reserve_kernel(const ReserveArgs a)
{
    __shared__ int warp_sum[32];
    __shared__ alignas(16) int last_sm[kMaxReqs];             // shared last page of a row, or -1
    __shared__ int end_sm[kMaxReqs];            // pages that rows 0 .. r need together
    __shared__ int col_sm[kMaxReqs];            // column of the row's first page needed
    __shared__ int job_sm[kMaxReqs];            // the row's copy, or -1
    __shared__ int window[kReserveThreads];
    __shared__ int placed, refused;             // pages given out; the first row without its pages
    asm volatile("griddepcontrol.launch_dependents;");
    const int r = threadIdx.x;
    // the first sweep's counts are on their way while the rows' needs are worked out
    uint32_t bits = free_bits(a.counts, 16 * r, a.num_pages);
    int need = 0, part = 0, last = -1, holders = 0, col = 0, add = 0;
    bool valid = false, parts = false;          // the last page has other holders
    if (r < a.num_reqs) {
        const int len = a.lens[r];
        add = a.n_new_of != nullptr ? a.n_new_of[r] : a.n_new;
        const int64_t want = ((int64_t)len + add + kPageTokens - 1) / kPageTokens;
        if (len < 0 || add < 0) {
            report(a.status, kStatusAppendPosition);
        } else if (want > a.cols) {
            report(a.status, kStatusAppendPage);
        } else if (add > 0) {
            valid = true;
            part = len % kPageTokens;
            col = pages_of(len);
            need = (int)want - col;
            if (part != 0) {
                last = a.table[(int64_t)r * a.ld + col - 1];
                if (last < 0 || last >= a.num_pages) {
                    report(a.status, kStatusAppendPage);
                    need = 0;
                    valid = false;
                } else {
                    holders = a.counts[last];
                    parts = holders > 1;
                    if (holders < 1) {          // it may go to another row
                        report(a.status, kStatusPageCount);
                        need = 0;
                        valid = false;
                    }
                }
            }
        }
    }
    last_sm[r] = parts ? last : -1;
    const bool shares = parts;
    if (__syncthreads_or(parts) && parts) {
        int earlier = 0;
        const int4 *rows = reinterpret_cast<const int4 *>(last_sm);
#pragma unroll 4
        for (int j = 0; j < (r + 3) / 4; ++j) {
            const int4 v = rows[j];
            earlier += (v.x == last && 4 * j < r) + (v.y == last && 4 * j + 1 < r) +
                       (v.z == last && 4 * j + 2 < r) + (v.w == last && 4 * j + 3 < r);
        }
        parts = holders - earlier > 1;          // the last holder keeps the page
    }
    need += parts ? 1 : 0;
    int total, jobs;
    const int first = block_scan(need, warp_sum, &total);
    int job = block_scan(parts ? 1 : 0, warp_sum, &jobs);
    end_sm[r] = first + need;
    col_sm[r] = col - (parts ? 1 : 0);
    job_sm[r] = parts ? job : -1;
    if (r == 0) {
        placed = 0;
        refused = kReserveThreads;
    }
    __syncthreads();

    // the free pages that there are, as far as they are needed
    int found = 0, rank = 0;
    int64_t base = 0;
    for (; base < a.num_pages && found < total; base += kSweep) {
        if (base > 0)
            bits = free_bits(a.counts, base + 16 * r, a.num_pages);
        int here;
        rank = found + block_scan(__popc(bits), warp_sum, &here);
        found += here;
    }
    const bool served = need > 0 && first + need <= found;
    if (need > 0 && !served)
        atomicMin(&refused, r);
    if (served)
        atomicMax(&placed, first + need);
    if (parts && served) {
        a.jobs[job].x = last;
        a.jobs[job].z = part;
        atomicSub(a.counts + last, 1);
    }
    const int copies = __syncthreads_count(parts && served);
    if (r == 0)
        *a.num_jobs = copies;                   // served rows come first
    const int most = placed;

    // Page number q of them belongs to the row whose pages end past q.  The sweep's free pages
    // are listed a window at a time, and a thread places one: pages in a row often lie in few
    // threads' 16, which one by one took 5 us for 64 rows.
    const bool once = base <= kSweep;           // one sweep: its bits are at hand
    int before = 0;
    for (int64_t at = 0; at < base && before < most; at += kSweep) {
        int here = found;
        if (!once) {
            bits = free_bits(a.counts, at + 16 * r, a.num_pages);
            rank = before + block_scan(__popc(bits), warp_sum, &here);
        }
        const int upto = min(before + here, most);
        for (int q0 = before; q0 < upto; q0 += kReserveThreads) {
            __syncthreads();                    // the last window has been placed
            int q = rank;
            for (uint32_t left = bits; left != 0; left &= left - 1, ++q)
                if (q >= q0 && q < q0 + kReserveThreads)
                    window[q - q0] = (int)(at + 16 * r) + __ffs(left) - 1;
            __syncthreads();
            q = q0 + r;
            if (q < upto) {
                const int page = window[r];
                int lo = 0, hi = a.num_reqs - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (end_sm[mid] > q)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                const int nth = q - (lo == 0 ? 0 : end_sm[lo - 1]);
                a.table[(int64_t)lo * a.ld + col_sm[lo] + nth] = page;
                a.counts[page] = 1;
                if (nth == 0 && job_sm[lo] >= 0)
                    a.jobs[job_sm[lo]].y = page;
            }
        }
        before += here;
    }

    bool denied = need > 0 && !served;
    if (r > refused && shares && need == 0) {
        // the page was to be its own, but earlier holders had to stay: it would need one too
        int left = holders;
#pragma unroll 1
        for (int j = 0; j < refused; ++j)
            left -= last_sm[j] == last;
        denied = left > 1;
    }
    if (denied)
        report(a.status, kStatusNoPage);
    if (a.granted != nullptr && r < a.num_reqs)
        a.granted[r] = valid && !denied ? add : 0;
}

struct CopyArgs {
    void *slab[kCompactLayers];
    const int4 *jobs;                           // (from, to, rows)
    const int32_t *num_jobs;
    int64_t page_bytes;
    int layers, row_vecs, pieces;               // 16-byte vectors of a row, pieces of a page
};

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t all = (int64_t)*a.num_jobs * a.layers * a.pieces;
    for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const int piece = (int)(u % a.pieces);
        const int layer = (int)(u / a.pieces % a.layers);
        const int4 job = a.jobs[u / a.pieces / a.layers];
        const int vecs = job.z * a.row_vecs, v0 = piece * kCopyPiece + (int)threadIdx.x;
        if (piece * kCopyPiece >= vecs)
            continue;
        unsigned char *slab = static_cast<unsigned char *>(a.slab[layer]);
        const uint4 *src = reinterpret_cast<const uint4 *>(slab + job.x * a.page_bytes);
        uint4 *dst = reinterpret_cast<uint4 *>(slab + job.y * a.page_bytes);
        uint4 v[kCopyVecs];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j)
            if (v0 + j * kCopyThreads < vecs)
                v[j] = src[v0 + j * kCopyThreads];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j)
            if (v0 + j * kCopyThreads < vecs)
                dst[v0 + j * kCopyThreads] = v[j];
    }
}

}  // namespace

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream)
{
    const int rows = a.out_rows, blocks = rows < kForkCluster ? rows : kForkCluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (rows <= kForkCluster * (kForkBlock / kForkThreads)) {
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3((unsigned)((rows + blocks - 1) / blocks * kForkThreads));
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, fork_kernel<BOTH>, a);
    }
    fork_kernel<HOLD><<<(unsigned)rows, kForkThreads, 0, stream>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kForkThreads);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, fork_kernel<GIVE>, a);
}

cudaError_t launch_free(const int32_t *table, int64_t ld, int64_t cols, int32_t *lens, int rows,
                        int32_t *counts, int64_t num_pages, int32_t *status, cudaStream_t stream)
{
    free_kernel<<<(unsigned)rows, kForkThreads, 0, stream>>>(table, ld, cols, lens, counts,
                                                            num_pages, status);
    return cudaGetLastError();
}

cudaError_t launch_reserve(const ReserveArgs &a, int num_layers, void *const *slabs, bool fp8,
                           int64_t page_bytes, int sms, cudaStream_t stream)
{
    reserve_kernel<<<1, kReserveThreads, 0, stream>>>(a);
    cudaError_t err = cudaGetLastError();
    for (int l0 = 0; l0 < num_layers && err == cudaSuccess; l0 += kCompactLayers) {
        CopyArgs c = {};
        c.layers = num_layers - l0 < kCompactLayers ? num_layers - l0 : kCompactLayers;
        for (int l = 0; l < c.layers; ++l)
            c.slab[l] = slabs[l0 + l];
        c.jobs = a.jobs;
        c.num_jobs = a.num_jobs;
        c.page_bytes = page_bytes;
        c.row_vecs = (fp8 ? kRow : 2 * kRow) / 16;
        c.pieces = (kPageTokens * c.row_vecs + kCopyPiece - 1) / kCopyPiece;
        const int64_t most = (int64_t)a.num_reqs * c.layers * c.pieces;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(most < 8 * sms ? most : 8 * sms));
        cfg.blockDim = dim3(kCopyThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = l0 == 0 ? 1 : 0;
        err = cudaLaunchKernelEx(&cfg, page_copy_kernel, c);
    }
    return err;
}

}  // namespace plmla
