// plmla_beam.cu -- beam search's selection over beams and vocabulary.
//
//   cand[b, k, v] = scores[b, k] + x[b, k, v] - ln sum_u exp x[b, k, u]
//
// and of a batch entry's beams * vocab candidates the `beams` largest, ties to the lowest
// k * vocab + v.  A beam that has ended offers its end token alone, at its score; a beam whose
// score or log-sum-exp is not finite (an unused beam, a row with NaN) offers nothing: its
// candidates are -inf, which count only where too few others exist.
//
// The logits are read once.  slice_kernel: a block holds a slice of a row in registers, takes
// its maximum and sum of exponentials, and its `beams` largest logits: the beams'th
// largest of the threads' maxima is a bound that few elements reach, those go to a list in
// shared memory, and the list is ranked by counting.  A row's order by logits is its order
// by candidates, so no more than `beams` of a slice can matter.  merge_kernel: a block per
// batch entry joins each row's sorted lists by bitonic merges in registers (a warp per
// row), then the rows'.  Sums over slices, logarithms and candidates are held in 64 bits there:
// candidates of different rows are compared, and a rounding must not change their order.
//
// Bound: HBM for the logits of a large batch; else latency of two launches.
#include <math.h>

#include <cuda_fp16.h>

#include "plmla_internal.cuh"

namespace plmla {
namespace {

constexpr int kSliceThreads = 256;
constexpr int kMergeThreads = 1024;
constexpr float kLog2e = 1.4426950408889634f;

// A 32-bit key in the order of the floats (-0 as 0, so that equal logits tie).
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// 16 bytes of logits as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    __device__ static void load(const float *p, float (&x)[4])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    __device__ static float one(const float *p) { return *p; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static void load(const __nv_bfloat16 *p, float (&x)[8])
    {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
};
template <>
struct Vec<__half> {
    static constexpr int n = 8;
    __device__ static void load(const __half *p, float (&x)[8])
    {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ static float one(const __half *p) { return __half2float(*p); }
};

struct SliceOut {
    float *high, *sum;                  // [rows, slices]
    uint32_t *keys;                     // [rows, slices, beams], descending
    int32_t *ids;
    int slices;
};

// E logits a thread, in groups of 16 bytes: group g of thread t starts at element
// (g * threads + t) * n of the slice, so that element order is (group, thread, element).
template <typename T, int E>
__global__ void __launch_bounds__(kSliceThreads)
slice_kernel(const T *logits, int64_t ld, const uint8_t *ended, int beams, int vocab, int vec_ok,
             SliceOut o)
{
    constexpr int N = Vec<T>::n, G = E / N, kSlice = E * kSliceThreads;
    constexpr int kCap = 2048 + 4 * kMaxBeams;
    __shared__ uint32_t keys[kCap];
    __shared__ int32_t ids[kCap];
    __shared__ alignas(16) uint32_t tops[kSliceThreads];
    __shared__ float warp_f[kSliceThreads / 32];
    __shared__ int warp_i[kSliceThreads / 32];
    __shared__ uint32_t bound;
    __shared__ int count, ties;
    asm volatile("griddepcontrol.launch_dependents;");
    const int row = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t at = (int64_t)row * o.slices + blockIdx.x;
    if (ended != nullptr && ended[row] != 0)
        return;                                 // its logits count nothing
    const int v0 = blockIdx.x * kSlice, left = vocab - v0;
    const T *src = logits + (int64_t)row * ld + v0;
    float x[E];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int e0 = (g * kSliceThreads + t) * N;
        float v[N];
        if (vec_ok && e0 + N <= left) {
            Vec<T>::load(src + e0, v);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[e] = e0 + e < left ? Vec<T>::one(src + e0 + e) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[g * N + e] = v[e];
    }
    // the slice's maximum and sum; elements past the row are -inf and add nothing
    float high = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e)
        high = fmaxf(high, x[e]);
    const uint32_t top = key_of(high);
    float m = high;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    if (lane == 0)
        warp_f[warp] = m;
    tops[t] = top;
    if (t == 0) {
        count = ties = 0;
        bound = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSliceThreads / 32; ++w)
        m = fmaxf(m, warp_f[w]);
    // the beams'th largest of the threads' maxima: at least that many elements reach it
    {
        int above = 0;
        const uint4 *p = reinterpret_cast<const uint4 *>(tops);
#pragma unroll 8
        for (int j = 0; j < kSliceThreads / 4; ++j) {
            const uint4 k = p[j];
            above += (k.x > top || (k.x == top && 4 * j < t)) +
                     (k.y > top || (k.y == top && 4 * j + 1 < t)) +
                     (k.z > top || (k.z == top && 4 * j + 2 < t)) +
                     (k.w > top || (k.w == top && 4 * j + 3 < t));
        }
        if (above == beams - 1)
            bound = top;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        sum += fast_exp2((x[e] - ref) * kLog2e);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, w);
    __syncthreads();                            // the maxima have been read, the bound is set
    if (lane == 0)
        warp_f[warp] = sum;
    const uint32_t least = bound;
    // elements above the bound: at most beams - 1 threads have any, so at most
    // (kMaxBeams - 1) * E <= kCap of them (more only in a row with NaN, which counts nothing)
    if (top >= least) {
        int equal = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t k = key_of(x[e]);
            const int id = ((e / N) * kSliceThreads + t) * N + e % N;
            if (k > least && id < left) {
                const int i = atomicAdd(&count, 1);
                if (i < kCap) {
                    keys[i] = k;
                    ids[i] = v0 + id;
                }
            }
            equal += k == least && id < left ? 1 : 0;
        }
        if (equal != 0)
            atomicAdd(&ties, equal);
    }
    __syncthreads();
    if (t == 0) {
        float s = 0.f;
        for (int w = 0; w < kSliceThreads / 32; ++w)
            s += warp_f[w];
        o.high[at] = m;
        o.sum[at] = s;
    }
    // elements at the bound fill the list up: all of them where they are few (the ranking
    // puts them in order), else the first ones in element order
    const int above = min(count, kCap), equal = ties;
    int n = above;
    if (above < beams && equal <= 4 * kMaxBeams) {
        __syncthreads();                        // count has been read
        if (top >= least) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int id = ((e / N) * kSliceThreads + t) * N + e % N;
                if (key_of(x[e]) == least && id < left) {
                    const int i = atomicAdd(&count, 1);
                    keys[i] = least;
                    ids[i] = v0 + id;
                }
            }
        }
        n = above + equal;
    } else if (above < beams) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            int mine = 0;
#pragma unroll
            for (int e = 0; e < N; ++e)
                mine += key_of(x[g * N + e]) == least && (g * kSliceThreads + t) * N + e < left;
            int y = mine;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const int z = __shfl_up_sync(0xffffffffu, y, w);
                if (lane >= w)
                    y += z;
            }
            __syncthreads();                    // the last group's sums have been read
            if (lane == 31)
                warp_i[warp] = y;
            __syncthreads();
            int i = n + y - mine;
            for (int w = 0; w < kSliceThreads / 32; ++w) {
                i += w < warp ? warp_i[w] : 0;
                n += warp_i[w];
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int id = (g * kSliceThreads + t) * N + e;
                if (key_of(x[g * N + e]) == least && id < left) {
                    if (i < beams) {
                        keys[i] = least;
                        ids[i] = v0 + id;
                    }
                    ++i;
                }
            }
        }
        n = min(n, beams);
    }
    __syncthreads();
    for (int i = t; i < max(n, beams); i += kSliceThreads) {
        int rank = i;
        uint32_t k = 0;
        int id = 0x7FFFFFFF;
        if (i < n) {
            k = keys[i];
            id = ids[i];
            rank = 0;
            for (int j = 0; j < n; ++j)
                rank += keys[j] > k || (keys[j] == k && ids[j] < id);
        }
        if (rank < beams) {
            o.keys[at * beams + rank] = k;
            o.ids[at * beams + rank] = id;
        }
    }
}

// Lists of 32 P entries in descending order, entry p * 32 + lane in register p of a lane.
// An entry is (key, id): the larger key first, then the lower id.
template <typename K>
__device__ __forceinline__ bool before(K k, int id, K k2, int id2)
{
    return k > k2 || (k == k2 && id < id2);
}

// The upper 32 P of this list and another, whose entries come in ascending order.
template <int P, typename K>
__device__ __forceinline__ void join(K (&k)[P], int (&id)[P], const K (&k2)[P], const int (&id2)[P])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (before(k2[p], id2[p], k[p], id[p])) {
            k[p] = k2[p];
            id[p] = id2[p];
        }
    if constexpr (P == 2) {
        if (before(k[1], id[1], k[0], id[0])) {
            const K x = k[0];
            const int y = id[0];
            k[0] = k[1], id[0] = id[1];
            k[1] = x, id[1] = y;
        }
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const K x = __shfl_xor_sync(0xffffffffu, k[p], w);
            const int y = __shfl_xor_sync(0xffffffffu, id[p], w);
            if (before(x, y, k[p], id[p]) == ((lane & w) == 0)) {
                k[p] = x;
                id[p] = y;
            }
        }
}

__device__ __forceinline__ unsigned long long wide_key(double x)
{
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double wide_value(unsigned long long k)
{
    return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

template <int P>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const BeamArgs a, const SliceOut o)
{
    constexpr int kWarps = kMergeThreads / 32, kList = 32 * P;
    __shared__ unsigned long long keys[kWarps * kList / 2];
    __shared__ int ids[kWarps * kList / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
    const int K = a.beams, per_row = K >= kWarps ? 1 : kWarps / K;
    const int part = warp % per_row;
    unsigned long long best[P];
    int flat[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        best[p] = 0;                            // no candidate: below -inf
        flat[p] = 0x7FFFFFFF;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = warp / per_row; k < K; k += kWarps / per_row) {
        const int64_t row = (int64_t)b * K + k;
        const double score = (double)a.scores[row];
        const bool ended = a.ended != nullptr && a.ended[row] != 0;
        unsigned long long wk[P];
        int wi[P];
        double shift = score;
        if (!ended) {
            float high = -INFINITY;
            for (int s = lane; s < o.slices; s += 32)
                high = fmaxf(high, o.high[row * o.slices + s]);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1)
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, w));
            double sum = 0.0;
            for (int s = lane; s < o.slices; s += 32) {
                const float h = o.high[row * o.slices + s];
                // (a NaN among the logits is in the sum, not in the maximum)
                const double e = h == high ? 1.0 : exp((double)h - (double)high);
                sum += e * (double)o.sum[row * o.slices + s];
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, w);
            shift = score - ((double)high + log(sum));
        }
        if (!isfinite(shift) || ended) {
            // its first tokens in order, at -inf; an ended beam's end token before them
            const bool end = ended && isfinite(shift);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = kList - 1 - (32 * p + lane);          // ascending for join
                const bool is_end = end && i == 0;
                const int v = is_end ? a.end_token : end && i - 1 < a.end_token ? i - 1 : i;
                const bool in = part == 0 && i < K && v < a.vocab;
                wk[p] = !in ? 0 : wide_key(is_end ? score : -(double)INFINITY);
                wi[p] = !in ? 0x7FFFFFFF : k * a.vocab + v;
            }
            join<P>(best, flat, wk, wi);
            continue;
        }
        // this warp's slices of the row by logits (a part in each warp of the row)
        uint32_t key[P];
        int id[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            key[p] = 0;
            id[p] = 0x7FFFFFFF;
        }
        for (int s = part; s < o.slices; s += per_row) {
            const int64_t at = (row * o.slices + s) * K;
            uint32_t k2[P];
            int id2[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = kList - 1 - (32 * p + lane);
                k2[p] = i < K ? o.keys[at + i] : 0;
                id2[p] = i < K ? o.ids[at + i] : 0x7FFFFFFF;
            }
            join<P>(key, id, k2, id2);
        }
        // as candidates, in ascending order: entry i comes from kList - 1 - i
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint32_t x = __shfl_sync(0xffffffffu, key[P - 1 - p], 31 - lane);
            const int v = __shfl_sync(0xffffffffu, id[P - 1 - p], 31 - lane);
            const bool in = x != 0 && v < a.vocab;
            wk[p] = in ? wide_key((double)value_of(x) + shift) : 0;
            wi[p] = in ? k * a.vocab + v : 0x7FFFFFFF;
        }
        join<P>(best, flat, wk, wi);
    }
    // the warps' lists: the upper half hands its lists to the lower half
#pragma unroll 1
    for (int half = kWarps / 2; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                keys[(warp - half) * kList + 32 * p + lane] = best[p];
                ids[(warp - half) * kList + 32 * p + lane] = flat[p];
            }
        __syncthreads();
        if (warp < half) {
            unsigned long long wk[P];
            int wi[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = kList - 1 - (32 * p + lane);
                wk[p] = keys[warp * kList + i];
                wi[p] = ids[warp * kList + i];
            }
            join<P>(best, flat, wk, wi);
        }
        __syncthreads();
    }
    if (warp == 0)
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (32 * p + lane < K) {
                const int64_t at = (int64_t)b * K + 32 * p + lane;
                a.tokens[at] = flat[p] % a.vocab;
                a.parents[at] = b * K + flat[p] / a.vocab;
                a.out_scores[at] = (float)wide_value(best[p]);
            }
}

// Logits a thread: slices of 8,192 where they fill the device, else of 2,048, so that a few
// rows are read by more SMs.
int thread_logits(int64_t rows, int vocab, int sms)
{
    constexpr int wide = 32 * kSliceThreads;
    return rows * ((vocab + wide - 1) / wide) >= sms ? 32 : 8;
}

int slice_count(int64_t rows, int vocab, int sms)
{
    const int slice = thread_logits(rows, vocab, sms) * kSliceThreads;
    return (vocab + slice - 1) / slice;
}

template <typename T>
void launch_slices(const BeamArgs &a, int wide, const SliceOut &o, cudaStream_t stream)
{
    const T *x = static_cast<const T *>(a.logits);
    const int vec_ok = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && a.ld * sizeof(T) % 16 == 0;
    const dim3 grid((unsigned)o.slices, (unsigned)(a.batch * a.beams));
    if (wide)
        slice_kernel<T, 32><<<grid, kSliceThreads, 0, stream>>>(x, a.ld, a.ended, a.beams, a.vocab,
                                                                vec_ok, o);
    else
        slice_kernel<T, 8><<<grid, kSliceThreads, 0, stream>>>(x, a.ld, a.ended, a.beams, a.vocab,
                                                               vec_ok, o);
}

}  // namespace

size_t beam_workspace(int batch, int beams, int vocab, int sms)
{
    const size_t rows = (size_t)batch * beams;
    return rows * slice_count((int64_t)rows, vocab, sms) * 8 * (1 + (size_t)beams);
}

cudaError_t launch_beams(const BeamArgs &a, void *workspace, int sms, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.batch * a.beams;
    SliceOut o;
    o.slices = slice_count(rows, a.vocab, sms);
    const int64_t lists = rows * o.slices;
    o.high = static_cast<float *>(workspace);
    o.sum = o.high + lists;
    o.keys = reinterpret_cast<uint32_t *>(o.sum + lists);
    o.ids = reinterpret_cast<int32_t *>(o.keys + lists * a.beams);
    const int wide = thread_logits(rows, a.vocab, sms) == 32;
    if (a.type == kRopeBf16)
        launch_slices<__nv_bfloat16>(a, wide, o, stream);
    else if (a.type == kRopeFp16)
        launch_slices<__half>(a, wide, o, stream);
    else
        launch_slices<float>(a, wide, o, stream);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.beams <= 32 ? cudaLaunchKernelEx(&cfg, merge_kernel<1>, a, o)
                         : cudaLaunchKernelEx(&cfg, merge_kernel<2>, a, o);
}

}  // namespace plmla
