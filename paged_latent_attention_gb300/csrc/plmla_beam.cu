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
// row), then the rows'.  Sums over slices, logarithms and candidates are held in pairs of
// floats there: candidates of different rows are compared, and a rounding must not change
// their order.
//
// Bound: latencies, of two launches and of a block's chain (loads, two barriers, the list); the
// logits' bytes are a fifth to a third of it.  128 rows of 150,001 bf16 logits 15.4-16.5 us (5.7 us
// of HBM), 128 of 100,257 fp16 20.9 (3.8; lists of 32), 4 of 32,000 fp32 6.8.
#include <math.h>
#include <algorithm>

#include <cuda_fp16.h>

#include "plmla_internal.cuh"

namespace plmla {
namespace {

constexpr int kSliceThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kCentre = 8.f, kFixed = 0x1p36f, kUnfixed = 0x1p-44f;   // of a slice's terms

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

// 32 bits of logits, kept as they came: 16-bit ones in pairs, compared as pairs (a bound is
// one of the logits, so it has their type) and unpacked for the exponentials alone.
template <typename T>
struct Word;
template <>
struct Word<float> {
    static constexpr int n = 1;
    static constexpr uint32_t none = 0xFF800000u;             // -inf in every element
    __device__ static uint32_t max(uint32_t a, uint32_t b)
    {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ static float get(uint32_t w, int) { return __uint_as_float(w); }
    // of all elements, in any order, added up
    __device__ static uint32_t mark(uint32_t w, uint32_t sum) { return sum + w; }
    __device__ static uint32_t both(float x) { return __float_as_uint(x); }
    // bit e: element e reaches x
    __device__ static uint32_t reach(uint32_t w, uint32_t x)
    {
        return __uint_as_float(w) >= __uint_as_float(x) ? 1u : 0u;
    }
};
template <>
struct Word<__nv_bfloat16> {
    static constexpr int n = 2;
    static constexpr uint32_t none = 0xFF80FF80u;
    __device__ static __nv_bfloat162 as(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
    __device__ static uint32_t max(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 m = __hmax2(as(a), as(b));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    __device__ static float get(uint32_t w, int e)
    {
        return __uint_as_float(e ? w & 0xFFFF0000u : w << 16);
    }
    __device__ static uint32_t mark(uint32_t w, uint32_t sum) { return __dp4a(w, 0xFB01FB01u, sum); }
    __device__ static uint32_t both(float x)
    {
        const uint32_t b = __float_as_uint(x) >> 16;          // x is a bf16
        return b << 16 | b;
    }
    __device__ static uint32_t reach(uint32_t w, uint32_t x)
    {
        const uint32_t m = __hge2_mask(as(w), as(x));
        return (m & 1u) | (m >> 31 << 1);
    }
};
template <>
struct Word<__half> {
    static constexpr int n = 2;
    static constexpr uint32_t none = 0xFC00FC00u;
    __device__ static __half2 as(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
    __device__ static uint32_t max(uint32_t a, uint32_t b)
    {
        const __half2 m = __hmax2(as(a), as(b));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    __device__ static float get(uint32_t w, int e)
    {
        const float2 f = __half22float2(as(w));
        return e ? f.y : f.x;
    }
    __device__ static uint32_t mark(uint32_t w, uint32_t sum) { return __dp4a(w, 0xFB01FB01u, sum); }
    __device__ static uint32_t both(float x)
    {
        const __half2 h = __float2half2_rn(x);                // x is a fp16
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static uint32_t reach(uint32_t w, uint32_t x)
    {
        const uint32_t m = __hge2_mask(as(w), as(x));
        return (m & 1u) | (m >> 31 << 1);
    }
};

// Two floats in one register pair, added and multiplied by one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b)
{
    return fma2(b, pack2(-1.f, -1.f), a);
}

// What the sum of a and b lost (as in two_sum).
__device__ __forceinline__ uint64_t lost2(uint64_t a, uint64_t b, uint64_t sum)
{
    const uint64_t t = sub2(sum, a);
    return add2(sub2(a, sub2(sum, t)), sub2(b, t));
}

// A number as the unevaluated sum of two floats, hi = hi + lo rounded (error-free transforms:
// Dekker, 1971; Knuth, The Art of Computer Programming 2, 4.2.2).  48 bits are plenty here,
// and this device's 64-bit unit is so slow that with it the merge took 25 us.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, float b)
{
    const Pair s = two_sum(a.hi, b);
    const float lo = __fadd_rn(s.lo, a.lo), hi = __fadd_rn(s.hi, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}

__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const Pair s = two_sum(a.hi, b.hi);
    const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s.hi, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}

constexpr float kSameSum = 3e-6f;               // what two logarithms of the same sum may differ by

struct SliceOut {
    float *high, *sum;                  // [rows, slices]
    uint32_t *mark;                     // the same
    uint64_t *lists;                    // [rows, slices, beams] entries, descending
    int slices;
};

// A logit and its token as one number: the larger logit first, then the lower token.  0 is none.
__device__ __forceinline__ uint64_t entry_of(float x, int v)
{
    return (uint64_t)key_of(x) << 32 | (uint32_t)~v;
}

// What a block shares.
struct SliceShared {
    static constexpr int kFew = 512;            // a list that is ranked by counting
    uint64_t list[kFew];
    uint32_t tops[kSliceThreads];
    long long warp_sum[kSliceThreads / 32];
    uint32_t warp_mark[kSliceThreads / 32];
    uint32_t warp_high[kSliceThreads / 32], warp_least[kSliceThreads / 32];
    int warp_i[kSliceThreads / 32];
    uint32_t bound;
    int count;
};

// Slices in which more elements reach the first bound than the list holds: equal logits (masked
// ones, say), or few threads with many.  A tighter bound is the beams'th largest of all
// threads' maxima.  What exceeds it, if that is few, and of what equals it the first in
// element order fill the list; else the block takes the largest out one by one.  The logits
// are read again.  Returns the list's length.
template <typename T, int G>
__device__ __noinline__ int pick_list(const T *head, int v0, int lo, int left, float top, int beams,
                                      SliceShared &s)
{
    constexpr int N = 16 / sizeof(T), kEach = G * N;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    auto id_at = [&](int e) { return (e / N * kSliceThreads + t) * N + e % N; };
    auto in_row = [&](int id) { return id >= lo && id < left; };
    auto logit = [&](int id) { return in_row(id) ? (float)head[v0 + id] : -INFINITY; };
    const uint32_t mine = key_of(top);
    s.tops[t] = mine;
    __syncthreads();                            // and count has been read
    int before = 0;
    for (int j = 0; j < kSliceThreads; ++j)
        before += s.tops[j] > mine || (s.tops[j] == mine && j < t);
    if (before == beams - 1)
        s.bound = mine;
    if (t == 0)
        s.count = 0;
    __syncthreads();
    const uint32_t least = s.bound;
    const float reach = value_of(least);
    for (int e = 0; e < kEach; ++e) {
        const float x = logit(id_at(e));
        if (x > reach) {                        // (-inf past the row)
            const int i = atomicAdd(&s.count, 1);
            if (i < SliceShared::kFew)
                s.list[i] = entry_of(x, v0 + id_at(e));
        }
    }
    __syncthreads();
    int n = s.count;
    if (n <= SliceShared::kFew) {
        for (int g = 0; g < G && n < beams; ++g) {
            int equal = 0;
            for (int e = g * N; e < g * N + N; ++e)
                equal += logit(id_at(e)) == reach && in_row(id_at(e));
            int y = equal;
            for (int w = 1; w < 32; w <<= 1) {
                const int z = __shfl_up_sync(0xffffffffu, y, w);
                if (lane >= w)
                    y += z;
            }
            __syncthreads();                    // the last group's sums have been read
            if (lane == 31)
                s.warp_i[warp] = y;
            __syncthreads();
            int i = n + y - equal;
            for (int w = 0; w < kSliceThreads / 32; ++w) {
                i += w < warp ? s.warp_i[w] : 0;
                n += s.warp_i[w];
            }
            for (int e = g * N; e < g * N + N; ++e)
                if (logit(id_at(e)) == reach && in_row(id_at(e))) {
                    if (i < beams)
                        s.list[i] = entry_of(reach, v0 + id_at(e));
                    ++i;
                }
        }
        __syncthreads();
        return n < beams ? n : s.count > beams ? s.count : beams;
    }
    uint64_t last = ~0ull;
    for (int i = 0; i < beams; ++i) {
        uint64_t best = 0;                      // the first behind the last one taken
        for (int e = 0; e < kEach; ++e) {
            const float x = logit(id_at(e));
            if (x == x && in_row(id_at(e))) {
                const uint64_t k = entry_of(x, v0 + id_at(e));
                best = k < last && k > best ? k : best;
            }
        }
        for (int w = 16; w > 0; w >>= 1) {
            const uint64_t k = __shfl_xor_sync(0xffffffffu, best, w);
            best = k > best ? k : best;
        }
        __syncthreads();                        // the last round's entries have been read
        if (lane == 0) {
            s.tops[2 * warp] = (uint32_t)(best >> 32);
            s.tops[2 * warp + 1] = (uint32_t)best;
        }
        __syncthreads();
        last = 0;
        for (int w = 0; w < kSliceThreads / 32; ++w) {
            const uint64_t k = (uint64_t)s.tops[2 * w] << 32 | s.tops[2 * w + 1];
            last = k > last ? k : last;
        }
        if (t == 0)
            s.list[i] = last;
    }
    __syncthreads();
    return beams;
}

// G groups of 16 bytes a thread: group g of thread t starts at element (g * threads + t) * n of
// the slice (n elements in 16 bytes), so that element order is (group, thread, element).
// Latency-bound: four or five blocks an SM hide each other's loads and barriers (four blocks that
// go on to further slices, whose logits they load ahead: 128 rows of 150,001 bf16 25 us instead of
// the 18 it took then).
template <typename T, int G>
__global__ void __launch_bounds__(kSliceThreads, G == 8 ? 4 : 5)
slice_kernel(const T *logits, int64_t ld, const uint8_t *ended, int beams, int vocab, SliceOut o)
{
    using W = Word<T>;
    constexpr int N = 4 * W::n, kSlice = G * N * kSliceThreads, kWarps = kSliceThreads / 32;
    __shared__ SliceShared s;
    __shared__ uint4 copies[G][kSliceThreads];   // of threads that have candidates
    asm volatile("griddepcontrol.launch_dependents;");
    const int row = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t at = (int64_t)row * o.slices + blockIdx.x;
    if (ended != nullptr && ended[row] != 0)
        return;                                 // its logits count nothing
    // 16-byte groups at aligned addresses, whatever the row's own: element 0 of the first slice
    // lies up to N - 1 elements before the row.  Groups across either end are read by
    // elements.
    const T *head = logits + (int64_t)row * ld;
    const int skip = (int)(reinterpret_cast<uintptr_t>(head) % 16 / sizeof(T));
    // (a last slice that no token reaches is empty)
    const int v0 = (int)min((int64_t)blockIdx.x * kSlice - skip, (int64_t)vocab);
    const int left = (int)min((int64_t)vocab - v0, (int64_t)kSlice), lo = max(0, -v0);
    const T *src = head + v0;
    auto in_row = [&](int id) { return id >= lo && id < left; };
    uint32_t raw[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int e0 = (g * kSliceThreads + t) * N;
        if (e0 >= lo && e0 + N <= left) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src + e0);
            raw[g][0] = v.x, raw[g][1] = v.y, raw[g][2] = v.z, raw[g][3] = v.w;
        } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                raw[g][w] = W::none;
#pragma unroll
                for (int e = 0; e < W::n; ++e) {
                    const int i = e0 + W::n * w + e;
                    if (in_row(i)) {
                        if constexpr (W::n == 1) {
                            raw[g][w] = *reinterpret_cast<const uint32_t *>(src + i);
                        } else {
                            const uint32_t b = *reinterpret_cast<const uint16_t *>(src + i);
                            raw[g][w] = e ? (raw[g][w] & 0xFFFFu) | b << 16
                                          : (raw[g][w] & 0xFFFF0000u) | b;
                        }
                    }
                }
            }
        }
    }
    if (t == 0)
        s.count = 0;
    // this thread's maximum; elements past the row are -inf
    uint32_t most = raw[0][0];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int w = 0; w < 4; ++w)
            most = W::max(most, raw[g][w]);
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < W::n; ++e)
        top = fmaxf(top, W::get(most, e));      // (a NaN is left out)
    const uint32_t top_key = key_of(top), warp_top = __reduce_max_sync(0xffffffffu, top_key);
    // A bound that at least `beams` elements reach: the least of the warps' share'th largest
    // thread maxima.  Only warps count whose every thread has an element (a slice that the
    // row does not fill has fewer; with too few, all of its elements are taken).
    const int skipped = (lo + 32 * N - 1) / (32 * N);
    const int whole = min(left, kSliceThreads * N) / (32 * N) - skipped;
    const int share = whole > 0 ? (beams + whole - 1) / whole : 33;
    uint32_t warp_key = share > 32 ? key_of(-INFINITY) : warp_top;
    {
        uint32_t rest = top_key;
        for (int j = 1; j < share && share <= 32; ++j) {
            const uint32_t first = __ballot_sync(0xffffffffu, rest == warp_key);
            if (lane == __ffs(first) - 1)
                rest = 0;                       // below every key
            warp_key = __reduce_max_sync(0xffffffffu, rest);
        }
    }
    if (lane == 0) {
        s.warp_high[warp] = warp_top;
        s.warp_least[warp] = warp >= skipped && warp < skipped + whole ? warp_key : 0xFFFFFFFFu;
    }
    __syncthreads();
    uint32_t high_key = 0, least = whole > 0 ? 0xFFFFFFFFu : key_of(-INFINITY);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        high_key = max(high_key, s.warp_high[w]);
        least = min(least, s.warp_least[w]);
    }
    const float reach = value_of(least);
    if (top >= reach) {
        const uint32_t x = W::both(reach);
        auto offer = [&](float logit, int id) {
            const int i = atomicAdd(&s.count, 1);
            if (i < SliceShared::kFew)
                s.list[i] = entry_of(logit, v0 + id);
        };
        if constexpr (G == 1) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t hit = W::reach(raw[0][w], x);
#pragma unroll
                for (int e = 0; e < W::n; ++e) {
                    const int id = t * N + W::n * w + e;
                    if ((hit >> e & 1u) != 0 && in_row(id))
                        offer(W::get(raw[0][w], e), id);
                }
            }
        } else {
            // A bit for each element, then a loop over those set: with the offers unrolled over all
            // elements the blocks waited for instructions (128 rows of 150,001 18.2 us, not 16.2;
            // of a single group they are few: 32 rows of 1,000, 32 beams, 9.8 us, in a loop 10.3).
            unsigned long long hits = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                copies[g][t] = make_uint4(raw[g][0], raw[g][1], raw[g][2], raw[g][3]);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    hits |= (unsigned long long)W::reach(raw[g][w], x) << (g * N + w * W::n);
            }
#pragma unroll 1
            for (; hits != 0; hits &= hits - 1) {
                const int bit = __ffsll((long long)hits) - 1, g = bit / N, e = bit % N;
                const int id = (g * kSliceThreads + t) * N + e;
                if (in_row(id))
                    offer((float)reinterpret_cast<const T *>(&copies[g][t])[e], id);
            }
        }
    }
    // Sum of exponentials of d = x - high, each 2^kCentre times itself: the argument d log2 e + kCentre
    // is then near 0, where its rounding is small, for the terms that a large vocabulary is
    // made of (d = -11: half a step of 2^-22 instead of 2^-20, which many equal logits, all
    // rounded alike, would carry into the sum).  Added as a tree for the same reason; across threads
    // in fixed point, without a rounding.
    const float high = value_of(high_key), ref = high == -INFINITY ? 0.f : high;
    float own;
    uint32_t mark = 0;
    {
        const uint64_t shift = pack2(-ref, -ref), scale = pack2(kLog2e, kLog2e);
        const uint64_t centre = pack2(kCentre, kCentre);
        uint64_t sums[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint64_t e[4];
#pragma unroll
            for (int w = 0; w < 2 * W::n; ++w) {
                const uint64_t v = W::n == 2 ? pack2(W::get(raw[g][w], 0), W::get(raw[g][w], 1))
                                             : pack2(W::get(raw[g][2 * w % 4], 0),
                                                     W::get(raw[g][(2 * w + 1) % 4], 0));
                const uint64_t d = add2(v, shift);
                uint64_t p = fma2(d, scale, centre);
                float x, y;
                if constexpr (W::n == 1) {
                    // what d lost (16-bit logits differ exactly, but for those next to 0); it is not a
                    // number where d is -inf
                    unpack2(lost2(v, shift, d), x, y);
                    p = fma2(pack2(fminf(x, 0x1p-18f), fminf(y, 0x1p-18f)), scale, p);
                }
                unpack2(p, x, y);
                e[w] = pack2(fast_exp2(x), fast_exp2(y));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w)
                mark = W::mark(raw[g][w], mark);
            sums[g] = add2(e[0], e[1]);
            if constexpr (W::n == 2)
                sums[g] = add2(sums[g], add2(e[2], e[3]));
        }
#pragma unroll
        for (int w = 1; w < G; w *= 2)
#pragma unroll
            for (int g = 0; g < G; g += 2 * w)
                sums[g] = add2(sums[g], sums[g + w]);
        float x, y;
        unpack2(sums[0], x, y);
        own = x + y;
    }
    // (a thread's sum is 2^14 at most: 23 bits above the lower 27)
    const unsigned long long fixed = __float2ull_rn(own * kFixed);
    const uint32_t sum_lo = __reduce_add_sync(0xffffffffu, (uint32_t)fixed & 0x7FFFFFFu);
    const uint32_t sum_hi = __reduce_add_sync(0xffffffffu, (uint32_t)(fixed >> 27));
    const bool nan = __any_sync(0xffffffffu, own != own);
    mark = __reduce_add_sync(0xffffffffu, mark);
    if (lane == 0) {
        s.warp_mark[warp] = mark;
        s.warp_sum[warp] = nan ? -1 : ((long long)sum_hi << 27) + sum_lo;
    }
    __syncthreads();
    if (t == 0) {
        bool bad = false;
        long long sum = 0;
        mark = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mark += s.warp_mark[w];
            sum += s.warp_sum[w];
            bad |= s.warp_sum[w] < 0;
        }
        o.high[at] = high;
        o.mark[at] = mark;
        o.sum[at] = bad ? NAN : __ll2float_rn(sum) * kUnfixed;
    }
    int n = s.count;
    if (n > SliceShared::kFew)
        n = pick_list<T, G>(head, v0, lo, left, top, beams, s);
    for (int i = t; i < max(n, beams); i += kSliceThreads) {
        const uint64_t k = i < n ? s.list[i] : 0;
        int rank = i < n ? 0 : i;
        if (i < n)
#pragma unroll 8
            for (int j = 0; j < n; ++j)
                rank += s.list[j] > k;
        if (rank < beams)
            o.lists[at * beams + rank] = k;
    }
}

// Lists of 32 P entries in descending order, entry p * 32 + lane in register p of a lane: the
// upper 32 P of this list and another, whose entries come in ascending order (a bitonic
// merge).  An entry is a number, or (key, id): the larger key first, then the lower id.
template <typename A>
__device__ __forceinline__ bool before(A a, A b)
{
    return a > b;
}
struct Candidate {
    unsigned long long key;
    int id;
};
__device__ __forceinline__ bool before(Candidate a, Candidate b)
{
    return a.key > b.key || (a.key == b.key && a.id < b.id);
}
__device__ __forceinline__ uint64_t shuffle_xor(uint64_t a, int w)
{
    return __shfl_xor_sync(0xffffffffu, a, w);
}
__device__ __forceinline__ Candidate shuffle_xor(Candidate a, int w)
{
    return {__shfl_xor_sync(0xffffffffu, a.key, w), __shfl_xor_sync(0xffffffffu, a.id, w)};
}

template <int P, typename A>
__device__ __forceinline__ void join(A (&list)[P], const A (&other)[P])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (before(other[p], list[p]))
            list[p] = other[p];
    if constexpr (P == 2) {
        if (before(list[1], list[0])) {
            const A x = list[0];
            list[0] = list[1];
            list[1] = x;
        }
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const A x = shuffle_xor(list[p], w);
            if (before(x, list[p]) == ((lane & w) == 0))
                list[p] = x;
        }
}

__device__ __forceinline__ Pair product(float a, float b)
{
    const float hi = __fmul_rn(a, b);
    return {hi, fmaf(a, b, -hi)};
}

// ln s of a positive sum: s = 2^e m with m around 1; ln 2 in a part whose products with e are
// exact and a rest.  Off by some 2^-25.
__device__ __forceinline__ Pair ln(float s)
{
    constexpr float kLn2Hi = 2839.f / 4096.f;
    constexpr float kLn2Lo = (float)(0.69314718055994530942 - 2839.0 / 4096.0);
    int e;
    float m = frexpf(s, &e);                    // [1/2, 1)
    if (m < 0.70710678f) {
        m *= 2.f;
        --e;
    }
    return add(two_sum((float)e * kLn2Hi, logf(m)), (float)e * kLn2Lo);
}

// Keys in the order of pairs.  -inf, alone in hi, is above 0, which stands for no candidate.
__device__ __forceinline__ unsigned long long wide_key(Pair x)
{
    return (unsigned long long)key_of(x.hi) << 32 | key_of(x.lo);
}
__device__ __forceinline__ float wide_value(unsigned long long k)
{
    return value_of((uint32_t)(k >> 32));       // lo is below half a unit of hi
}

template <int P, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) merge_kernel(const BeamArgs a, const SliceOut o)
{
    constexpr int kWarps = WARPS, kList = 32 * P;
    __shared__ unsigned long long keys[kWarps * kList / 2];
    __shared__ int ids[kWarps * kList / 2];
    __shared__ Pair logs[kMaxBeams];            // of the rows' sums
    __shared__ float tops[kMaxBeams];           // their largest logits; NaN: no candidates
    __shared__ uint32_t marks[kMaxBeams];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
    const int K = a.beams, per_row = K >= kWarps ? 1 : kWarps / K;
    const int part = warp % per_row;
    const Candidate none = {0, 0x7FFFFFFF};     // below -inf
    Candidate best[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
        best[p] = none;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint64_t next[P];
    auto fetch = [&](int64_t row, int s) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = kList - 1 - (32 * p + lane);        // ascending for join
            next[p] = s < o.slices && i < K ? o.lists[(row * o.slices + s) * K + i] : 0;
        }
    };
    // this warp's first list is on its way while the sums are taken, a warp a row
    if (warp / per_row < K)
        fetch((int64_t)b * K + warp / per_row, part);
    for (int k = warp; k < K; k += kWarps) {
        const int64_t row = (int64_t)b * K + k;
        float high = -INFINITY;
        Pair sum = {0.f, 0.f};
        uint32_t mark = 0;
        if (a.ended == nullptr || a.ended[row] == 0) {
            for (int s = lane; s < o.slices; s += 32) {
                high = fmaxf(high, o.high[row * o.slices + s]);
                mark += o.mark[row * o.slices + s];
            }
            mark = __reduce_add_sync(0xffffffffu, mark);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1)
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, w));
            for (int s = lane; s < o.slices; s += 32) {
                const float h = o.high[row * o.slices + s];
                // (a NaN among the logits is in the sum, not in the maximum)
                const Pair d = two_sum(h, -high);
                const float e = h == high ? 1.f : expf(h - high);
                const float more = h == high || e == 0.f ? 0.f : d.lo;
                sum = add(sum, product(fmaf(e, more, e), o.sum[row * o.slices + s]));
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) {
                const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, w);
                const float lo = __shfl_xor_sync(0xffffffffu, sum.lo, w);
                sum = add(sum, Pair{hi, lo});                 // the same in both lanes
            }
        }
        if (lane == 0) {
            const Pair l = ln(sum.hi);
            logs[k] = {l.hi, l.lo + sum.lo / sum.hi};
            marks[k] = mark;
            tops[k] = isfinite(sum.hi) && sum.hi > 0.f ? high : NAN;
        }
    }
    __syncthreads();
    for (int k = warp / per_row; k < K; k += kWarps / per_row) {
        const int64_t row = (int64_t)b * K + k;
        if (k >= kWarps / per_row)
            fetch(row, part);
        const float score = a.scores[row], high = tops[k];
        const bool ended = a.ended != nullptr && a.ended[row] != 0;
        // Rows with the same logits have to have the same sum, so that ties stay ties, but what is
        // added first depends on where they start within 16 bytes: the first one's is taken.
        // (Known by their marks: the largest logit and the sum alone can be close in rows of
        // nearly equal logits.)
        Pair l = logs[k];
        int same = K;
#pragma unroll
        for (int j0 = 0; j0 < 32 * P; j0 += 32) {
            const int j = min(j0 + lane, k);
            const bool alike = marks[j] == marks[k] && tops[j] == high &&
                               fabsf((logs[j].hi - l.hi) + (logs[j].lo - l.lo)) <= kSameSum;
            const uint32_t found = __ballot_sync(0xffffffffu, alike);
            if (same == K && found != 0)
                same = min(j0 + __ffs(found) - 1, k);
        }
        l = logs[min(same, k)];
        Pair shift = add(add(two_sum(score, -high), -l.hi), -l.lo);
        if (!isfinite(high))
            shift.hi = -INFINITY;
        Candidate mine[P];
        if (!isfinite(shift.hi) || ended) {
            // its first tokens in order, at -inf; an ended beam's end token before them
            const bool end = ended && isfinite(score);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = kList - 1 - (32 * p + lane);
                const bool is_end = end && i == 0;
                const int v = is_end ? a.end_token : end && i - 1 < a.end_token ? i - 1 : i;
                mine[p] = none;
                if (part == 0 && i < K && v < a.vocab)
                    mine[p] = {wide_key({is_end ? score : -INFINITY, 0.f}), k * a.vocab + v};
            }
        } else {
            // its slices by logits (a part in each warp of the row)
            uint64_t list[P];
#pragma unroll
            for (int p = 0; p < P; ++p)
                list[p] = 0;
            for (int s = part; s < o.slices; s += per_row) {
                uint64_t now[P];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    now[p] = next[p];
                fetch(row, s + per_row);
                join<P>(list, now);
            }
            // as candidates, in ascending order: entry i comes from kList - 1 - i
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint64_t x = __shfl_sync(0xffffffffu, list[P - 1 - p], 31 - lane);
                const int v = (int)~(uint32_t)x;
                Pair c = add(shift, value_of((uint32_t)(x >> 32)));
                if (!isfinite(c.hi))
                    c = {-INFINITY, 0.f};       // a masked token
                mine[p] = none;
                if (x != 0)
                    mine[p] = {wide_key(c), k * a.vocab + v};
            }
        }
        join<P>(best, mine);
    }
    // the warps' lists: the upper half hands its lists to the lower half
#pragma unroll 1
    for (int half = kWarps / 2; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                keys[(warp - half) * kList + 32 * p + lane] = best[p].key;
                ids[(warp - half) * kList + 32 * p + lane] = best[p].id;
            }
        __syncthreads();
        if (warp < half) {
            Candidate other[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = kList - 1 - (32 * p + lane);
                other[p] = {keys[warp * kList + i], ids[warp * kList + i]};
            }
            join<P>(best, other);
        }
        __syncthreads();
    }
    if (warp == 0)
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (32 * p + lane < K) {
                const int64_t at = (int64_t)b * K + 32 * p + lane;
                a.tokens[at] = best[p].id % a.vocab;
                a.parents[at] = b * K + best[p].id / a.vocab;
                a.out_scores[at] = wide_value(best[p].key);
            }
}

// Groups of 16 bytes a thread: one where that holds a row (2,000 rows of 2,000 bf16 tokens: 14.6
// us; of four groups 19, of eight 26), four where those do (7,000: 18.3; one 34, eight 26), else
// eight (512 fp32 rows of 32,000: 21.4; four 25.5, one 46).  With few rows shorter slices on more
// SMs gain nothing, since the merge has more lists: 4 rows of 150,000 bf16 tokens 8.4 us, in
// slices of four groups 9.6, of one 12.5.
int thread_groups(int vocab, int type)
{
    const int one = (type == kRopeFp32 ? 4 : 8) * kSliceThreads;
    return vocab > 4 * one ? 8 : vocab > one ? 4 : 1;
}

int slice_count(int vocab, int type)
{
    const int group = type == kRopeFp32 ? 4 : 8;
    const int slice = thread_groups(vocab, type) * group * kSliceThreads;
    return (int)(((int64_t)vocab + group - 2) / slice + 1);   // a row may start inside a group
}

template <typename T>
void launch_slices(const BeamArgs &a, int groups, const SliceOut &o, cudaStream_t stream)
{
    const T *x = static_cast<const T *>(a.logits);
    const dim3 grid((unsigned)o.slices, (unsigned)(a.batch * a.beams));
    if (groups == 8)
        slice_kernel<T, 8><<<grid, kSliceThreads, 0, stream>>>(x, a.ld, a.ended, a.beams, a.vocab,
                                                               o);
    else if (groups == 4)
        slice_kernel<T, 4><<<grid, kSliceThreads, 0, stream>>>(x, a.ld, a.ended, a.beams, a.vocab,
                                                               o);
    else
        slice_kernel<T, 1><<<grid, kSliceThreads, 0, stream>>>(x, a.ld, a.ended, a.beams, a.vocab,
                                                               o);
}

}  // namespace

size_t beam_workspace(int batch, int beams, int vocab)
{
    const size_t rows = (size_t)batch * beams;
    // fp32 slices are half as long, but hold rows of a length that 16-bit ones cut at less
    const int slices = std::max(slice_count(vocab, kRopeFp32), slice_count(vocab, kRopeBf16));
    return rows * slices * (8 * (size_t)beams + 12);
}

cudaError_t launch_beams(const BeamArgs &a, void *workspace, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.batch * a.beams;
    SliceOut o;
    o.slices = slice_count(a.vocab, a.type);
    const int64_t lists = rows * o.slices;
    o.lists = static_cast<uint64_t *>(workspace);
    o.high = reinterpret_cast<float *>(o.lists + lists * a.beams);
    o.sum = o.high + lists;
    o.mark = reinterpret_cast<uint32_t *>(o.sum + lists);
    const int groups = thread_groups(a.vocab, a.type);
    if (a.type == kRopeBf16)
        launch_slices<__nv_bfloat16>(a, groups, o, stream);
    else if (a.type == kRopeFp16)
        launch_slices<__half>(a, groups, o, stream);
    else
        launch_slices<float>(a, groups, o, stream);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    // Eight warps where each has one beam at most and few lists, else 32: fewer levels of joins,
    // and more blocks an SM (4 beams of 2,000 tokens 6.0 us, not 7.8, 500 times 4 of 1,000 14, not
    // 30, 4 of 150,000 8.4, not 9.6; but 32 of 1,000 12.8, not 9.8, 32 of 30,000 15.8, not 11.7).
    const bool few = a.beams <= 8 && a.beams * (int64_t)o.slices <= 64;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch);
    cfg.blockDim = dim3(few ? 256 : 1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = few ? merge_kernel<1, 8> : a.beams <= 32 ? merge_kernel<1, 32> : merge_kernel<2, 32>;
    return cudaLaunchKernelEx(&cfg, kernel, a, o);
}

}  // namespace plmla
