// plmla_rope.cu -- rotary positions: rotation of query (or key) heads, and the
// KV append that rotates the new tokens' rope keys on their way into the pages.
//
// Pair i of a head's rotated part at position p turns by the angle p f_i:
//   (x, y) -> m (x cos a - y sin a, x sin a + y cos a),   a = p f_i
// (Su et al., RoFormer, 2021); m is a magnitude (1, or the attention factor of
// a scaled rotation).  A pair is (x_i, x_{i + d/2}) in the half layout and
// (x_{2i}, x_{2i+1}) in the interleaved one.
//
// Angles.  f_i comes as turns[i] = f_i / (2 pi) in units of 2^-64 turns, so
// p * turns[i] in 64-bit integers wraps modulo whole turns: the reduction of
// the angle is exact for every position, where an fp32 product p f_i would be
// off by 0.06 rad at a million.  (turns itself is as good as a double: below
// 1e-9 rad at a million, a few 1e-7 rad at 2^31.)  The top 32 bits (2^-32 turns) are split into a
// quadrant and a remainder in [-1/8, 1/8) turns before the conversion to fp32,
// which then rounds by at most 2^-26 half turns.
//
// Bound by memory: every element is read and written once.  A block computes
// the (cos, sin) pairs of its tokens once in shared memory and applies them to
// all its heads; its loads are issued before that, so that the trigonometry
// hides behind them.  Instructions count as well as bytes: with 16-bit elements
// converted one by one, units placed by integer divisions and 16 KB in flight per
// block at two blocks an SM, 8,192 tokens of 64 bf16 heads took 38-41 us; converted in
// pairs, placed by multiplications and at four blocks an SM they take 24-25 us (5.5
// TB/s), fp32 heads 40-44 us (6.1-6.7 TB/s).
#include <cuda_fp16.h>

#include "plmla_internal.cuh"

namespace plmla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 2;              // units of one thread in flight
constexpr int kRopeBlocks = 4;              // blocks of an SM
constexpr int kRopeTable = 2048;            // (cos, sin) pairs of one block

// m cos(a), m sin(a) of a = pos * turns (2^-64 turns), negated angle for sign < 0.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, uint64_t turns, float magnitude,
                                               bool inverse)
{
    const uint64_t a = (uint64_t)(int64_t)pos * turns;
    const uint32_t h = (uint32_t)((a + 0x80000000ull) >> 32);   // 2^-32 turns, rounded
    const uint32_t quadrant = (h + 0x20000000u) >> 30;
    const int32_t rem = (int32_t)(h - (quadrant << 30));
    float s, c;
    sincospif((float)rem * 0x1p-31f, &s, &c);
    float cs = (quadrant & 1u) ? s : c, sn = (quadrant & 1u) ? c : s;
    // quadrants 0..3: (c, s), (-s, c), (-c, -s), (s, -c)
    if (quadrant == 1u || quadrant == 2u)
        cs = -cs;
    if (quadrant >= 2u)
        sn = -sn;
    return make_float2(magnitude * cs, magnitude * (inverse ? -sn : sn));
}

// VEC elements of T as one access, widened to and rounded from fp32 a 32-bit word
// (two 16-bit elements) at a time.
template <typename T, int VEC>
struct Vec;

template <int VEC>
struct alignas(4 * VEC) Vec<float, VEC> {
    float v[VEC];
    __device__ __forceinline__ void widen(float (&f)[VEC]) const
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = v[e];
    }
    __device__ __forceinline__ void round(const float (&f)[VEC])
    {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            v[e] = f[e];
    }
};

template <int VEC>
struct alignas(2 * VEC) Vec<__nv_bfloat16, VEC> {
    uint32_t w[VEC / 2];
    __device__ __forceinline__ void widen(float (&f)[VEC]) const
    {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void round(const float (&f)[VEC])
    {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
};

template <int VEC>
struct alignas(2 * VEC) Vec<__half, VEC> {
    __half2 w[VEC / 2];
    __device__ __forceinline__ void widen(float (&f)[VEC]) const
    {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float2 x = __half22float2(w[e]);
            f[2 * e] = x.x;
            f[2 * e + 1] = x.y;
        }
    }
    __device__ __forceinline__ void round(const float (&f)[VEC])
    {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
            w[e] = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
    }
};

template <>
struct Vec<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = __bfloat162float(v); }
    __device__ __forceinline__ void round(const float (&f)[1]) { v = __float2bfloat16_rn(f[0]); }
};

template <>
struct Vec<__half, 1> {
    __half v;
    __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = __half2float(v); }
    __device__ __forceinline__ void round(const float (&f)[1]) { v = __float2half_rn(f[0]); }
};

// u / d by one multiplication, exact for u d < 2^32 (a block's units and rows).
struct Divisor {
    uint32_t d, m;
    Divisor() = default;
    explicit Divisor(uint32_t n) : d(n), m(n > 1 ? (uint32_t)((1ull << 32) / n + 1) : 0u) {}
    __device__ __forceinline__ int div(int u) const
    {
        return m != 0u ? (int)__umulhi((uint32_t)u, m) : u;
    }
};

struct RopeArgs {
    const void *x;
    void *out;
    int64_t tok_stride, head_stride, out_tok_stride, out_head_stride;   // elements
    const int32_t *positions;
    const uint64_t *turns;
    float magnitude;
    int inverse;
    int64_t tokens;
    int heads, half;              // pairs per head
    int tok_block, head_block;    // tokens and heads of one block
    int head_blocks;
    Divisor per_head, by_heads, by_half;   // units of a head, heads, pairs of a head
};

// Block `block` of the rotation: tokens [t0, t0 + tok_block), heads
// [h0, h0 + head_block).  A unit is VEC pairs: two VEC-wide vectors of one head.
// `position(t)` gives token t's position.
template <typename T, int VEC, bool INTER, typename Position>
__device__ __forceinline__ void rope_block(const RopeArgs &a, int64_t block, float2 *table,
                                           Position position)
{
    const int64_t t0 = block / a.head_blocks * a.tok_block;
    const int h0 = (int)(block % a.head_blocks) * a.head_block;
    const int nt = (int)min((int64_t)a.tok_block, a.tokens - t0);
    const int nh = min(a.head_block, a.heads - h0);
    const int per_head = (int)a.per_head.d;
    const int units = nt * nh * per_head;
    const T *in = static_cast<const T *>(a.x);
    T *out = static_cast<T *>(a.out);
    bool have_table = false;
    for (int u0 = threadIdx.x; u0 < units || !have_table; u0 += kRopeThreads * kRopeUnroll) {
        Vec<T, VEC> lo[kRopeUnroll], hi[kRopeUnroll];
        int tok[kRopeUnroll], pair[kRopeUnroll];
        int64_t dst[kRopeUnroll];
#pragma unroll
        for (int j = 0; j < kRopeUnroll; ++j) {
            const int u = u0 + j * kRopeThreads;
            if (u >= units)
                break;
            // a block of several tokens has all the heads
            const int row = a.per_head.div(u);
            tok[j] = nt > 1 ? a.by_heads.div(row) : 0;
            const int h = h0 + row - tok[j] * nh;
            pair[j] = (u - row * per_head) * VEC;
            const int first = INTER ? 2 * pair[j] : pair[j];
            const T *src = in + (t0 + tok[j]) * a.tok_stride + h * a.head_stride + first;
            dst[j] = (t0 + tok[j]) * a.out_tok_stride + h * a.out_head_stride + first;
            lo[j] = *reinterpret_cast<const Vec<T, VEC> *>(src);
            hi[j] = *reinterpret_cast<const Vec<T, VEC> *>(src + (INTER ? VEC : a.half));
        }
        if (!have_table) {
            for (int i = threadIdx.x; i < nt * a.half; i += kRopeThreads) {
                const int t = a.by_half.div(i), p = i - t * a.half;
                table[i] = rope_cos_sin(position(t0 + t), a.turns[p], a.magnitude, a.inverse != 0);
            }
            __syncthreads();
            have_table = true;
        }
#pragma unroll
        for (int j = 0; j < kRopeUnroll; ++j) {
            if (u0 + j * kRopeThreads >= units)
                break;
            const float2 *cs = table + tok[j] * a.half + pair[j];
            float x[VEC], y[VEC], u[VEC], v[VEC];
            lo[j].widen(x);
            hi[j].widen(y);
            if constexpr (INTER && VEC > 1) {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float2 p = cs[e / 2], q = cs[(VEC + e) / 2];
                    u[e] = x[e] * p.x - x[e + 1] * p.y;
                    u[e + 1] = x[e] * p.y + x[e + 1] * p.x;
                    v[e] = y[e] * q.x - y[e + 1] * q.y;
                    v[e + 1] = y[e] * q.y + y[e + 1] * q.x;
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 p = cs[e];
                    u[e] = x[e] * p.x - y[e] * p.y;
                    v[e] = x[e] * p.y + y[e] * p.x;
                }
            }
            Vec<T, VEC> olo, ohi;
            olo.round(u);
            ohi.round(v);
            *reinterpret_cast<Vec<T, VEC> *>(out + dst[j]) = olo;
            *reinterpret_cast<Vec<T, VEC> *>(out + dst[j] + (INTER ? VEC : a.half)) = ohi;
        }
    }
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kernel(const RopeArgs a)
{
    __shared__ float2 table[kRopeTable];
    rope_block<T, VEC, INTER>(a, blockIdx.x, table, [&](int64_t t) { return a.positions[t]; });
}

// Tokens and heads per block, and the grid: a block takes up to kRopeUnroll
// units a thread when that still gives every SM several blocks, else one.
int64_t rope_tiling(RopeArgs *a, int vec, int sms)
{
    const int per_head = a->half / vec;
    a->per_head = Divisor((uint32_t)per_head);
    a->by_heads = Divisor((uint32_t)a->heads);
    a->by_half = Divisor((uint32_t)a->half);
    const int64_t total = a->tokens * a->heads * per_head;
    const int unroll = total >= (int64_t)4 * sms * kRopeThreads * kRopeUnroll ? kRopeUnroll : 1;
    const int want = kRopeThreads * unroll;
    a->head_block = want / per_head > 1 ? want / per_head : 1;
    if (a->head_block > a->heads)
        a->head_block = a->heads;
    int64_t tb = want / (a->head_block * per_head);
    const int64_t fit = kRopeTable / a->half;
    tb = tb > fit ? fit : tb;
    a->tok_block = (int)(tb > 1 ? tb : 1);
    a->head_blocks = (a->heads + a->head_block - 1) / a->head_block;
    return (a->tokens + a->tok_block - 1) / a->tok_block * a->head_blocks;
}

// Whether rows of x and out can be accessed in vectors of `vec` elements of `size` bytes.
bool rope_vectors(const RopeArgs &a, int vec, int size)
{
    const uintptr_t bytes = (uintptr_t)vec * size;
    return a.half % vec == 0 && reinterpret_cast<uintptr_t>(a.x) % bytes == 0 &&
           reinterpret_cast<uintptr_t>(a.out) % bytes == 0 && a.tok_stride % vec == 0 &&
           a.head_stride % vec == 0 && a.out_tok_stride % vec == 0 && a.out_head_stride % vec == 0;
}

// 16-byte accesses where the addresses, the strides and the head's half allow them,
// else single elements.
template <typename T>
cudaError_t launch_typed(RopeArgs a, bool inter, int sms, cudaStream_t stream)
{
    constexpr int wide = 16 / sizeof(T);
    const bool vec = rope_vectors(a, wide, sizeof(T));
    const int64_t blocks = rope_tiling(&a, vec ? wide : 1, sms);
    if (blocks > INT32_MAX)
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)blocks;
    if (vec && inter)
        rope_kernel<T, wide, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else if (vec)
        rope_kernel<T, wide, false><<<grid, kRopeThreads, 0, stream>>>(a);
    else if (inter)
        rope_kernel<T, 1, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else
        rope_kernel<T, 1, false><<<grid, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// rotating append
// ---------------------------------------------------------------------------

struct AppendRopeArgs {
    const uint4 *latent, *rope;
    void *slab;
    int64_t num_pages, page_stride;
    float kv_scale;
    const int32_t *table;
    int64_t table_ld, table_cols;
    const int32_t *seq_lens;
    int num_reqs, n_new;
    int32_t *status;
    const int32_t *positions;     // [num_reqs * n_new], or null: the row's own index
    int64_t rows;
    int append_blocks;            // blocks [0, append_blocks) write rows, the rest rotate queries
};

// One warp per new row, as the plain append; lane i < 32 computes the (cos, sin)
// of pair i, and the eight lanes that hold the 64 rope values fetch theirs by
// shuffles.  Rows that cannot be placed are skipped and reported.
template <bool F8, bool INTER>
__device__ __forceinline__ void append_rope_row(const AppendRopeArgs &a, const RopeArgs &q,
                                                int64_t row)
{
    const int lane = threadIdx.x & 31;
    const int r = (int)(row / a.n_new), j = (int)(row % a.n_new);
    const int64_t p = (int64_t)a.seq_lens[r] - a.n_new + j;
    if (p < 0) {
        if (lane == 0 && a.status != nullptr)
            atomicExch(a.status, kStatusAppendPosition);
        return;
    }
    int page = -1;
    if (p / kPageTokens < a.table_cols)
        page = a.table[(int64_t)r * a.table_ld + p / kPageTokens];
    if (page < 0 || (int64_t)page >= a.num_pages) {
        if (lane == 0 && a.status != nullptr)
            atomicExch(a.status, kStatusAppendPage);
        return;
    }
    const uint4 *sl = a.latent + row * (kLatent / 8);
    const uint4 v0 = __ldg(sl + (F8 ? 2 * lane : lane));
    const uint4 v1 = __ldg(sl + (F8 ? 2 * lane + 1 : lane + 32));
    const uint4 c = __ldg(a.rope + row * (kRope / 8) + (lane & 7));
    const int32_t pos = a.positions != nullptr ? a.positions[row] : (int32_t)p;
    const float2 cs = rope_cos_sin(pos, q.turns[lane], q.magnitude, false);

    // elements 8 l .. 8 l + 7 of the rope part (l = lane & 7), rotated in fp32
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float co = __shfl_sync(0xffffffffu, cs.x, 4 * (lane & 7) + e);
            const float si = __shfl_sync(0xffffffffu, cs.y, 4 * (lane & 7) + e);
            y[2 * e] = x[2 * e] * co - x[2 * e + 1] * si;
            y[2 * e + 1] = x[2 * e] * si + x[2 * e + 1] * co;
        }
    } else {
        const bool second = (lane & 4) != 0;       // holds the pairs' second elements
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float co = __shfl_sync(0xffffffffu, cs.x, 8 * (lane & 3) + e);
            const float si = __shfl_sync(0xffffffffu, cs.y, 8 * (lane & 3) + e);
            const float other = __shfl_xor_sync(0xffffffffu, x[e], 4);
            y[e] = second ? other * si + x[e] * co : x[e] * co - other * si;
        }
    }
    if constexpr (F8) {
        uint8_t *dst = static_cast<uint8_t *>(a.slab) + (int64_t)page * a.page_stride +
                       (p % kPageTokens) * kRow;
        const uint32_t u[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f0 = __fdiv_rn(__uint_as_float(u[2 * i] << 16), a.kv_scale);
            const float f1 = __fdiv_rn(__uint_as_float(u[2 * i] & 0xFFFF0000u), a.kv_scale);
            const float f2 = __fdiv_rn(__uint_as_float(u[2 * i + 1] << 16), a.kv_scale);
            const float f3 = __fdiv_rn(__uint_as_float(u[2 * i + 1] & 0xFFFF0000u), a.kv_scale);
            o[i] = (uint32_t)e4m3x2(f0, f1) | ((uint32_t)e4m3x2(f2, f3) << 16);
        }
        *reinterpret_cast<uint4 *>(dst + 16 * lane) = make_uint4(o[0], o[1], o[2], o[3]);
        if (lane < 8) {
            // the rotated fp32 value is divided and rounded once, to E4M3
            uint32_t k[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                k[i] = (uint32_t)e4m3x2(__fdiv_rn(y[4 * i], a.kv_scale),
                                        __fdiv_rn(y[4 * i + 1], a.kv_scale)) |
                       ((uint32_t)e4m3x2(__fdiv_rn(y[4 * i + 2], a.kv_scale),
                                         __fdiv_rn(y[4 * i + 3], a.kv_scale))
                        << 16);
            *reinterpret_cast<uint2 *>(dst + kLatent + 8 * lane) = make_uint2(k[0], k[1]);
        }
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.slab) +
                                               (int64_t)page * a.page_stride +
                                               (p % kPageTokens) * kRow);
        dst[lane] = v0;
        dst[lane + 32] = v1;
        if (lane < 8) {
            uint32_t k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                k[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
            dst[kLatent / 8 + lane] = make_uint4(k[0], k[1], k[2], k[3]);
        }
    }
}

// The first blocks write the new rows (eight warps, a row each), the rest rotate
// the same tokens' query heads: one launch for the step.
template <bool F8, bool INTER, int VEC>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
append_rope_kernel(const AppendRopeArgs a, const RopeArgs q)
{
    __shared__ float2 table[kRopeTable];
    if ((int)blockIdx.x < a.append_blocks) {
        const int64_t row = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
        if (row < a.rows)
            append_rope_row<F8, INTER>(a, q, row);
        return;
    }
    rope_block<__nv_bfloat16, VEC, INTER>(
        q, (int64_t)blockIdx.x - a.append_blocks, table, [&](int64_t t) -> int32_t {
            if (a.positions != nullptr)
                return a.positions[t];
            return a.seq_lens[t / a.n_new] - a.n_new + (int32_t)(t % a.n_new);
        });
}

template <bool F8, bool INTER>
cudaError_t launch_append_typed(const AppendRopeArgs &a, const RopeArgs &q, bool vec,
                                unsigned grid, cudaStream_t stream)
{
    if (vec)
        append_rope_kernel<F8, INTER, 8><<<grid, kRopeThreads, 0, stream>>>(a, q);
    else
        append_rope_kernel<F8, INTER, 1><<<grid, kRopeThreads, 0, stream>>>(a, q);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeView &v, const int32_t *positions, const uint64_t *turns,
                        float magnitude, int inverse, int dtype, int interleaved, int sms,
                        cudaStream_t stream)
{
    if (v.tokens == 0 || v.heads == 0)
        return cudaSuccess;
    RopeArgs a = {v.x, v.out, v.tok_stride, v.head_stride, v.out_tok_stride, v.out_head_stride,
                  positions, turns, magnitude, inverse, v.tokens, v.heads, v.dim / 2};
    switch (dtype) {
    case kRopeBf16: return launch_typed<__nv_bfloat16>(a, interleaved != 0, sms, stream);
    case kRopeFp16: return launch_typed<__half>(a, interleaved != 0, sms, stream);
    case kRopeFp32: return launch_typed<float>(a, interleaved != 0, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_append_rope(const void *latent, const void *rope, void *slab, bool fp8,
                               int64_t num_pages, int64_t page_stride, float kv_scale,
                               const int32_t *table, int64_t table_ld, int64_t table_cols,
                               const int32_t *seq_lens, int num_reqs, int n_new,
                               const int32_t *positions, const uint64_t *turns, float magnitude,
                               int interleaved, const RopeView &v, int32_t *status, int sms,
                               cudaStream_t stream)
{
    const int64_t rows = (int64_t)num_reqs * n_new;
    if (rows == 0)
        return cudaSuccess;
    RopeArgs q = {v.x, v.out, v.tok_stride, v.head_stride, v.out_tok_stride, v.out_head_stride,
                  positions, turns, magnitude, 0, rows, v.heads, kRope / 2};
    const bool vec = rope_vectors(q, 8, 2);
    const int64_t q_blocks = v.heads > 0 ? rope_tiling(&q, vec ? 8 : 1, sms) : 0;
    const int64_t append_blocks = (rows + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (append_blocks + q_blocks > INT32_MAX)
        return cudaErrorInvalidValue;
    const AppendRopeArgs a = {static_cast<const uint4 *>(latent), static_cast<const uint4 *>(rope),
                              slab, num_pages, page_stride, kv_scale, table, table_ld,
                              table_cols, seq_lens, num_reqs, n_new, status, positions, rows,
                              (int)append_blocks};
    const unsigned grid = (unsigned)(append_blocks + q_blocks);
    if (fp8)
        return interleaved ? launch_append_typed<true, true>(a, q, vec, grid, stream)
                           : launch_append_typed<true, false>(a, q, vec, grid, stream);
    return interleaved ? launch_append_typed<false, true>(a, q, vec, grid, stream)
                       : launch_append_typed<false, false>(a, q, vec, grid, stream);
}

}  // namespace plmla
