// plmla_branch_abi.cu -- host side of the entries for several continuations of one prompt
// (decode with shared prefixes, page ownership, beam selection), declared in include/plmla.h.
//
// Arguments are checked and the kernels enqueued on the caller's stream; nothing here
// allocates device memory, synchronises, or reads device data back.
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "plmla.h"
#include "plmla_internal.cuh"

using namespace plmla;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SMs of the current device (kept per device), or 0.
int device_sms()
{
    static std::atomic<int> cached[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0)
        return 0;
    if (dev < 64 && (sms = cached[dev].load(std::memory_order_relaxed)) > 0)
        return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (dev < 64)
        cached[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

bool table_ok(const int32_t *table, int64_t ld, int64_t cols, int32_t rows)
{
    return table != nullptr && aligned(table, 4) && cols >= 1 && ld >= cols && rows >= 1 &&
           rows <= kMaxReqs;
}

bool words_ok(const int32_t *p) { return p != nullptr && aligned(p, 4); }

bool counts_ok(const int32_t *counts, int64_t num_pages, const int32_t *status)
{
    return words_ok(counts) && num_pages >= 1 && num_pages <= INT32_MAX &&
           (status == nullptr || aligned(status, 4));
}

// Whether two ranges of bytes share none.
bool apart(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a == nullptr || b == nullptr || x + na <= y || y + nb <= x;
}

// Whether two tables share no entry: their ranges do not meet, or their rows lie in different
// columns of one grid (of the shorter stride, of which the other is a multiple).  A vector is a
// table of one row.
bool tables_apart(const int32_t *a, int64_t lda, int64_t na, int32_t rows_a, const int32_t *b,
                  int64_t ldb, int64_t nb, int32_t rows_b)
{
    if (apart(a, 4 * (size_t)((rows_a - 1) * lda + na), b, 4 * (size_t)((rows_b - 1) * ldb + nb)))
        return true;
    const int64_t step = rows_a == 1 ? (rows_b == 1 ? 0 : ldb)
                         : rows_b == 1 || lda < ldb ? lda : ldb;
    if (step == 0 || (rows_a > 1 && lda % step != 0) || (rows_b > 1 && ldb % step != 0))
        return false;
    int64_t off = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / 4 % step;
    if (off < 0)
        off += step;
    return na <= off && off <= step - nb;
}

plmla_status result(cudaError_t err) { return err == cudaSuccess ? PLMLA_OK : PLMLA_CUDA_ERROR; }

}  // namespace

namespace {

bool shared_ok(int32_t num_reqs, int32_t n_q, int32_t num_heads, int32_t num_groups)
{
    return num_reqs >= 1 && num_reqs <= kMaxReqs && n_q >= 1 && n_q <= kMaxNq &&
           num_heads >= 1 && num_heads <= 128 && num_groups >= 1 && num_groups <= kMaxReqs;
}

struct SharedLayout {
    size_t total, sources, parts, q8, qexp, lse_part, o_part, size;
};

SharedLayout shared_layout(int32_t num_reqs, int32_t rows, int32_t num_groups, bool fp8, int sms)
{
    const size_t slots = (size_t)shared_slots(num_reqs, rows, num_groups, sms);
    const size_t all = (size_t)num_reqs * rows;
    SharedLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes);
        return here;
    };
    l.total = take(sizeof(int64_t));
    l.sources = take(sizeof(SharedSource) * (size_t)num_reqs);
    l.parts = take(sizeof(SharedPart) * ((size_t)num_groups + num_reqs));
    l.q8 = take(fp8 ? 2 * (size_t)kRow * all : 0);
    l.qexp = take(fp8 ? 4 * all : 0);
    l.lse_part = take(4 * 128 * slots);
    l.o_part = take(4 * 128 * (size_t)kLatent * slots);
    l.size = at;
    return l;
}

plmla_status shared_impl(const void *q_nope_absorbed, const void *q_rope, const void *gate,
                         const void *slab_base, bool fp8, int64_t num_pages,
                         int64_t page_stride_elems, float kv_scale, const int32_t *page_table,
                         int64_t page_table_ld, int64_t page_table_cols, const int32_t *seq_lens,
                         int32_t num_reqs, int32_t n_q_per_req, int32_t num_heads,
                         const int32_t *group_starts, const int32_t *shared_lens,
                         int32_t num_groups, float scale, void *out, float *lse, void *workspace,
                         size_t workspace_bytes, int32_t *status, void *stream)
{
    if (!shared_ok(num_reqs, n_q_per_req, num_heads, num_groups) ||
        !table_ok(page_table, page_table_ld, page_table_cols, num_reqs) || num_pages < 1 ||
        num_pages > INT32_MAX || page_stride_elems < (int64_t)kPageTokens * kRow ||
        page_stride_elems % (fp8 ? 16 : 8) != 0 || !(isfinite(scale) && scale > 0.f) ||
        !(isfinite(kv_scale) && kv_scale > 0.f))
        return PLMLA_INVALID_ARGUMENT;
    const void *rows16[] = {q_nope_absorbed, q_rope, gate, slab_base, out};
    for (const void *p : rows16)
        if (p == nullptr || !aligned(p, 16))
            return PLMLA_INVALID_ARGUMENT;
    if (!words_ok(seq_lens) || !words_ok(group_starts) || !words_ok(shared_lens) ||
        (lse != nullptr && !aligned(lse, 4)) || (status != nullptr && !aligned(status, 4)) ||
        workspace == nullptr || !aligned(workspace, kAlign))
        return PLMLA_INVALID_ARGUMENT;
    // a block of the merge reads its part of the gate before it writes the same part of out
    const size_t all_rows = (size_t)num_reqs * n_q_per_req * num_heads;
    if ((out != gate && !apart(out, 2 * kLatent * all_rows, gate, 2 * kLatent * all_rows)) ||
        !apart(lse, 4 * all_rows, out, 2 * kLatent * all_rows) ||
        !apart(lse, 4 * all_rows, gate, 2 * kLatent * all_rows))
        return PLMLA_INVALID_ARGUMENT;
    const int sms = device_sms();
    if (sms < 2)
        return PLMLA_CUDA_ERROR;
    SharedArgs a = {};
    a.rows = n_q_per_req * num_heads;
    const SharedLayout l = shared_layout(num_reqs, a.rows, num_groups, fp8, sms);
    if (workspace_bytes < l.size)
        return PLMLA_WORKSPACE_TOO_SMALL;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    a.q_nope = static_cast<const __nv_bfloat16 *>(q_nope_absorbed);
    a.q_rope = static_cast<const __nv_bfloat16 *>(q_rope);
    a.gate = static_cast<const __nv_bfloat16 *>(gate);
    a.slab = slab_base;
    a.num_pages = num_pages;
    a.page_stride = page_stride_elems;
    a.page_table = page_table;
    a.table_ld = page_table_ld;
    a.table_cols = page_table_cols;
    a.seq_lens = seq_lens;
    a.num_reqs = num_reqs;
    a.n_q = n_q_per_req;
    a.heads = num_heads;
    a.group_starts = group_starts;
    a.shared_lens = shared_lens;
    a.num_groups = num_groups;
    a.scale = scale;
    a.kv_scale = kv_scale;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.total = reinterpret_cast<int64_t *>(w + l.total);
    a.sources = reinterpret_cast<SharedSource *>(w + l.sources);
    a.parts = reinterpret_cast<SharedPart *>(w + l.parts);
    a.lse_part = reinterpret_cast<float *>(w + l.lse_part);
    a.o_part = reinterpret_cast<float *>(w + l.o_part);
    a.status = status;
    if (fp8) {
        a.q8 = w + l.q8;
        a.qexp = reinterpret_cast<int32_t *>(w + l.qexp);
    }
    return result(launch_shared(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" size_t mla_shared_workspace_size(int32_t num_reqs, int32_t n_q_per_req,
                                            int32_t num_heads, int32_t num_groups, int32_t fp8)
{
    const int sms = device_sms();
    if (!shared_ok(num_reqs, n_q_per_req, num_heads, num_groups) || sms < 2)
        return 0;
    return shared_layout(num_reqs, n_q_per_req * num_heads, num_groups, fp8 != 0, sms).size;
}

extern "C" plmla_status mla_decode_shared(
    const void *q_nope_absorbed, const void *q_rope, const void *gate, const void *slab_base,
    int64_t num_pages, int64_t page_stride_elems, const int32_t *page_table, int64_t page_table_ld,
    int64_t page_table_cols, const int32_t *seq_lens, int32_t num_reqs, int32_t n_q_per_req,
    int32_t num_heads, const int32_t *group_starts, const int32_t *shared_lens, int32_t num_groups,
    float scale, void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *status,
    void *stream)
{
    return shared_impl(q_nope_absorbed, q_rope, gate, slab_base, false, num_pages,
                       page_stride_elems, 1.f, page_table, page_table_ld, page_table_cols,
                       seq_lens, num_reqs, n_q_per_req, num_heads, group_starts, shared_lens,
                       num_groups, scale, out, lse, workspace, workspace_bytes, status, stream);
}

extern "C" plmla_status mla_decode_shared_fp8(
    const void *q_nope_absorbed, const void *q_rope, const void *gate, const void *slab_base,
    int64_t num_pages, int64_t page_stride_elems, float kv_scale, const int32_t *page_table,
    int64_t page_table_ld, int64_t page_table_cols, const int32_t *seq_lens, int32_t num_reqs,
    int32_t n_q_per_req, int32_t num_heads, const int32_t *group_starts,
    const int32_t *shared_lens, int32_t num_groups, float scale, void *out, float *lse,
    void *workspace, size_t workspace_bytes, int32_t *status, void *stream)
{
    return shared_impl(q_nope_absorbed, q_rope, gate, slab_base, true, num_pages,
                       page_stride_elems, kv_scale, page_table, page_table_ld, page_table_cols,
                       seq_lens, num_reqs, n_q_per_req, num_heads, group_starts, shared_lens,
                       num_groups, scale, out, lse, workspace, workspace_bytes, status, stream);
}

extern "C" plmla_status mla_pages_fork(const int32_t *page_table, int64_t page_table_ld,
                                       int64_t page_table_cols, const int32_t *seq_lens,
                                       int32_t num_rows, const int32_t *parents, int32_t out_rows,
                                       int32_t *ref_counts, int64_t num_pages, int32_t *out_table,
                                       int64_t out_table_ld, int64_t out_table_cols,
                                       int32_t *out_lens, int32_t *status, void *stream)
{
    if (!table_ok(page_table, page_table_ld, page_table_cols, num_rows) ||
        !table_ok(out_table, out_table_ld, out_table_cols, out_rows) || !words_ok(seq_lens) ||
        !words_ok(parents) || !words_ok(out_lens) || !counts_ok(ref_counts, num_pages, status) ||
        !tables_apart(page_table, page_table_ld, page_table_cols, num_rows, out_table, out_table_ld,
                      out_table_cols, out_rows) ||
        !apart(seq_lens, 4 * (size_t)num_rows, out_lens, 4 * (size_t)out_rows) ||
        !tables_apart(page_table, page_table_ld, page_table_cols, num_rows, out_lens, out_rows,
                      out_rows, 1) ||
        !tables_apart(out_table, out_table_ld, out_table_cols, out_rows, seq_lens, num_rows, num_rows,
                      1) ||
        !tables_apart(out_table, out_table_ld, out_table_cols, out_rows, out_lens, out_rows, out_rows,
                      1))
        return PLMLA_INVALID_ARGUMENT;
    const ForkArgs a = {page_table, page_table_ld, page_table_cols, seq_lens, num_rows,
                        parents,    out_rows,      out_table,       out_table_ld, out_table_cols,
                        out_lens,   ref_counts,    num_pages,       status};
    return result(launch_fork(a, static_cast<cudaStream_t>(stream)));
}

extern "C" plmla_status mla_pages_free(const int32_t *page_table, int64_t page_table_ld,
                                       int64_t page_table_cols, int32_t *seq_lens,
                                       int32_t num_rows, int32_t *ref_counts, int64_t num_pages,
                                       int32_t *status, void *stream)
{
    if (!table_ok(page_table, page_table_ld, page_table_cols, num_rows) || !words_ok(seq_lens) ||
        !counts_ok(ref_counts, num_pages, status))
        return PLMLA_INVALID_ARGUMENT;
    return result(launch_free(page_table, page_table_ld, page_table_cols, seq_lens, num_rows,
                              ref_counts, num_pages, status, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t mla_pages_workspace_size(int32_t num_reqs)
{
    if (num_reqs < 1 || num_reqs > kMaxReqs)
        return 0;
    return kAlign + align_up(sizeof(int4) * (size_t)num_reqs);
}

extern "C" plmla_status mla_pages_reserve_ex(int32_t num_layers, void *const *slab_base,
                                             int32_t elem_bytes, int64_t num_pages,
                                             int64_t page_stride_elems, int32_t *page_table,
                                             int64_t page_table_ld, int64_t page_table_cols,
                                             const int32_t *seq_lens, int32_t num_reqs,
                                             int32_t n_new, const int32_t *n_new_of,
                                             int32_t *granted, int32_t *ref_counts, void *workspace,
                                             size_t workspace_bytes, int32_t *status, void *stream)
{
    if (num_layers < 1 || num_layers > kMaxLayers || slab_base == nullptr ||
        (elem_bytes != 1 && elem_bytes != 2) ||
        page_stride_elems < (int64_t)kPageTokens * kRow ||
        page_stride_elems % (elem_bytes == 1 ? 16 : 8) != 0 ||
        !table_ok(page_table, page_table_ld, page_table_cols, num_reqs) || !words_ok(seq_lens) ||
        (n_new_of == nullptr ? n_new < 0 : !aligned(n_new_of, 4)) ||
        (granted != nullptr &&
         (!aligned(granted, 4) || !apart(granted, 4 * (size_t)num_reqs, seq_lens, 4 * (size_t)num_reqs) ||
          (granted != n_new_of &&
           !apart(granted, 4 * (size_t)num_reqs, n_new_of, 4 * (size_t)num_reqs)) ||
          !tables_apart(page_table, page_table_ld, page_table_cols, num_reqs, granted, num_reqs,
                        num_reqs, 1))) ||
        !counts_ok(ref_counts, num_pages, status) ||
        !apart(granted, 4 * (size_t)num_reqs, ref_counts, 4 * (size_t)num_pages) ||
        !apart(granted, 4 * (size_t)num_reqs, status, 4) || workspace == nullptr ||
        !aligned(workspace, kAlign))
        return PLMLA_INVALID_ARGUMENT;
    for (int32_t l = 0; l < num_layers; ++l)
        if (slab_base[l] == nullptr || !aligned(slab_base[l], 16))
            return PLMLA_INVALID_ARGUMENT;
    if (workspace_bytes < mla_pages_workspace_size(num_reqs))
        return PLMLA_WORKSPACE_TOO_SMALL;
    const int sms = device_sms();
    if (sms <= 0)
        return PLMLA_CUDA_ERROR;
    ReserveArgs a = {};
    a.table = page_table;
    a.ld = page_table_ld;
    a.cols = page_table_cols;
    a.lens = seq_lens;
    a.num_reqs = num_reqs;
    a.n_new = n_new;
    a.n_new_of = n_new_of;
    a.counts = ref_counts;
    a.num_pages = num_pages;
    a.num_jobs = static_cast<int32_t *>(workspace);
    a.jobs = reinterpret_cast<int4 *>(static_cast<unsigned char *>(workspace) + kAlign);
    a.granted = granted;
    a.status = status;
    return result(launch_reserve(a, num_layers, slab_base, elem_bytes == 1,
                                 page_stride_elems * elem_bytes, sms,
                                 static_cast<cudaStream_t>(stream)));
}

extern "C" plmla_status mla_pages_reserve(int32_t num_layers, void *const *slab_base,
                                          int32_t elem_bytes, int64_t num_pages,
                                          int64_t page_stride_elems, int32_t *page_table,
                                          int64_t page_table_ld, int64_t page_table_cols,
                                          const int32_t *seq_lens, int32_t num_reqs, int32_t n_new,
                                          const int32_t *n_new_of, int32_t *ref_counts,
                                          void *workspace, size_t workspace_bytes, int32_t *status,
                                          void *stream)
{
    return mla_pages_reserve_ex(num_layers, slab_base, elem_bytes, num_pages, page_stride_elems,
                                page_table, page_table_ld, page_table_cols, seq_lens, num_reqs,
                                n_new, n_new_of, nullptr, ref_counts, workspace, workspace_bytes,
                                status, stream);
}

namespace {

bool beams_ok(int32_t batch, int32_t beams, int32_t vocab)
{
    return batch >= 1 && beams >= 1 && beams <= kMaxBeams && vocab >= 1 &&
           (int64_t)batch * beams <= kMaxBeamRows && (int64_t)beams * vocab <= INT32_MAX;
}

}  // namespace

extern "C" size_t mla_beam_workspace_size(int32_t batch, int32_t beams, int32_t vocab)
{
    return beams_ok(batch, beams, vocab) ? beam_workspace(batch, beams, vocab) : 0;
}

extern "C" plmla_status mla_beam_select(const void *logits, int64_t logits_ld, int32_t dtype,
                                        const float *scores, const uint8_t *ended,
                                        int32_t end_token, int32_t batch, int32_t beams,
                                        int32_t vocab, int32_t *tokens, int32_t *parents,
                                        float *out_scores, void *workspace, size_t workspace_bytes,
                                        void *stream)
{
    if (!beams_ok(batch, beams, vocab) || logits_ld < vocab ||
        (dtype != PLMLA_BF16 && dtype != PLMLA_FP16 && dtype != PLMLA_FP32) ||
        logits == nullptr || !aligned(logits, dtype == PLMLA_FP32 ? 4 : 2) || scores == nullptr ||
        !aligned(scores, 4) || (ended != nullptr && (end_token < 0 || end_token >= vocab)) ||
        !words_ok(tokens) || !words_ok(parents) || out_scores == nullptr ||
        !aligned(out_scores, 4) || workspace == nullptr || !aligned(workspace, kAlign))
        return PLMLA_INVALID_ARGUMENT;
    const size_t words = 4 * (size_t)batch * beams;
    const void *outs[] = {tokens, parents, out_scores};
    for (int i = 0; i < 3; ++i)
        if (!apart(outs[i], words, outs[(i + 1) % 3], words) || !apart(outs[i], words, scores, words) ||
            !apart(outs[i], words, ended, words / 4))
            return PLMLA_INVALID_ARGUMENT;
    if (workspace_bytes < beam_workspace(batch, beams, vocab))
        return PLMLA_WORKSPACE_TOO_SMALL;
    const BeamArgs a = {logits, logits_ld, dtype, scores, ended, end_token, batch,
                        beams,  vocab,     tokens, parents, out_scores};
    return result(launch_beams(a, workspace, static_cast<cudaStream_t>(stream)));
}
