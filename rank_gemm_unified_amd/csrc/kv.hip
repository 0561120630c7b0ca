// The KV-cache calls: argument checks and dispatch (kernels in k_kv_*.hip).
#include <algorithm>

#include "kv.h"

using namespace lorapool;

namespace {

bool aligned(const void *ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

bool layout_ok(const lora_pool *p, const lora_kv_layout_t *l) {
    return l && l->n_heads >= 1 && l->n_heads <= LORA_MAX_HEADS && l->n_kv_heads >= 1 && l->n_heads % l->n_kv_heads == 0 &&
           (l->head_dim == 64 || l->head_dim == 128 || l->head_dim == 256) && l->tokens_per_page >= 1 &&
           l->tokens_per_page <= LORA_MAX_TOKENS_PER_PAGE &&
           (int64_t)l->n_kv_heads * l->head_dim * l->tokens_per_page <= p->hidden;
}

int check_layout(const lora_pool *p, const char *fn, const lora_kv_layout_t *l) {
    if (!l) return set_error(LORA_EINVAL, "%s: layout is NULL", fn);
    if (!layout_ok(p, l))
        return set_error(LORA_EINVAL, "%s: layout (%d heads, %d K/V heads, head_dim %d, %d tokens a page) does not fit "
                                      "pages of %d elements (at most %d heads, K/V heads divide them; head_dim 64, 128 or "
                                      "256; n_kv_heads * head_dim * tokens_per_page <= hidden)",
                         fn, l->n_heads, l->n_kv_heads, l->head_dim, l->tokens_per_page, p->hidden, LORA_MAX_HEADS);
    return LORA_OK;
}

struct Span {
    const char *at;
    size_t bytes;
    bool meets(const Span &o) const { return at && o.at && at < o.at + o.bytes && o.at < at + bytes; }
};
Span rows_span(const void *p, int64_t rows, int64_t ld, int64_t width, int64_t elem) {
    return {(const char *)p, rows > 0 ? (size_t)(((rows - 1) * ld + width) * elem) : 0};
}
Span pages_span(const lora_pool *p) {
    return {(const char *)p->pages, (size_t)p->num_pages * p->hidden * p->elem};
}

// Checks shared by the calls over rows of new tokens, and their KvArgs.  T >= 1 and n_seq >= 1.
int common(lora_pool *p, const char *fn, const lora_kv_layout_t *l, const int32_t *table, int32_t max_pages,
           const int32_t *q_start, const int32_t *lens, int32_t n_seq, int64_t T, int64_t max_len, KvArgs *a) {
    const int64_t cap = (int64_t)max_pages * l->tokens_per_page;
    if (max_pages < 1 || cap > LORA_MAX_KV_TOKENS)
        return set_error(LORA_EINVAL, "%s: max_pages %d: %lld tokens not in [1, %d]", fn, max_pages, (long long)cap,
                         LORA_MAX_KV_TOKENS);
    if (max_len < 1 || max_len > cap)
        return set_error(LORA_EINVAL, "%s: max_len %lld not in [1, %lld]", fn, (long long)max_len, (long long)cap);
    if (n_seq * max_len > (int64_t(1) << 34))
        return set_error(LORA_EINVAL, "%s: %d sequences of up to %lld tokens: more than 2^34", fn, n_seq, (long long)max_len);
    if (!table || !lens) return set_error(LORA_EINVAL, "%s: NULL pointer argument", fn);
    if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(q_start, 4))
        return set_error(LORA_EINVAL, "%s: misaligned pointer (table, q_start, lens: 4 B)", fn);
    // kernels address token rows in 32-bit units of 128 bytes
    if ((int64_t)p->num_pages * p->hidden * p->elem > (int64_t(1) << 39))
        return set_error(LORA_EINVAL, "%s: pool of more than 512 GiB", fn);
    a->pages = (char *)p->pages;
    a->num_pages = p->num_pages;
    a->page_bytes = (int64_t)p->hidden * p->elem;
    a->table = table;
    a->q_start = q_start;
    a->lens = lens;
    a->err = p->dev_err;
    a->max_pages = max_pages;
    a->n_seq = n_seq;
    a->T = (int32_t)T;
    a->cap = (int32_t)max_len;
    a->n_heads = l->n_heads;
    a->n_kv = l->n_kv_heads;
    a->head_dim = l->head_dim;
    a->group = l->n_heads / l->n_kv_heads;
    a->tpp = l->tokens_per_page;
    a->tpp_magic = a->tpp == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + a->tpp - 1) / a->tpp);
    a->tok_bytes = l->n_kv_heads * l->head_dim * p->elem;
    return LORA_OK;
}

// pool, sizes and layout: LORA_OK, an error, or 1 where there is nothing to do
int begin(lora_pool *p, const char *fn, const lora_kv_layout_t *l, int32_t n_seq, int64_t T) {
    if (!p) return set_error(LORA_EINVAL, "%s: pool is NULL", fn);
    if (int rc = check_layout(p, fn, l)) return rc;
    if (n_seq < 0 || n_seq > LORA_MAX_SEQS)
        return set_error(LORA_EINVAL, "%s: n_seq %d not in [0, %d]", fn, n_seq, LORA_MAX_SEQS);
    if (T < 0 || T > LORA_MAX_TOKENS)
        return set_error(LORA_EINVAL, "%s: T = %lld not in [0, %d]", fn, (long long)T, LORA_MAX_TOKENS);
    return n_seq == 0 || T == 0 ? 1 : LORA_OK;
}

int check_rows(const lora_pool *p, const char *fn, const char *what, const void *ptr, int64_t ld, int64_t width,
               bool one) {
    if (!ptr) return set_error(LORA_EINVAL, "%s: %s is NULL", fn, what);
    const int64_t step = 16 / p->elem;
    if (!aligned(ptr, 16) || (!one && (ld % step || ld < width)) || ld > (int64_t(1) << 31))
        return set_error(LORA_EINVAL, "%s: %s: rows of %lld elements, %lld apart: every row starts on 16 bytes and none "
                                      "overlaps the next", fn, what, (long long)width, (long long)ld);
    return LORA_OK;
}

int attend(lora_pool *p, const char *fn, const lora_kv_layout_t *l, const void *q, int64_t ldq, const int32_t *table,
           int32_t max_pages, const int32_t *q_start, const int32_t *lens, int32_t n_seq, int64_t T, int64_t max_len,
           float scale, void *out, int64_t ldo, const float *prior, float *scores, void *ws, size_t ws_bytes,
           void *stream, bool chunk) {
    const int rc0 = begin(p, fn, l, n_seq, T);
    if (rc0) return rc0 < 0 ? rc0 : LORA_OK;
    KvArgs a{};
    if (int rc = common(p, fn, l, table, max_pages, q_start, lens, n_seq, T, max_len, &a)) return rc;
    const int64_t width = (int64_t)l->n_heads * l->head_dim;
    if (int rc = check_rows(p, fn, "q", q, ldq, width, T == 1)) return rc;
    if (int rc = check_rows(p, fn, "out", out, ldo, width, T == 1)) return rc;
    if (!(scale == scale) || scale - scale != 0.f) return set_error(LORA_EINVAL, "%s: scale is not finite", fn);
    if (chunk && !q_start) return set_error(LORA_EINVAL, "%s: q_start is NULL", fn);
    if (prior && !scores) return set_error(LORA_EINVAL, "%s: prior without scores", fn);
    if (!aligned(scores, 4) || !aligned(prior, 4)) return set_error(LORA_EINVAL, "%s: misaligned scores", fn);
    const Span qs = rows_span(q, T, ldq, width, p->elem), os = rows_span(out, T, ldo, width, p->elem);
    if (os.meets(qs) || os.meets(pages_span(p))) return set_error(LORA_EINVAL, "%s: out overlaps q or the pages", fn);
    const int64_t score_ld = (int64_t)max_pages * l->tokens_per_page;
    const size_t need = chunk ? kv_chunk_ws_bytes(p->dtype, *l, n_seq, T, max_len, scores != nullptr)
                              : kv_attend_ws_need(p->dtype, *l, n_seq, max_len, scores != nullptr);
    if (need > 0 && (!ws || !aligned(ws, 256) || ws_bytes < need))
        return set_error(LORA_EINVAL, "%s: workspace %zu bytes at %p: %zu needed, 256-byte aligned", fn, ws_bytes, ws, need);
    // nothing that is written may overlap anything else, but for scores that are their own prior
    const size_t table_bytes = (size_t)n_seq * 2 * max_pages * 4, score_bytes = (size_t)n_seq * score_ld * 4;
    const Span written[] = {os, {(const char *)scores, score_bytes}, {(const char *)(need ? ws : nullptr), need}};
    const Span read[] = {qs, pages_span(p), {(const char *)table, table_bytes}, {(const char *)lens, (size_t)n_seq * 4},
                         {(const char *)q_start, ((size_t)n_seq + 1) * 4},
                         {(const char *)(prior == scores ? nullptr : prior), score_bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const Span &r : read)
            if (written[i].meets(r)) return set_error(LORA_EINVAL, "%s: out, scores or the workspace overlaps another argument", fn);
        for (int j = 0; j < i; ++j)
            if (written[i].meets(written[j])) return set_error(LORA_EINVAL, "%s: out, scores and the workspace overlap", fn);
    }
    if (p->bookkeeping_only) return set_error(LORA_EINVAL, "%s: bookkeeping-only pool", fn);
    DeviceGuard g(p->device);
    if (!g.ok) return set_error(LORA_EHIP, "%s: cannot select the pool's device", fn);
    const KvAttend at{q, out, ldq, ldo, scale, prior, scores, score_ld, ws};
    const hipError_t e = chunk ? launch_kv_chunk(p->dtype, a, at, (hipStream_t)stream)
                               : launch_kv_attend(p->dtype, a, at, (hipStream_t)stream);
    return e == hipSuccess ? LORA_OK : hip_error(e, fn);
}

}  // namespace

extern "C" int lora_kv_write(lora_pool *p, const lora_kv_layout_t *l, const void *k, int64_t ldk, const void *v,
                             int64_t ldv, const int32_t *table, int32_t max_pages, const int32_t *q_start,
                             const int32_t *lens, int32_t n_seq, int64_t T, void *stream) {
    const char *fn = "lora_kv_write";
    const int rc0 = begin(p, fn, l, n_seq, T);
    if (rc0) return rc0 < 0 ? rc0 : LORA_OK;
    KvArgs a{};
    if (int rc = common(p, fn, l, table, max_pages, q_start, lens, n_seq, T,
                        (int64_t)max_pages * l->tokens_per_page, &a)) return rc;
    if (!q_start && T != n_seq)
        return set_error(LORA_EINVAL, "%s: T = %lld rows for %d sequences without q_start", fn, (long long)T, n_seq);
    const int64_t width = (int64_t)l->n_kv_heads * l->head_dim;
    if (int rc = check_rows(p, fn, "k", k, ldk, width, T == 1)) return rc;
    if (int rc = check_rows(p, fn, "v", v, ldv, width, T == 1)) return rc;
    if (rows_span(k, T, ldk, width, p->elem).meets(pages_span(p)) || rows_span(v, T, ldv, width, p->elem).meets(pages_span(p)))
        return set_error(LORA_EINVAL, "%s: k or v lies in the pool's pages", fn);
    if (p->bookkeeping_only) return set_error(LORA_EINVAL, "%s: bookkeeping-only pool", fn);
    DeviceGuard g(p->device);
    if (!g.ok) return set_error(LORA_EHIP, "%s: cannot select the pool's device", fn);
    const hipError_t e = launch_kv_write(p->dtype, a, k, ldk, v, ldv, (hipStream_t)stream);
    return e == hipSuccess ? LORA_OK : hip_error(e, fn);
}

static bool sizes_ok(const lora_pool *p, const lora_kv_layout_t *l, int32_t n_seq, int64_t T, int64_t max_len) {
    return p && layout_ok(p, l) && n_seq >= 1 && n_seq <= LORA_MAX_SEQS && T >= 1 && T <= LORA_MAX_TOKENS &&
           max_len >= 1 && max_len <= LORA_MAX_KV_TOKENS && n_seq * max_len <= (int64_t(1) << 34);
}

extern "C" size_t lora_kv_attend_workspace_size(const lora_pool *p, const lora_kv_layout_t *l, int32_t n_seq,
                                                int64_t max_len, int32_t with_scores) {
    if (!sizes_ok(p, l, n_seq, 1, max_len)) return 0;
    return kv_attend_ws_bytes(p->dtype, *l, n_seq, max_len, with_scores != 0);
}

extern "C" size_t lora_kv_attend_chunk_workspace_size(const lora_pool *p, const lora_kv_layout_t *l, int32_t n_seq,
                                                      int64_t T, int64_t max_len, int32_t with_scores) {
    if (!sizes_ok(p, l, n_seq, T, max_len)) return 0;
    return kv_chunk_ws_bytes(p->dtype, *l, n_seq, T, max_len, with_scores != 0);
}

extern "C" int lora_kv_attend(lora_pool *p, const lora_kv_layout_t *l, const void *q, int64_t ldq,
                              const int32_t *table, int32_t max_pages, const int32_t *lens, int32_t n_seq,
                              int64_t max_len, float scale, void *out, int64_t ldo, const float *prior, float *scores,
                              void *ws, size_t ws_bytes, void *stream) {
    return attend(p, "lora_kv_attend", l, q, ldq, table, max_pages, nullptr, lens, n_seq, n_seq, max_len, scale, out,
                  ldo, prior, scores, ws, ws_bytes, stream, false);
}

extern "C" int lora_kv_attend_chunk(lora_pool *p, const lora_kv_layout_t *l, const void *q, int64_t ldq,
                                    const int32_t *table, int32_t max_pages, const int32_t *q_start,
                                    const int32_t *lens, int32_t n_seq, int64_t T, int64_t max_len, float scale,
                                    void *out, int64_t ldo, const float *prior, float *scores, void *ws,
                                    size_t ws_bytes, void *stream) {
    return attend(p, "lora_kv_attend_chunk", l, q, ldq, table, max_pages, q_start, lens, n_seq, T, max_len, scale, out,
                  ldo, prior, scores, ws, ws_bytes, stream, true);
}

extern "C" int lora_kv_evict(lora_pool *p, const lora_kv_layout_t *l, int32_t layers, int32_t n_seq,
                             const int32_t *table, int32_t *table_out, int32_t max_pages, const float *scores,
                             float *scores_out, const int32_t *lens, int32_t *lens_out, int32_t budget,
                             int32_t keep_first, int32_t keep_last, int32_t *dropped, int32_t max_drop,
                             int32_t *n_dropped, void *stream) {
    const char *fn = "lora_kv_evict";
    if (layers < 1 || layers > 65535) return set_error(LORA_EINVAL, "%s: layers %d not in [1, 65535]", fn, layers);
    const int rc0 = begin(p, fn, l, n_seq, 1);
    if (rc0) return rc0 < 0 ? rc0 : LORA_OK;
    const int64_t cap = (int64_t)max_pages * l->tokens_per_page;
    if (max_pages < 1 || cap > LORA_MAX_KV_TOKENS)
        return set_error(LORA_EINVAL, "%s: max_pages %d: %lld tokens not in [1, %d]", fn, max_pages, (long long)cap,
                         LORA_MAX_KV_TOKENS);
    if (budget < 0 || keep_first < 0 || keep_last < 0 || max_drop < 1 || max_drop > max_pages ||
        keep_first > LORA_MAX_KV_TOKENS || keep_last > LORA_MAX_KV_TOKENS)
        return set_error(LORA_EINVAL, "%s: budget %d, keep_first %d, keep_last %d (each >= 0, the last two <= %d), "
                                      "max_drop %d not in [1, %d]",
                         fn, budget, keep_first, keep_last, LORA_MAX_KV_TOKENS, max_drop, max_pages);
    const void *ptrs[] = {table, table_out, scores, scores_out, lens, lens_out, dropped, n_dropped};
    for (const void *q : ptrs) {
        if (!q) return set_error(LORA_EINVAL, "%s: NULL pointer argument", fn);
        if (!aligned(q, 4)) return set_error(LORA_EINVAL, "%s: misaligned pointer (4 B)", fn);
    }
    // nothing that is written may overlap anything else, but for the two pairs that may be one buffer
    const size_t rows = (size_t)layers * n_seq, tb = rows * 2 * max_pages * 4, sb = rows * (size_t)cap * 4,
                 db = rows * 2 * max_drop * 4, nb = (size_t)n_seq * 4;
    const Span sp[] = {{(const char *)table, tb}, {(const char *)table_out, tb}, {(const char *)scores, sb},
                       {(const char *)scores_out, sb}, {(const char *)lens, nb}, {(const char *)lens_out, nb},
                       {(const char *)dropped, db}, {(const char *)n_dropped, nb}};
    const bool written[] = {false, true, false, true, false, true, true, true};
    for (int i = 0; i < 8; ++i)
        for (int j = 0; j < i; ++j) {
            if (!written[i] && !written[j]) continue;
            if ((j == 0 && i == 1 && table == table_out) || (j == 2 && i == 3 && scores == scores_out)) continue;
            if (sp[i].meets(sp[j])) return set_error(LORA_EINVAL, "%s: an output overlaps another argument", fn);
        }
    if (p->bookkeeping_only) return set_error(LORA_EINVAL, "%s: bookkeeping-only pool", fn);
    DeviceGuard g(p->device);
    if (!g.ok) return set_error(LORA_EHIP, "%s: cannot select the pool's device", fn);
    const KvEvict e{layers, n_seq, max_pages, l->tokens_per_page, table, table_out, scores, scores_out, lens, lens_out,
                    budget, keep_first, keep_last, max_drop, dropped, n_dropped, p->dev_err};
    const hipError_t err = launch_kv_evict(e, (hipStream_t)stream);
    return err == hipSuccess ? LORA_OK : hip_error(err, fn);
}
