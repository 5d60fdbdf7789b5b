// C ABI of what a serving step does around the cache (declared in include/lora.h): norms and
// rotation of heads, page tables, copies of pages, choice of pages and attention over them.
// No call reads device memory on the host or allocates.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/lora.h"
#include "ctx.h"
#include "kv.h"
#include "kv_handle.h"

using namespace lora;

namespace {

// Vectors of a row, so that a CTA's items can be numbered and divided in 32 bits.
constexpr int64_t kMaxRowVectors = 16384;
// Cells times heads of a page that is copied: its parts are numbered in 32 bits.
constexpr int64_t kMaxCopyVectors = 1 << 24;

int take_rope(const lora_rope *r, RopeParams &p)
{
    if (!r || r->head_dim < 1 || r->rot_dim < 0 || r->rot_dim > r->head_dim || !(r->eps >= 0.f) ||
        !(r->eps - r->eps == 0.f) || (r->q_weight && !aligned(r->q_weight, 16)) ||
        (r->k_weight && !aligned(r->k_weight, 16)) || (r->rot_dim > 0 && !aligned(r->freqs, 4)))
        return LORA_E_INVAL;
    if (r->head_dim % 8 || r->head_dim > 256 || r->rot_dim % 16)
        return LORA_E_UNSUPPORTED;
    p.dim = r->head_dim;
    p.half = r->rot_dim / 2;
    p.interleaved = r->interleaved != 0;
    p.q_weight = r->q_weight;
    p.k_weight = r->k_weight;
    p.freqs = r->freqs;
    p.eps = r->eps;
    return LORA_OK;
}

int rope_call(lora_ctx *ctx, const lora_kv *kv, const lora_rope *rope, const lora_kv_batch *b, int64_t n,
              const void *q, int64_t ldq, int q_heads, void *q_out, int64_t ldqo, const void *k, int64_t ldk,
              int k_heads, void *k_out, int64_t ldko, const void *v, int64_t ldv, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (!ctx || (kv && kv->ctx != ctx) || q_heads < 0 || k_heads < 0)
        return LORA_E_INVAL;
    RopeParams p{};
    int rc = take_rope(rope, p);
    if (rc == LORA_OK)
        rc = take_batch(kv, b, n, p.b);
    if (rc != LORA_OK)
        return rc;
    if (kv && kv->view.dim != p.dim)
        return LORA_E_INVAL;
    const int64_t qw = int64_t(q_heads) * p.dim, kw = int64_t(k_heads) * p.dim;
    if (n > 0) {
        if (q_heads && (!rows_ok(q, ldq, qw) || !rows_ok(q_out, ldqo, qw)))
            return LORA_E_INVAL;
        if (k_heads && (!rows_ok(k, ldk, kw) || (kv ? !rows_ok(v, ldv, kw) : !rows_ok(k_out, ldko, kw))))
            return LORA_E_INVAL;
    }
    if (int64_t(q_heads) + 2 * int64_t(k_heads) > kMaxRowVectors)
        return LORA_E_CAPACITY;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0 || b->n_seqs == 0 || q_heads + k_heads == 0)
        return rc;
    if (kv)
        p.kv = kv->view;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldqo = ldqo;
    p.ldko = ldko;
    p.q_heads = q_heads;
    p.k_heads = k_heads;
    p.status = ctx_status(ctx);
    const cudaError_t e = launch_rope(p, kv != nullptr, ctx_sms(ctx), stream);
    if (e != cudaSuccess)
        return ctx_cuda_fail(ctx, e);
    ctx_launched(ctx, stream, 256);
    return LORA_OK;
}

int take_table(const lora_ctx *ctx, const lora_page_table *t, TableView &v)
{
    if (!ctx || !t || t->n_seqs < 0 || t->n_cols < 0 || t->ld_pages < t->n_cols || t->n_pages < 1 || t->page_size < 1 ||
        !aligned(t->refs, 4) || (t->n_seqs > 0 && (!aligned(t->lens, 4) || (t->n_cols > 0 && !aligned(t->pages, 4)))))
        return LORA_E_INVAL;
    if (t->n_seqs > kMaxTableSeqs || t->n_pages > kMaxPosition || t->page_size > (1 << 20))
        return LORA_E_CAPACITY;
    v.lens = t->lens;
    v.pages = t->pages;
    v.refs = t->refs;
    v.ld_pages = t->ld_pages;
    v.n_seqs = int(t->n_seqs);
    v.n_cols = int(std::min(t->n_cols, kMaxPosition));
    v.n_pages = int(t->n_pages);
    v.page_size = t->page_size;
    v.capacity = int(t->n_cols > kMaxPosition / t->page_size ? kMaxPosition : t->n_cols * t->page_size);
    v.status = ctx_status(ctx);
    return LORA_OK;
}

// A list of sequences.
int list_ok(const int32_t *list, int64_t n)
{
    return n < 0 || (n > 0 && !aligned(list, 4)) ? LORA_E_INVAL : n > kMaxTableSeqs ? LORA_E_CAPACITY : LORA_OK;
}

int done(lora_ctx *ctx, cudaStream_t stream, cudaError_t e, int path)
{
    if (e != cudaSuccess)
        return ctx_cuda_fail(ctx, e);
    ctx_launched(ctx, stream, path);
    return LORA_OK;
}

// The heads of a selection's call.
int take_selection(const lora_ctx *ctx, const lora_kv *kv, const lora_block_sel *sel, int64_t n, int n_heads)
{
    if (!ctx || !kv || kv->ctx != ctx || !sel || n < 0 || sel->n_rows < n || sel->blocks < 1 || n_heads < 1 ||
        n_heads % kv->view.heads || (n > 0 && (!aligned(sel->lens, 4) || !aligned(sel->pages, 4))))
        return LORA_E_INVAL;
    if (int64_t(sel->blocks) * kv->view.page_size > kMaxPosition || n >= (int64_t(1) << 28) || n * n_heads >= (int64_t(1) << 28))
        return LORA_E_CAPACITY;
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_head_rope(lora_ctx *ctx, const lora_rope *rope, const lora_kv_batch *b, int64_t n, const void *q,
                   int64_t ldq, int q_heads, void *q_out, int64_t ldqo, const void *k, int64_t ldk, int k_heads,
                   void *k_out, int64_t ldko, void *stream)
{
    return rope_call(ctx, nullptr, rope, b, n, q, ldq, q_heads, q_out, ldqo, k, ldk, k_heads, k_out, ldko, nullptr, 0, stream);
}

int lora_kv_write_rope(lora_ctx *ctx, const lora_kv *kv, const lora_rope *rope, const lora_kv_batch *b, int64_t n,
                       const void *q, int64_t ldq, int q_heads, void *q_out, int64_t ldqo, const void *k, int64_t ldk,
                       const void *v, int64_t ldv, void *stream)
{
    if (!kv)
        return LORA_E_INVAL;
    return rope_call(ctx, kv, rope, b, n, q, ldq, q_heads, q_out, ldqo, k, ldk, kv->view.heads, nullptr, 0, v, ldv, stream);
}

int lora_pages_extend(lora_ctx *ctx, const lora_page_table *t, const int32_t *grow, int32_t *got, int32_t *src,
                      int32_t *dst, int32_t *cells, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    TableView v{};
    int rc = take_table(ctx, t, v);
    if (rc != LORA_OK)
        return rc;
    if (v.n_seqs && (!aligned(grow, 4) || !aligned(got, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(cells, 4)))
        return LORA_E_INVAL;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || v.n_seqs == 0)
        return rc;
    return done(ctx, stream, launch_pages_extend(v, grow, got, src, dst, cells, stream), 512);
}

int lora_pages_fork(lora_ctx *ctx, const lora_page_table *t, const int32_t *from, const int32_t *to, int64_t n,
                    void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    TableView v{};
    int rc = take_table(ctx, t, v);
    if (rc == LORA_OK)
        rc = list_ok(from, n);
    if (rc == LORA_OK)
        rc = list_ok(to, n);
    if (rc == LORA_OK)
        rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0)
        return rc;
    return done(ctx, stream, launch_pages_fork(v, from, to, int(n), stream), 512);
}

int lora_pages_free(lora_ctx *ctx, const lora_page_table *t, const int32_t *seqs, const int32_t *keep, int64_t n,
                    void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    TableView v{};
    int rc = take_table(ctx, t, v);
    if (rc == LORA_OK)
        rc = list_ok(seqs, n);
    if (rc == LORA_OK && keep && !aligned(keep, 4))
        rc = LORA_E_INVAL;
    if (rc == LORA_OK)
        rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0)
        return rc;
    return done(ctx, stream, launch_pages_free(v, seqs, keep, int(n), stream), 512);
}

int lora_pages_compact(lora_ctx *ctx, const lora_page_table *t, int32_t *src, int32_t *dst, int64_t n, int32_t *top,
                       void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    TableView v{};
    int rc = take_table(ctx, t, v);
    if (rc != LORA_OK)
        return rc;
    if (n < 0 || (n > 0 && (!aligned(src, 4) || !aligned(dst, 4))) || (top && !aligned(top, 4)))
        return LORA_E_INVAL;
    if (n > kMaxPosition)
        return LORA_E_CAPACITY;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK)
        return rc;
    int launches = 0;
    const cudaError_t e = launch_pages_compact(v, src, dst, int(n), top, &launches, stream);
    for (int i = 0; i < launches; ++i)
        ctx_launched(ctx, stream, 512);
    return e == cudaSuccess ? LORA_OK : ctx_cuda_fail(ctx, e);
}

int lora_kv_copy(lora_ctx *ctx, const lora_kv *const *kvs, int n_kv, const int32_t *src, const int32_t *dst,
                 const int32_t *cells, int64_t n, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (!ctx || !kvs || n_kv < 1 || n < 0 || (n > 0 && (!aligned(src, 4) || !aligned(dst, 4))) || (cells && !aligned(cells, 4)))
        return LORA_E_INVAL;
    for (int i = 0; i < n_kv; ++i) {
        if (!kvs[i] || kvs[i]->ctx != ctx)
            return LORA_E_INVAL;
        const KvView &a = kvs[i]->view, &b = kvs[0]->view;
        if (a.page_size != b.page_size || a.heads != b.heads || a.dim != b.dim || a.format != b.format)
            return LORA_E_INVAL;
    }
    if (int64_t(kvs[0]->view.page_size) * kvs[0]->view.heads > kMaxCopyVectors || n > kMaxPosition)
        return LORA_E_CAPACITY;
    const int rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0)
        return rc;
    KvView views[kMaxCopyCaches];
    for (int at = 0; at < n_kv; at += kMaxCopyCaches) {
        const int some = std::min(n_kv - at, kMaxCopyCaches);
        for (int i = 0; i < some; ++i)
            views[i] = kvs[at + i]->view;
        const cudaError_t e = launch_kv_copy(views, some, KvCopyLists{src, dst, cells, int(n)}, ctx_status(ctx), ctx_sms(ctx), stream);
        if (e != cudaSuccess)
            return ctx_cuda_fail(ctx, e);
        ctx_launched(ctx, stream, 1024);
    }
    return LORA_OK;
}

int lora_kv_attach_bounds(lora_kv *kv, void *codes, float *unit)
{
    if (!kv || !codes != !unit || (codes && (!aligned(codes, 32) || !aligned(unit, 4))))
        return LORA_E_INVAL;
    kv->view.bounds = static_cast<int8_t *>(codes);
    kv->view.unit = unit;
    return LORA_OK;
}

int lora_kv_bounds(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (!ctx || !kv || kv->ctx != ctx || !kv->view.bounds)
        return LORA_E_INVAL;
    BoundsParams p{};
    p.kv = kv->view;
    int rc = take_batch(kv, b, n, p.b);
    if (rc == LORA_OK)
        rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0 || b->n_seqs == 0)
        return rc;
    p.status = ctx_status(ctx);
    return done(ctx, stream, launch_kv_bounds(p, ctx_sms(ctx), stream), 2048);
}

int lora_block_select(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, const void *q, int64_t ldq,
                      int n_heads, int first, int last, const lora_block_sel *sel, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    int rc = take_selection(ctx, kv, sel, n, n_heads);
    if (rc != LORA_OK)
        return rc;
    if (!kv->view.bounds || first < 0 || last < 1 || first > sel->blocks - last)
        return LORA_E_INVAL;
    SelectParams p{};
    p.kv = kv->view;
    rc = take_batch(kv, b, n, p.b);
    if (rc != LORA_OK)
        return rc;
    if (n > 0 && !rows_ok(q, ldq, int64_t(n_heads) * p.kv.dim))
        return LORA_E_INVAL;
    if (b->n_cols > kMaxSelectCols || n_heads / p.kv.heads > kMaxSelectGroup)
        return LORA_E_CAPACITY;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0)
        return rc;                             // without sequences too every row gets its length of -1
    p.n_cols = int(b->n_cols);
    p.q = static_cast<const uint16_t *>(q);
    p.ldq = ldq;
    p.group = n_heads / p.kv.heads;
    p.blocks = sel->blocks;
    p.first = first;
    p.last = last;
    p.lens = sel->lens;
    p.pages = sel->pages;
    p.status = ctx_status(ctx);
    return done(ctx, stream, launch_block_select(p, ctx_sms(ctx), stream), 2048);
}

int lora_block_attention(lora_ctx *ctx, const lora_kv *kv, const lora_block_sel *sel, int64_t n, const void *q,
                         int64_t ldq, int n_heads, float scale, void *out, int64_t ldo, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    int rc = take_selection(ctx, kv, sel, n, n_heads);
    if (rc != LORA_OK)
        return rc;
    const int64_t width = int64_t(n_heads) * kv->view.dim;
    if (!(scale - scale == 0.f) || (n > 0 && (!rows_ok(q, ldq, width) || !rows_ok(out, ldo, width))))
        return LORA_E_INVAL;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0)
        return rc;
    // each row a sequence of the tokens in its pages, with a list for each key head
    AttnParams p{};
    p.kv = kv->view;
    p.b.lens = sel->lens;
    p.b.pages = sel->pages;
    p.b.head_pages = sel->blocks;
    p.b.ld_pages = int64_t(sel->blocks) * p.kv.heads;
    p.b.n_seqs = p.b.n_rows = int(n);
    p.b.max_new = 1;
    p.b.capacity = sel->blocks * p.kv.page_size;
    p.q = static_cast<const uint16_t *>(q);
    p.ldq = ldq;
    p.out = static_cast<uint16_t *>(out);
    p.ldo = ldo;
    p.heads = n_heads;
    p.group = n_heads / p.kv.heads;
    p.scale = scale;
    p.status = ctx_status(ctx);
    return done(ctx, stream, launch_attn_blocks(p, ctx_sms(ctx), stream), 64);
}

}  // extern "C"
