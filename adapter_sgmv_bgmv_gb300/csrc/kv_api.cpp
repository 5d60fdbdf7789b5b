// C ABI of the paged key/value cache (declared in include/lora.h): argument checks and
// launches.  No call reads the batch on the host or allocates: all of them can be
// captured in a CUDA graph whose replays see the lengths of the moment.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "../../include/lora.h"
#include "ctx.h"
#include "kv.h"

using namespace lora;

struct lora_kv {
    lora_ctx *ctx = nullptr;           // not owned
    KvView view{};
    AttnScratch few{}, many{};         // in the context's scratch
};

namespace {

// Positions stay below this, so that position arithmetic with a window or a tile's
// width added fits in 32 bits.
constexpr int64_t kMaxPosition = int64_t(1) << 30;

bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows (new tokens times query heads per key head) up to which a sequence's attention
// goes to the few-rows kernel: one unit of it.  Its second unit would read the keys again.
// 16 sequences of 2000 keys, 32 query heads on 8: 20 rows take 76 us there and 46 us in the
// other in bf16 (int8 72 and 58, e4m3 73 and 60); 12 rows 50 us here and 57 there in int8
// (e4m3 50 and 60).  In bf16 12 rows take 55 us here and 45 there; they stay for the weights'
// second term, so that the rule and the precision do not depend on the format.
constexpr int kFewRows = 16;

int log2_exact(int v)
{
    for (int s = 0; s < 31; ++s)
        if ((1 << s) == v)
            return s;
    return -1;
}

// The batch of a call over `n` rows; LORA_OK or the error it gets.
int take_batch(const lora_kv *kv, const lora_kv_batch *b, int64_t n, BatchView &v)
{
    if (!b || n < 0 || b->n_seqs < 0 || b->n_cols < 0 || b->ld_pages < b->n_cols || b->max_new < 0)
        return LORA_E_INVAL;
    if (n >= (int64_t(1) << 31) || b->n_seqs >= (int64_t(1) << 31) - 1)
        return LORA_E_CAPACITY;
    if (b->n_seqs > 0 && (!aligned(b->starts, 4) || !aligned(b->lens, 4) ||
                          (b->n_cols > 0 && !aligned(b->pages, 4))))
        return LORA_E_INVAL;
    v.starts = b->starts;
    v.lens = b->lens;
    v.pages = b->pages;
    v.ld_pages = b->ld_pages;
    v.n_seqs = int(b->n_seqs);
    v.n_rows = int(n);
    v.max_new = int(std::min<int64_t>(b->max_new, n));
    const int64_t room = b->n_cols > kMaxPosition / kv->view.page_size ? kMaxPosition
                         : b->n_cols * kv->view.page_size;
    v.capacity = int(room);
    return LORA_OK;
}

bool rows_ok(const void *p, int64_t ld, int64_t width)
{
    return aligned(p, 16) && ld >= width && ld % 8 == 0;
}

int rows_call(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, const void *k,
              int64_t ldk, const void *v, int64_t ldv, void *stream_ptr, bool write)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (!ctx || !kv || kv->ctx != ctx)
        return LORA_E_INVAL;
    KvRowsParams p{};
    p.kv = kv->view;
    int rc = take_batch(kv, b, n, p.b);
    if (rc != LORA_OK)
        return rc;
    const int64_t width = int64_t(p.kv.heads) * p.kv.dim;
    if (n > 0 && (!rows_ok(k, ldk, width) || !rows_ok(v, ldv, width)))
        return LORA_E_INVAL;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0 || b->n_seqs == 0)
        return rc;
    p.k = const_cast<uint16_t *>(static_cast<const uint16_t *>(k));
    p.v = const_cast<uint16_t *>(static_cast<const uint16_t *>(v));
    p.ldk = ldk;
    p.ldv = ldv;
    p.status = ctx_status(ctx);
    const cudaError_t e = write ? launch_kv_write(p, stream) : launch_kv_read(p, stream);
    if (e != cudaSuccess)
        return ctx_cuda_fail(ctx, e);
    ctx_launched(ctx, stream, 32);
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_kv_create(lora_ctx *ctx, const lora_kv_desc *d, lora_kv **out)
{
    if (!out)
        return LORA_E_INVAL;
    *out = nullptr;
    if (!ctx || !d || d->format < LORA_KV_BF16 || d->format > LORA_KV_FP8 || d->n_pages < 1 ||
        d->page_size < 1 || d->n_heads < 1 || !aligned(d->k_pool, 16) || !aligned(d->v_pool, 16))
        return LORA_E_INVAL;
    if (d->head_dim != 64 && d->head_dim != 128)
        return LORA_E_UNSUPPORTED;
    if (d->n_pages >= (int64_t(1) << 31) || d->page_size > (1 << 20) || d->n_heads > 4096)
        return LORA_E_CAPACITY;
    const int size = d->format == LORA_KV_BF16 ? 2 : 1;
    const int64_t strides[3] = {d->page_stride, d->cell_stride, d->head_stride};
    const int64_t count[3] = {d->n_pages, d->page_size, d->n_heads};
    for (int i = 0; i < 3; ++i)
        if (count[i] > 1 && (strides[i] < d->head_dim || (strides[i] * size) % 16))
            return LORA_E_INVAL;
    if (size == 1) {
        if (!aligned(d->k_scale, 4) || !aligned(d->v_scale, 4))
            return LORA_E_INVAL;
        const int64_t st[3] = {d->scale_page_stride, d->scale_cell_stride, d->scale_head_stride};
        for (int i = 0; i < 3; ++i)
            if (count[i] > 1 && st[i] < 1)
                return LORA_E_INVAL;
    }
    lora_kv *kv = new (std::nothrow) lora_kv();
    if (!kv)
        return LORA_E_NOMEM;
    kv->ctx = ctx;
    KvView &v = kv->view;
    v.k = static_cast<uint8_t *>(d->k_pool);
    v.v = static_cast<uint8_t *>(d->v_pool);
    v.k_scale = size == 1 ? d->k_scale : nullptr;
    v.v_scale = size == 1 ? d->v_scale : nullptr;
    v.page_stride = d->n_pages > 1 ? d->page_stride * size : 0;
    v.cell_stride = d->page_size > 1 ? d->cell_stride * size : 0;
    v.head_stride = d->n_heads > 1 ? d->head_stride * size : 0;
    v.s_page = d->n_pages > 1 ? d->scale_page_stride : 0;
    v.s_cell = d->page_size > 1 ? d->scale_cell_stride : 0;
    v.s_head = d->n_heads > 1 ? d->scale_head_stride : 0;
    v.n_pages = int(d->n_pages);
    v.page_size = d->page_size;
    v.page_shift = log2_exact(d->page_size);
    v.heads = d->n_heads;
    v.dim = d->head_dim;
    v.format = d->format;
    if (ctx_device(ctx) >= 0) {
        int rc = ctx_begin(ctx, nullptr);
        if (rc == LORA_OK) {
            uint8_t *base = nullptr;
            const size_t few = attn_rows_scratch(nullptr, ctx_sms(ctx), nullptr);
            rc = ctx_attn_scratch(ctx, few + attn_tc_scratch(nullptr, ctx_sms(ctx), nullptr), &base);
            if (rc == LORA_OK) {
                attn_rows_scratch(base, ctx_sms(ctx), &kv->few);
                attn_tc_scratch(base + few, ctx_sms(ctx), &kv->many);
            }
        }
        if (rc != LORA_OK) {
            delete kv;
            return rc;
        }
    }
    *out = kv;
    return LORA_OK;
}

int lora_kv_destroy(lora_kv *kv)
{
    if (!kv)
        return LORA_E_INVAL;
    delete kv;
    return LORA_OK;
}

int lora_kv_write(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, const void *k,
                  int64_t ldk, const void *v, int64_t ldv, void *stream)
{
    return rows_call(ctx, kv, b, n, k, ldk, v, ldv, stream, true);
}

int lora_kv_read(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, void *k,
                 int64_t ldk, void *v, int64_t ldv, void *stream)
{
    return rows_call(ctx, kv, b, n, k, ldk, v, ldv, stream, false);
}

int lora_attention(lora_ctx *ctx, const lora_kv *kv, const lora_kv_batch *b, int64_t n, const void *q,
                   int64_t ldq, int n_heads, float scale, int window, int sinks, void *out,
                   int64_t ldo, void *stream_ptr)
{
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (!ctx || !kv || kv->ctx != ctx || n_heads < 1 || n_heads % kv->view.heads || window < 0 ||
        sinks < 0 || !(scale - scale == 0.f))
        return LORA_E_INVAL;
    AttnParams p{};
    p.kv = kv->view;
    int rc = take_batch(kv, b, n, p.b);
    if (rc != LORA_OK)
        return rc;
    const int64_t width = int64_t(n_heads) * p.kv.dim;
    if (n > 0 && (!rows_ok(q, ldq, width) || !rows_ok(out, ldo, width)))
        return LORA_E_INVAL;
    if (n * n_heads >= (int64_t(1) << 31))
        return LORA_E_CAPACITY;
    rc = ctx_begin(ctx, stream);
    if (rc != LORA_OK || n == 0 || b->n_seqs == 0)
        return rc;
    p.q = static_cast<const uint16_t *>(q);
    p.ldq = ldq;
    p.out = static_cast<uint16_t *>(out);
    p.ldo = ldo;
    p.heads = n_heads;
    p.group = n_heads / p.kv.heads;
    p.scale = scale;
    p.window = int(std::min<int64_t>(window, kMaxPosition));
    p.sinks = int(std::min<int64_t>(sinks, kMaxPosition));
    p.status = ctx_status(ctx);
    // Sequences of few rows (decoding, a few tokens at once) and of many go to a kernel
    // each; which of them the batch has is known on the device only, so both are launched
    // unless max_new leaves out the second.
    const bool many = int64_t(p.b.max_new) * p.group > kFewRows;
    cudaError_t e = cudaSuccess;
    if (many) {
        p.min_rows = kFewRows + 1;
        p.max_rows = int64_t(1) << 40;
        p.part = kv->many;
        e = launch_attn_tc(p, ctx_sms(ctx), stream);
        if (e != cudaSuccess)
            return ctx_cuda_fail(ctx, e);
        ctx_launched(ctx, stream, 128);
    }
    p.min_rows = 1;
    p.max_rows = kFewRows + 1;
    p.part = kv->few;
    p.behind = many;
    e = launch_attn_rows(p, ctx_sms(ctx), stream);
    if (e != cudaSuccess)
        return ctx_cuda_fail(ctx, e);
    ctx_launched(ctx, stream, 64);
    return LORA_OK;
}

}  // extern "C"
