// What the files of the cache's C ABI share: the handle and the checks of its arguments.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/lora.h"
#include "ctx.h"
#include "kv.h"

struct lora_kv {
    lora_ctx *ctx = nullptr;           // not owned
    lora::KvView view{};
    lora::AttnScratch few{}, many{};   // in the context's scratch
};

namespace lora {

// Positions stay below this, so that position arithmetic with a window or a tile's
// width added fits in 32 bits.
constexpr int64_t kMaxPosition = int64_t(1) << 30;

inline bool aligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool rows_ok(const void *p, int64_t ld, int64_t width)
{
    return aligned(p, 16) && ld >= width && ld % 8 == 0;
}

// The batch of a call over `n` rows; LORA_OK or the error it gets.  Without a cache the page
// table is not looked at.
inline int take_batch(const lora_kv *kv, const lora_kv_batch *b, int64_t n, BatchView &v)
{
    if (!b || n < 0 || b->n_seqs < 0 || b->n_cols < 0 || b->ld_pages < b->n_cols || b->max_new < 0)
        return LORA_E_INVAL;
    if (n >= (int64_t(1) << 31) || b->n_seqs >= (int64_t(1) << 31) - 1)
        return LORA_E_CAPACITY;
    if (b->n_seqs > 0 && (!aligned(b->starts, 4) || !aligned(b->lens, 4) ||
                          (kv && b->n_cols > 0 && !aligned(b->pages, 4))))
        return LORA_E_INVAL;
    v.starts = b->starts;
    v.lens = b->lens;
    v.pages = b->pages;
    v.ld_pages = b->ld_pages;
    v.n_seqs = int(b->n_seqs);
    v.n_rows = int(n);
    v.max_new = int(std::min<int64_t>(b->max_new, n));
    const int64_t room = !kv || b->n_cols > kMaxPosition / kv->view.page_size ? kMaxPosition
                         : b->n_cols * kv->view.page_size;
    v.capacity = int(room);
    return LORA_OK;
}

}  // namespace lora
