// Paged key/value cache: what its kernels (kv.cu, attn_rows.cu, attn_tc.cu) and the
// C-ABI layer share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "status.h"
#ifdef __CUDACC__
#include "ptx.cuh"
#endif

struct lora_ctx;

namespace lora {

enum KvFormat : int { kKvBf16 = 0, kKvInt8 = 1, kKvFp8 = 2 };

// The cache: element (page, cell, head, d) of the key pool is at
// k + page * page_stride + cell * cell_stride + head * head_stride (bytes), d
// consecutive; the value pool has the same strides.  Its scale (8-bit formats) is at
// k_scale[page * s_page + cell * s_cell + head * s_head].
struct KvView {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, cell_stride, head_stride;
    int64_t s_page, s_cell, s_head;
    int n_pages;
    int page_size;
    int page_shift;           // log2(page_size), or -1
    int heads;
    int dim;
    int format;
    // each page's smallest and largest keys, where the cache has them (bounds below): codes
    // at bounds[((page * heads + head) * 2 + side) * dim + d], units at unit[page * heads + head]
    int8_t *bounds;
    float *unit;
};

// The sequences of one call: rows [starts[s], starts[s + 1]) of q / k / v are the last
// new tokens of sequence s, whose length with them is lens[s]; position p is cell
// p % page_size of page pages[s * ld_pages + p / page_size].
struct BatchView {
    const int32_t *starts, *lens, *pages;
    int64_t ld_pages;
    int n_seqs;
    int n_rows;               // rows of q / k / v
    int max_new;              // upper bound on a sequence's new tokens
    int capacity;             // positions the page table has room for
    // Without `starts`, row s is sequence s (none where lens[s] is negative), and each key head
    // has a page list of its own, head_pages apart.
    int64_t head_pages;
};

// i / d by a product, for 0 <= i and i * d < 2^32.
struct Divider {
    uint32_t m = 0;
    Divider() = default;
    explicit Divider(int d) : m(d > 1 ? uint32_t(((uint64_t(1) << 32) + d - 1) / d) : 0) {}
#ifdef __CUDACC__
    __device__ __forceinline__ int quotient(int i) const { return int(m ? __umulhi(uint32_t(i), m) : uint32_t(i)); }
#endif
};

struct KvRowsParams {
    KvView kv;
    BatchView b;
    uint16_t *k, *v;          // bf16 rows, read by the write and written by the read
    int64_t ldk, ldv;
    Divider per_row;          // by a row's vectors
    unsigned *status;
};
cudaError_t launch_kv_write(const KvRowsParams &p, cudaStream_t stream);
cudaError_t launch_kv_read(const KvRowsParams &p, cudaStream_t stream);

// Partial results of units split over workers, in device memory.  A partial is each of a
// unit's rows' unnormalised output [dim] (fp32) and its running maximum and sum of
// weights.  `arrived` has one counter per CTA, zero between calls.
struct AttnScratch {
    float *cta_o;             // two partials per CTA
    float2 *cta_ml;
    float *warp_o;            // one per warp
    float2 *warp_ml;
    int *arrived;
};
// Lay the partials of the few-rows / many-rows kernel out in `base`; return their bytes.
size_t attn_rows_scratch(uint8_t *base, int sms, AttnScratch *s);
size_t attn_tc_scratch(uint8_t *base, int sms, AttnScratch *s);

struct AttnParams {
    KvView kv;
    BatchView b;
    const uint16_t *q;
    int64_t ldq;
    uint16_t *out;
    int64_t ldo;
    int heads;                // query heads
    int group;                // query heads that share a key head
    float scale;
    int window;               // 0: none
    int sinks;
    int64_t min_rows, max_rows;   // sequences this launch serves: min <= new * group < max
    AttnScratch part;
    unsigned *status;
    int behind;               // launched right behind the call's other kernel, which waited
                              // for the stream: start at once, wait for it before the end
};
cudaError_t launch_attn_rows(const AttnParams &p, int sms, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnParams &p, int sms, cudaStream_t stream);
// Rows over page lists of their own (no `starts`).
cudaError_t launch_attn_blocks(const AttnParams &p, int sms, cudaStream_t stream);

// Norm and rotation of heads (rope.cu), of a row's q_heads queries and k_heads keys; with
// `kv.k`, keys and values go to their cells instead of k_out.
struct RopeParams {
    KvView kv;
    BatchView b;
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out;
    int64_t ldq, ldk, ldv, ldqo, ldko;
    int q_heads, k_heads, dim, half, interleaved;
    const float *q_weight, *k_weight, *freqs;
    float eps;
    Divider per_row;          // by a row's items (rope.cu)
    unsigned *status;
};
cudaError_t launch_rope(const RopeParams &p, bool store, int sms, cudaStream_t stream);

// Page tables (pages.cu).
struct TableView {
    int32_t *lens, *pages, *refs;
    int64_t ld_pages;
    int n_seqs, n_cols, n_pages, page_size;
    int capacity;             // positions a sequence's row has room for
    unsigned *status;
};
constexpr int kMaxTableSeqs = 16384;
cudaError_t launch_pages_extend(const TableView &t, const int32_t *grow, int32_t *got, int32_t *src,
                                int32_t *dst, int32_t *cells, cudaStream_t stream);
cudaError_t launch_pages_fork(const TableView &t, const int32_t *from, const int32_t *to, int n, cudaStream_t stream);
cudaError_t launch_pages_free(const TableView &t, const int32_t *seqs, const int32_t *keep, int n, cudaStream_t stream);
cudaError_t launch_pages_compact(const TableView &t, int32_t *src, int32_t *dst, int n, int32_t *top, int *launches,
                                 cudaStream_t stream);

// Copies of pages within each of some caches of one shape (copy.cu).
constexpr int kMaxCopyCaches = 64;
struct KvCopyLists {
    const int32_t *src, *dst, *cells;
    int n;
};
cudaError_t launch_kv_copy(const KvView *kv, int n_kv, const KvCopyLists &lists, unsigned *status, int sms, cudaStream_t stream);

// Bounds of pages, and the choice of pages by them (blocks.cu).
struct BoundsParams {
    KvView kv;
    BatchView b;
    unsigned *status;
};
cudaError_t launch_kv_bounds(const BoundsParams &p, int sms, cudaStream_t stream);

constexpr int kMaxSelectCols = 44 << 10;
constexpr int kMaxSelectGroup = 128;
struct SelectParams {
    KvView kv;
    BatchView b;
    int n_cols;               // of the page table
    const uint16_t *q;
    int64_t ldq;
    int group, blocks, first, last;
    int32_t *lens, *pages;    // of the selection: [n_rows], [n_rows][heads][blocks]
    unsigned *status;
};
cudaError_t launch_block_select(const SelectParams &p, int sms, cudaStream_t stream);

#ifdef __CUDACC__
struct SeqInfo {
    int start, n_new, len;
};

// A sequence with rows [start, end) and length len; one whose rows or length are out of range
// counts as having no rows and raises the status.
__device__ __forceinline__ SeqInfo checked_seq(const BatchView &b, int start, int end, int len, unsigned *status)
{
    SeqInfo q;
    q.start = start;
    q.len = len;
    q.n_new = end - start;
    if (q.start < 0 || end < q.start || end > b.n_rows || q.n_new > b.max_new || q.len < 0 ||
        q.len > b.capacity) {
        raise_status(status, kDevBadBatch);
        q.start = q.n_new = q.len = 0;
    }
    return q;
}

// Sequence s of the batch.
__device__ __forceinline__ SeqInfo seq_info(const BatchView &b, int s, unsigned *status)
{
    return checked_seq(b, b.starts[s], b.starts[s + 1], b.lens[s], status);
}

// Sequence s of a batch without `starts`.
__device__ __forceinline__ SeqInfo row_info(const BatchView &b, int s, unsigned *status)
{
    SeqInfo q{s, 0, 0};
    const int len = b.lens[s];
    if (len > b.capacity)
        raise_status(status, kDevBadBatch);
    else if (len >= 0)
        q = SeqInfo{s, 1, len};
    return q;
}

__device__ __forceinline__ int page_of(const KvView &kv, int pos)
{
    return kv.page_shift >= 0 ? pos >> kv.page_shift : pos / kv.page_size;
}

// Whether the token at position p sees position j.
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks)
{
    return j <= p && (window == 0 || j > p - window || j < sinks);
}
#endif

}  // namespace lora
