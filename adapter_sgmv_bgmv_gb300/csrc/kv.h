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

#ifdef __CUDACC__
struct SeqInfo {
    int start, n_new, len;
};

// Sequence s of the batch; one whose rows or length are out of range counts as having
// no rows and raises the status.
__device__ __forceinline__ SeqInfo seq_info(const BatchView &b, int s, unsigned *status)
{
    SeqInfo q;
    q.start = b.starts[s];
    const int end = b.starts[s + 1];
    q.len = b.lens[s];
    q.n_new = end - q.start;
    if (q.start < 0 || end < q.start || end > b.n_rows || q.n_new > b.max_new || q.len < 0 ||
        q.len > b.capacity) {
        raise_status(status, kDevBadBatch);
        q.start = q.n_new = q.len = 0;
    }
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
