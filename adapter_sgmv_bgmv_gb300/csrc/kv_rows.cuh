// Where a row of a call is: its sequence and position, and its cell in the cache.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "kv.h"
#include "ptx.cuh"

namespace lora {

struct RowAt {
    bool live;                // the row belongs to a sequence of the batch
    int s, pos;               // which one, and the row's position in it (may be negative)
    SeqInfo q;
};

// Row `row`'s sequence and position, found by a whole warp.
__device__ __forceinline__ RowAt find_pos(const BatchView &b, int row, unsigned *status)
{
    const int lane = threadIdx.x & 31;
    // A decode batch has one row per sequence: row r is sequence r (its length is on its way with
    // its rows).  Otherwise a 32-way search for the last sequence that starts at or before the row.
    const bool may = row < b.n_seqs;
    const int start = may ? b.starts[row] : -1, end = may ? b.starts[row + 1] : -1, len = may ? b.lens[row] : 0;
    RowAt r{false, row, -1, {}};
    if (b.n_seqs == 0)
        return r;
    if (start == row && end == row + 1) {
        r.q = checked_seq(b, start, end, len, status);
    } else {
        int lo = 0, n = b.n_seqs;                    // starts[lo] <= row, answer in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int i = lo + lane * step;
            const bool le = lane * step < n && b.starts[i] <= row;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            const int last = m ? 31 - __clz(m) : 0;
            n = min(step, n - last * step);
            lo += last * step;
        }
        r.s = lo;
        r.q = seq_info(b, lo, status);
    }
    if (row < r.q.start || row >= r.q.start + r.q.n_new)
        return r;
    r.live = true;
    r.pos = r.q.len - r.q.n_new + (row - r.q.start);
    return r;
}

// Row `row`'s place in the cache: byte offset of the page's cell in the pools (without
// the head) and element offset in the scales.
struct Place {
    bool live;
    bool stored;              // the row has a position and a valid page
    int64_t at, s_at;
};

__device__ __forceinline__ Place place_of(const KvView &kv, const BatchView &b, const RowAt &r, unsigned *status)
{
    Place pl{r.live, false, 0, 0};
    if (!r.live || r.pos < 0)
        return pl;
    const int j = page_of(kv, r.pos);
    const int page = b.pages[int64_t(r.s) * b.ld_pages + j];
    if (page < 0 || page >= kv.n_pages) {
        raise_status(status, kDevBadPage);
        return pl;
    }
    const int cell = r.pos - j * kv.page_size;
    pl.stored = true;
    pl.at = page * kv.page_stride + cell * kv.cell_stride;
    pl.s_at = page * kv.s_page + cell * kv.s_cell;
    return pl;
}

__device__ __forceinline__ Place find_row(const KvView &kv, const BatchView &b, int row, unsigned *status)
{
    return place_of(kv, b, find_pos(b, row, status), status);
}

}  // namespace lora
