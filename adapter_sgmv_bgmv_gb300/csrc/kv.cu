// Writing new keys and values into the pages of the cache, and reading cached ones
// back as bf16 rows.
//
// One vector is the dim elements of one (row, head): dim / 16 lanes take 16 elements
// (32 bytes of bf16) each.  A CTA serves up to eight rows: a warp finds each row's sequence
// and cell, then all go over the rows' 2 * heads vectors (keys, then values).
//
// 8-bit formats, per vector: scale = max |x| / T (T = 127 for int8, 448 for e4m3; one
// fp32 division, rounded to nearest), code = x / scale rounded to nearest even and
// limited to +-T.  x / scale is the quotient as one fp32 division gives it (rounded to
// nearest), which a product with a rounded reciprocal may miss next to a tie.  A vector that
// holds an infinity or a NaN gets a NaN scale and zero codes, so it reads back as NaN; a zero vector gets
// scale 0.
//
// Bound: DRAM at prefill sizes (the vectors are read and written once), and one
// launch plus three dependent loads (starts and lens, page id, data) for a decode batch.
// Measured: 61,623 tokens of 8 heads of 128 from int8 to bf16 62 us, 6.1 TB/s (0.92 of a
// copy's rate); 16,896 tokens of 32 heads of 128 to e4m3 136 us and back 74 us, the write bound
// by the instructions of exact rounding; 64 tokens of 32 heads in bf16 4.5 us.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv.h"
#include "ptx.cuh"

#include "kv.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = kThreads / 32;      // rows a CTA: a warp looks up each

// Row `row`'s place in the cache, found by a whole warp: byte offset of the page's
// cell in the pools (without the head) and element offset in the scales.
struct Place {
    bool live;                // the row belongs to a sequence of the batch
    bool stored;              // ... and has a position and a valid page
    int64_t at, s_at;
};

__device__ __forceinline__ Place find_row(const KvView &kv, const BatchView &b, int row,
                                          unsigned *status)
{
    const int lane = threadIdx.x & 31;
    Place pl{false, false, 0, 0};
    // A decode batch has one row per sequence: row r is sequence r.  Otherwise a
    // 32-way search for the last sequence that starts at or before the row.
    int s = row;
    bool hit = s < b.n_seqs && b.starts[s] == row && b.starts[s + 1] == row + 1;
    if (!hit) {
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
        s = lo;
    }
    const SeqInfo q = seq_info(b, s, status);
    if (row < q.start || row >= q.start + q.n_new)
        return pl;
    pl.live = true;
    const int pos = q.len - q.n_new + (row - q.start);
    if (pos < 0)
        return pl;
    const int j = page_of(kv, pos);
    const int page = b.pages[int64_t(s) * b.ld_pages + j];
    if (page < 0 || page >= kv.n_pages) {
        raise_status(status, kDevBadPage);
        return pl;
    }
    const int cell = pos - j * kv.page_size;
    pl.stored = true;
    pl.at = page * kv.page_stride + cell * kv.cell_stride;
    pl.s_at = page * kv.s_page + cell * kv.s_cell;
    return pl;
}

// `rows` rows from the CTA's first: their vectors one after another, kPer at a time.
template <int DIM, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_write(const __grid_constant__ KvRowsParams p, int rows)
{
    constexpr int kLanes = DIM / 16;                 // lanes per vector
    constexpr int kPer = kThreads / kLanes;          // vectors per pass of the CTA
    constexpr int kUnroll = 2;
    __shared__ Place places[kMaxRows];
    const int row0 = blockIdx.x * rows, sub = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
    const int warp = threadIdx.x >> 5;
    const KvView &kv = p.kv;
    grid_dep_wait();
    grid_dep_launch();
    const int nvec = 2 * kv.heads, all = min(rows, p.b.n_rows - row0) * nvec;
    const int stride = gridDim.y * kPer * kUnroll;
    uint4 x[kUnroll][2];
    auto load = [&](int v0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = v0 + u * kPer + sub, r = p.per_row.quotient(i), row = row0 + r, vec = i - r * nvec;
            const bool is_v = vec >= kv.heads;
            const uint16_t *src = (is_v ? p.v + int64_t(row) * p.ldv - kv.heads * DIM : p.k + int64_t(row) * p.ldk) + vec * DIM + l * 16;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                x[u][e] = i < all ? reinterpret_cast<const uint4 *>(src)[e] : uint4{0, 0, 0, 0};
        }
    };
    // the first vectors are on their way while the rows' places are looked up
    int v0 = blockIdx.y * kPer * kUnroll;
    load(v0);
    if (warp < rows) {
        const Place pl = row0 + warp < p.b.n_rows ? find_row(kv, p.b, row0 + warp, p.status) : Place{false, false, 0, 0};
        if ((threadIdx.x & 31) == 0)
            places[warp] = pl;
    }
    __syncthreads();
    for (; v0 < all; v0 += stride) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = v0 + u * kPer + sub, r = p.per_row.quotient(i), vec = i - r * nvec;
            const Place &pl = places[min(r, rows - 1)];
            const bool on = i < all && pl.stored, is_v = vec >= kv.heads;
            const int head = is_v ? vec - kv.heads : vec;
            uint8_t *dst = (is_v ? kv.v : kv.k) + pl.at + head * kv.head_stride;
            if (FMT == kKvBf16) {
                if (on) {
                    reinterpret_cast<uint4 *>(dst + l * 32)[0] = x[u][0];
                    reinterpret_cast<uint4 *>(dst + l * 32)[1] = x[u][1];
                }
            } else {
                float scale;
                const uint4 code = encode16<FMT, kLanes>(x[u], scale);
                if (on) {
                    *reinterpret_cast<uint4 *>(dst + l * 16) = code;
                    if (l == 0)
                        (is_v ? kv.v_scale : kv.k_scale)[pl.s_at + head * kv.s_head] = scale;
                }
            }
        }
        if (v0 + stride < all)
            load(v0 + stride);
    }
}

template <int DIM, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_read(const __grid_constant__ KvRowsParams p, int rows)
{
    constexpr int kLanes = DIM / 16;
    constexpr int kPer = kThreads / kLanes;
    constexpr int kUnroll = 2;
    __shared__ Place places[kMaxRows];
    const int row0 = blockIdx.x * rows, sub = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
    const int warp = threadIdx.x >> 5;
    const KvView &kv = p.kv;
    grid_dep_wait();
    grid_dep_launch();
    const int nvec = 2 * kv.heads, all = min(rows, p.b.n_rows - row0) * nvec;
    if (warp < rows) {
        const Place pl = row0 + warp < p.b.n_rows ? find_row(kv, p.b, row0 + warp, p.status) : Place{false, false, 0, 0};
        if ((threadIdx.x & 31) == 0)
            places[warp] = pl;
    }
    __syncthreads();
    for (int v0 = blockIdx.y * kPer * kUnroll; v0 < all; v0 += gridDim.y * kPer * kUnroll) {
        uint4 x[kUnroll][2];
        float scale[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = v0 + u * kPer + sub, r = p.per_row.quotient(i), vec = i - r * nvec;
            const Place &pl = places[min(r, rows - 1)];
            x[u][0] = x[u][1] = uint4{0, 0, 0, 0};
            scale[u] = 0.f;
            if (i < all && pl.stored) {
                const bool is_v = vec >= kv.heads;
                const int head = is_v ? vec - kv.heads : vec;
                const uint8_t *src = (is_v ? kv.v : kv.k) + pl.at + head * kv.head_stride;
                if (FMT == kKvBf16) {
                    x[u][0] = reinterpret_cast<const uint4 *>(src + l * 32)[0];
                    x[u][1] = reinterpret_cast<const uint4 *>(src + l * 32)[1];
                } else {
                    x[u][0] = *reinterpret_cast<const uint4 *>(src + l * 16);
                    scale[u] = (is_v ? kv.v_scale : kv.k_scale)[pl.s_at + head * kv.s_head];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = v0 + u * kPer + sub, r = p.per_row.quotient(i), row = row0 + r, vec = i - r * nvec;
            const Place &pl = places[min(r, rows - 1)];
            if (i >= all || !pl.live)
                continue;
            const bool is_v = vec >= kv.heads;
            uint16_t *dst = (is_v ? p.v + int64_t(row) * p.ldv - kv.heads * DIM : p.k + int64_t(row) * p.ldk) + vec * DIM + l * 16;
            uint4 y[2] = {x[u][0], x[u][1]};
            if (FMT != kKvBf16)
                decode16<FMT>(x[u][0], scale[u], y);       // no cell: zero codes, zero scale
            reinterpret_cast<uint4 *>(dst)[0] = y[0];
            reinterpret_cast<uint4 *>(dst)[1] = y[1];
        }
    }
}

template <typename F>
cudaError_t launch(F kernel, KvRowsParams p, cudaStream_t stream)
{
    // As many rows a CTA as leave two CTAs for each of 152 SMs (their look-ups then run side
    // by side); a few rows of many vectors are cut instead, to spread over the SMs.
    const int rows = int(std::min<int64_t>(kMaxRows, std::max<int64_t>(1, p.b.n_rows / 304)));
    const int per = kThreads / (p.kv.dim / 16) * 2;
    p.per_row = Divider(2 * p.kv.heads);
    const int parts = rows == 1 ? (2 * p.kv.heads + per - 1) / per : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((p.b.n_rows + rows - 1) / rows), unsigned(parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, rows);
}

}  // namespace

cudaError_t launch_kv_write(const KvRowsParams &p, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    switch (p.kv.format) {
    case kKvBf16: return wide ? launch(k_kv_write<128, kKvBf16>, p, stream) : launch(k_kv_write<64, kKvBf16>, p, stream);
    case kKvInt8: return wide ? launch(k_kv_write<128, kKvInt8>, p, stream) : launch(k_kv_write<64, kKvInt8>, p, stream);
    default: return wide ? launch(k_kv_write<128, kKvFp8>, p, stream) : launch(k_kv_write<64, kKvFp8>, p, stream);
    }
}

cudaError_t launch_kv_read(const KvRowsParams &p, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    switch (p.kv.format) {
    case kKvBf16: return wide ? launch(k_kv_read<128, kKvBf16>, p, stream) : launch(k_kv_read<64, kKvBf16>, p, stream);
    case kKvInt8: return wide ? launch(k_kv_read<128, kKvInt8>, p, stream) : launch(k_kv_read<64, kKvInt8>, p, stream);
    default: return wide ? launch(k_kv_read<128, kKvFp8>, p, stream) : launch(k_kv_read<64, kKvFp8>, p, stream);
    }
}

}  // namespace lora
