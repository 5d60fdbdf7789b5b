// Attention over a part of the cache: bounds of each page's keys, and the choice of pages for
// every new token and key head by a cheap score (the attention over what is chosen is
// attn_rows.cu's, each row a sequence with a page list for each key head).
//
// Bounds: the smallest and largest key of a page for each element, as 8-bit codes with one
// power-of-two unit for a page and head.  Score of a page for a row:
//
//   max over the group's query heads g of  unit_page unit_g sum_d max(c_d lo_d, c_d hi_d)
//
// with c the codes of query head g, taken the same way.  Units that are powers of two make
// every step exact: codes are x / unit rounded once, the sum is of integers below 2^21 (dp4a),
// the products with the units only move the exponent.  The choice so depends on the inputs
// alone, not on the order of sums, and equal scores go to the lower page.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv.h"
#include "kv.cuh"
#include "kv_rows.cuh"
#include "launch.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The unit for numbers up to `top`: 2^(e - 6) with 2^e <= top < 2^(e + 1), e at least -100; and
// its reciprocal.  NaN where top is not finite.
__device__ __forceinline__ float unit_for(float top, float &inverse)
{
    const int e = max(int(__float_as_uint(top) >> 23 & 0xffu) - 127, -100);
    inverse = __uint_as_float(uint32_t(127 + 6 - e) << 23);
    return top < INFINITY ? __uint_as_float(uint32_t(127 - 6 + e) << 23) : __int_as_float(0x7fffffff);
}

__device__ __forceinline__ int code_of(float x, float inverse) { return max(-127, min(127, __float2int_rn(x * inverse))); }

// ---------------------------------------------------------------- bounds

// A CTA looks at `rows` rows of the call: each that is its sequence's first in a page stands for
// the page, and the page's vectors [cells][dim] of each head are a warp's.  Every page touched
// is read once; DRAM bounds it.
template <int DIM, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_bounds(const __grid_constant__ BoundsParams p, int rows)
{
    constexpr int E = FMT == kKvBf16 ? 8 : 16;       // elements of a lane's 16 bytes
    constexpr int L = DIM / E, CW = 32 / L;          // lanes of a cell, cells a warp's load
    constexpr int U = 8;
    __shared__ int pages[kThreads], filled[kThreads], n_pages;
    const KvView &kv = p.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x == 0)
        n_pages = 0;
    __syncthreads();
    const int row = blockIdx.x * rows + int(threadIdx.x);
    if (int(threadIdx.x) < rows && row < p.b.n_rows) {
        int s = row;
        if (!(s < p.b.n_seqs && p.b.starts[s] == row && p.b.starts[s + 1] == row + 1)) {
            int lo = 0, hi = p.b.n_seqs - 1;         // the last sequence that starts at or before the row
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.b.starts[mid] <= row)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            s = lo;
        }
        const SeqInfo q = seq_info(p.b, s, p.status);
        const int pos = q.len - q.n_new + (row - q.start);
        if (row >= q.start && row < q.start + q.n_new && pos >= 0) {
            const int col = page_of(kv, pos), cell = pos - col * kv.page_size;
            if (row == q.start || cell == 0) {
                const int page = p.b.pages[int64_t(s) * p.b.ld_pages + col];
                if (page < 0 || page >= kv.n_pages) {
                    raise_status(p.status, kDevBadPage);
                } else {
                    const int at = atomicAdd(&n_pages, 1);
                    pages[at] = page;
                    filled[at] = min(kv.page_size, q.len - col * kv.page_size);
                }
            }
        }
    }
    __syncthreads();
    const int items = n_pages * kv.heads;
    const int sub = lane % L, off = lane / L;
    for (int it = int(blockIdx.y) * kWarps + warp; it < items; it += int(gridDim.y) * kWarps) {
        const int slot = it / kv.heads, head = it - slot * kv.heads, n = filled[slot];
        const int64_t page = pages[slot];
        const uint8_t *src = kv.k + page * kv.page_stride + head * kv.head_stride + sub * 16;
        const float *scales = FMT == kKvBf16 ? nullptr : kv.k_scale + page * kv.s_page + head * kv.s_head;
        float lo[E], hi[E];
        __nv_bfloat162 lo2[4], hi2[4];
#pragma unroll
        for (int e = 0; e < E; ++e)
            lo[e] = INFINITY, hi[e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo2[e] = __floats2bfloat162_rn(INFINITY, INFINITY);
            hi2[e] = __floats2bfloat162_rn(-INFINITY, -INFINITY);
        }
        for (int c0 = off; c0 < n; c0 += CW * U) {
            uint4 x[U];
            float sc[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past the end the first cell again: it changes nothing
                const int c = c0 + u * CW < n ? c0 + u * CW : 0;
                x[u] = *reinterpret_cast<const uint4 *>(src + c * kv.cell_stride);
                sc[u] = FMT == kKvBf16 ? 1.f : scales[c * kv.s_cell];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (FMT == kKvBf16) {
                    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x[u]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        lo2[e] = __hmin2_nan(lo2[e], h[e]);
                        hi2[e] = __hmax2_nan(hi2[e], h[e]);
                    }
                } else {
                    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 v = widen4<FMT == kKvFp8 ? kKvFp8 : kKvInt8>(w[i]);
                        const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                            __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            lo[(4 * i + e) % E] = min_nan(lo[(4 * i + e) % E], f[e] * sc[u]);
                            hi[(4 * i + e) % E] = max_nan(hi[(4 * i + e) % E], f[e] * sc[u]);
                        }
                    }
                }
            }
        }
        if (FMT == kKvBf16)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[2 * e] = __low2float(lo2[e]), lo[2 * e + 1] = __high2float(lo2[e]);
                hi[2 * e] = __low2float(hi2[e]), hi[2 * e + 1] = __high2float(hi2[e]);
            }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int o = L; o < 32; o <<= 1) {
                lo[e] = min_nan(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
                hi[e] = max_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
            }
            top = max_nan(top, max_nan(fabsf(lo[e]), fabsf(hi[e])));
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        float inverse;
        const float unit = unit_for(top, inverse);
        if (off == 0) {
            uint32_t c[2][E / 4];
#pragma unroll
            for (int w = 0; w < E / 4; ++w) {
                c[0][w] = c[1][w] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (unit == unit) {
                        c[0][w] |= uint32_t(code_of(lo[4 * w + e], inverse) & 0xff) << (8 * e);
                        c[1][w] |= uint32_t(code_of(hi[4 * w + e], inverse) & 0xff) << (8 * e);
                    }
            }
            int8_t *dst = kv.bounds + (page * kv.heads + head) * 2 * DIM + sub * E;
#pragma unroll
            for (int side = 0; side < 2; ++side)
                if (E == 16)
                    *reinterpret_cast<uint4 *>(dst + side * DIM) = make_uint4(c[side][0], c[side][1], c[side][E / 4 - 2], c[side][E / 4 - 1]);
                else
                    *reinterpret_cast<uint2 *>(dst + side * DIM) = make_uint2(c[side][0], c[side][1]);
            if (sub == 0)
                kv.unit[page * kv.heads + head] = unit;
        }
    }
}

template <int DIM, int FMT>
cudaError_t launch(const BoundsParams &p, cudaStream_t stream)
{
    // A CTA has about one page: its rows of a prompt, one row where sequences have few each.
    const int64_t n = p.b.n_rows, touched = n / p.kv.page_size + p.b.n_seqs;
    const int rows = int(std::max<int64_t>(1, std::min<int64_t>(kThreads, n / std::max<int64_t>(1, touched))));
    const dim3 grid(unsigned((n + rows - 1) / rows), unsigned(std::min((p.kv.heads + kWarps - 1) / kWarps, 64)));
    return start(k_kv_bounds<DIM, FMT>, grid, kThreads, 0, 0, stream, p, rows);
}

// ---------------------------------------------------------------- select

constexpr int kMaxCluster = 8;
constexpr int kPassBits[3] = {11, 11, 10};
constexpr int kBins = 1 << 11;
constexpr int kMaxShare = 1 << 15;           // columns of a CTA: four bytes of shared memory each

// An order-preserving integer of a score; no zero is negative.
__device__ __forceinline__ uint32_t key_of(float score)
{
    const uint32_t b = __float_as_uint(score + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int ld_cluster(const int *local, int rank)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_cluster(smem_u32(local), uint32_t(rank))) : "memory");
    return v;
}

// Exclusive prefix of one small value a thread over the block, and the sum.
__device__ __forceinline__ int block_prefix(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp)
            before += sums[w];
        total += sums[w];
    }
    return before + x - v;
}

// One (row, key head) a cluster of n_cta CTAs, which share its pages' columns.
template <int DIM>
__global__ void __launch_bounds__(kThreads) k_block_select(const __grid_constant__ SelectParams p, int n_cta)
{
    constexpr int L = DIM / 16, PW = 32 / L;         // lanes of a page, pages a warp's load
    constexpr int U = 4;
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *qpos = reinterpret_cast<uint32_t *>(smem), *qneg = qpos + p.group * DIM / 4;   // codes above and below zero
    float *q_unit = reinterpret_cast<float *>(qneg + p.group * DIM / 4);
    int *hist = reinterpret_cast<int *>(q_unit + ((p.group + 3) & ~3));                       // one for each pass
    uint32_t *keys = reinterpret_cast<uint32_t *>(hist + 3 * kBins);
    __shared__ int sums[kWarps], counts[2], found[2];
    const KvView &kv = p.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = int(cluster_ctarank());
    const int64_t work = int64_t(blockIdx.x) / n_cta;
    const int row = int(work / kv.heads), head = int(work - int64_t(row) * kv.heads);
    grid_dep_wait();
    grid_dep_launch();

    const RowAt at = find_pos(p.b, row, head == 0 && rank == 0 ? p.status : nullptr);
    const int pos = at.live ? at.pos : -1;
    const int cols = pos >= 0 ? page_of(kv, pos) + 1 : 0;    // pages the row sees
    const int32_t *table = p.b.pages + int64_t(at.s) * p.b.ld_pages;
    int32_t *out = p.pages + work * p.blocks;
    if (head == 0 && rank == 0 && threadIdx.x == 0)
        p.lens[row] = !at.live ? -1 : pos < 0 ? 0 : (min(cols, p.blocks) - 1) * kv.page_size + pos - (cols - 1) * kv.page_size + 1;
    const int choose = p.blocks - p.first - p.last;
    if (cols <= p.blocks || choose == 0) {
        // all of them, or no choice: the first and the last
        if (rank == 0)
            for (int i = threadIdx.x; i < p.blocks; i += kThreads)
                out[i] = i >= cols ? -1 : cols <= p.blocks || i < p.first ? table[i] : table[cols - p.blocks + i];
        return;
    }
    // the columns to choose from, this CTA's share of them
    const int n_cand = cols - p.first - p.last, share = (n_cand + n_cta - 1) / n_cta;
    const int c_lo = p.first + min(n_cand, rank * share), n = min(n_cand, (rank + 1) * share) - min(n_cand, rank * share);

    for (int g = warp; g < p.group; g += kWarps) {
        constexpr int N = DIM / 32;
        const uint16_t *src = p.q + row * p.ldq + int64_t(head * p.group + g) * DIM + lane * N;
        float f[N], top = 0.f, inverse;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            f[e] = __uint_as_float(uint32_t(src[e]) << 16);
            top = max_nan(top, fabsf(f[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float unit = unit_for(top, inverse);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int c = unit == unit ? code_of(f[e], inverse) : 0;
            reinterpret_cast<int8_t *>(qpos)[g * DIM + lane * N + e] = int8_t(max(c, 0));
            reinterpret_cast<int8_t *>(qneg)[g * DIM + lane * N + e] = int8_t(min(c, 0));
        }
        if (lane == 0)
            q_unit[g] = unit;
    }
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads)
        hist[i] = 0;
    __syncthreads();

    // Scores: L lanes a page, 16 elements of both bounds each.
    const int sub = lane % L, off = lane / L;
    for (int base = warp * PW * U; base < n; base += kWarps * PW * U) {
        uint4 lo[U], hi[U];
        float unit[U], best[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * PW + off;
            int page = i < n ? table[c_lo + i] : 0;
            if (page < 0 || page >= kv.n_pages) {
                raise_status(p.status, kDevBadPage);
                page = -1;
            }
            const int64_t at = int64_t(max(page, 0)) * kv.heads + head;
            const uint8_t *src = reinterpret_cast<const uint8_t *>(kv.bounds) + at * 2 * DIM + sub * 16;
            lo[u] = *reinterpret_cast<const uint4 *>(src);
            hi[u] = *reinterpret_cast<const uint4 *>(src + DIM);
            unit[u] = kv.unit[at];
            best[u] = -INFINITY;
            if (page < 0)
                unit[u] = -1.f;                      // chosen last
        }
#pragma unroll 1
        for (int g = 0; g < p.group; ++g) {
            const uint4 a = *reinterpret_cast<const uint4 *>(qpos + (g * DIM + sub * 16) / 4);
            const uint4 b = *reinterpret_cast<const uint4 *>(qneg + (g * DIM + sub * 16) / 4);
            const float ug = q_unit[g];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int d = __dp4a(int(hi[u].x), int(a.x), __dp4a(int(lo[u].x), int(b.x), 0));
                d = __dp4a(int(hi[u].y), int(a.y), __dp4a(int(lo[u].y), int(b.y), d));
                d = __dp4a(int(hi[u].z), int(a.z), __dp4a(int(lo[u].z), int(b.z), d));
                d = __dp4a(int(hi[u].w), int(a.w), __dp4a(int(lo[u].w), int(b.w), d));
#pragma unroll
                for (int o = 1; o < L; o <<= 1)
                    d += __shfl_xor_sync(0xffffffffu, d, o);
                best[u] = fmaxf(best[u], float(d) * unit[u] * ug);       // a query that is not finite has no say
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * PW + off;
            if (sub == 0 && i < n)
                // a page that is not finite is looked at: its keys reach the result as they would
                keys[i] = unit[u] < 0.f ? 0u : unit[u] != unit[u] ? key_of(INFINITY) : key_of(best[u]);
        }
    }

    // The choose-th largest key over the cluster, digit by digit.
    uint32_t prefix = 0;
    int want = choose, shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        int *h = hist + pass * kBins;
        const int bits = pass < 2 ? 11 : 10;
        const uint32_t above = pass == 0 ? 0u : ~0u << shift;
        shift -= bits;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads)
            if ((keys[i] & above) == prefix)
                atomicAdd(&h[keys[i] >> shift & ((1u << bits) - 1)], 1);
        if (n_cta > 1) {
            __syncwarp();
            cluster_sync();
        } else
            __syncthreads();
        // thread t has bins of falling keys: eight (four) from the top down
        constexpr int B = kBins / kThreads;
        const int per = (1 << bits) / kThreads, top_bin = (1 << bits) - 1 - int(threadIdx.x) * per;
        int bin[B], mine = 0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            bin[b] = 0;
            if (b < per) {
                if (n_cta > 1)
                    for (int c = 0; c < n_cta; ++c)
                        bin[b] += ld_cluster(h + top_bin - b, c);
                else
                    bin[b] = h[top_bin - b];
            }
            mine += bin[b];
        }
        int total;
        int before = block_prefix(mine, sums, total);
        if (before < want && before + mine >= want) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (before < want && before + bin[b] >= want) {
                    found[0] = top_bin - b;
                    found[1] = want - before;
                }
                before += bin[b];
            }
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        want = found[1];                             // of the keys equal so far
    }
    // prefix is the key itself: all above it, and the first `want` equal ones by column

    int gt = 0, eq = 0;                              // ahead of this CTA's columns
    if (n_cta > 1) {
        int a = 0, b = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            a += keys[i] > prefix;
            b += keys[i] == prefix;
        }
        int t;
        block_prefix(a, sums, t);
        if (threadIdx.x == 0)
            counts[0] = t;
        block_prefix(b, sums, t);
        if (threadIdx.x == 0)
            counts[1] = t;
        __syncwarp();
        cluster_sync();
        for (int c = 0; c < rank; ++c) {
            gt += ld_cluster(&counts[0], c);
            eq += ld_cluster(&counts[1], c);
        }
    }
    for (int base = 0; base < n; base += kThreads) {
        const int i = base + int(threadIdx.x);
        const uint32_t key = i < n ? keys[i] : 0u;
        const bool more = i < n && key > prefix, same = i < n && key == prefix;
        int total;
        const int before = block_prefix(int(more) | int(same) << 16, sums, total);
        const int g = gt + (before & 0xffff), e = eq + (before >> 16);
        if (more || (same && e < want))
            out[p.first + g + min(e, want)] = table[c_lo + i];
        gt += total & 0xffff;
        eq += total >> 16;
    }
    if (rank == 0)
        for (int i = threadIdx.x; i < p.first; i += kThreads)
            out[i] = table[i];
    if (rank == n_cta - 1)
        for (int i = threadIdx.x; i < p.last; i += kThreads)
            out[p.blocks - p.last + i] = table[cols - p.last + i];
    if (n_cta > 1) {
        __syncwarp();
        cluster_sync();                              // others may still read this CTA's counts
    }
}

template <int DIM>
cudaError_t launch(const SelectParams &p, int sms, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, k_block_select<DIM>, 226 * 1024);
    if (e != cudaSuccess)
        return e;
    // Few rows over many pages are cut over more SMs, not below 256 pages a CTA.
    const int64_t units = int64_t(p.b.n_rows) * p.kv.heads;
    int c = 1;
    while (c < kMaxCluster && ((p.n_cols + c - 1) / c > kMaxShare || (units * c < 2 * sms && p.n_cols / c > 256)))
        c *= 2;
    const size_t codes = size_t(p.group) * DIM * 2 + size_t((p.group + 3) & ~3) * 4;
    return start(k_block_select<DIM>, dim3(unsigned(units * c)), kThreads,
                 codes + (3 * kBins + size_t((p.n_cols + c - 1) / c)) * 4, c, stream, p, c);
}

}  // namespace

cudaError_t launch_kv_bounds(const BoundsParams &p, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    switch (p.kv.format) {
    case kKvBf16: return wide ? launch<128, kKvBf16>(p, stream) : launch<64, kKvBf16>(p, stream);
    case kKvInt8: return wide ? launch<128, kKvInt8>(p, stream) : launch<64, kKvInt8>(p, stream);
    default: return wide ? launch<128, kKvFp8>(p, stream) : launch<64, kKvFp8>(p, stream);
    }
}

cudaError_t launch_block_select(const SelectParams &p, int sms, cudaStream_t stream)
{
    return p.kv.dim == 128 ? launch<128>(p, sms, stream) : launch<64>(p, sms, stream);
}

}  // namespace lora
