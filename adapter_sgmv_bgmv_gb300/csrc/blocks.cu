// Attention over a part of the cache: bounds of each page's keys, and the choice of pages for
// every new token and key head by a cheap score (the attention over what is chosen is
// attn_blocks.cu's).
//
// Bounds: the smallest and largest key of a page for each element, as 8-bit codes with one
// power-of-two unit for a page and head.  Score of a page for a row:
//
//   max over the group's query heads g of  unit_page unit_g sum_d max(c_d lo_d, c_d hi_d)
//
// with c the codes of query head g, taken the same way.  Units that are powers of two make
// every step exact: codes are x / unit rounded once, the sum is of integers below 2^21,
// the products with the units only move the exponent, which has nine bits here (score_of): in fp32 they
// would leave its range, where keys and queries are both small or both large.  The choice so depends on
// the inputs alone, not on the order of sums, and equal scores go to the lower page.
//
// Measured (heads of 128).  Bounds: 16 prompts of 1056 tokens, 32 heads, bf16 24.6 us, 5.8 TB/s (0.86
// of a copy's rate); one decode's page of 64 tokens of 8 heads 3 us.  Choice: one row of 512 pages 6.3 us, 32
// rows of up to 409 pages, 64 heads on 8, 11.7 us (128 heads 16.4), 39 rows of up to 1504 pages, 28 heads on 4, 19 us:
// chains of latencies (lengths, pages, bounds, products, three passes over the scores, output).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

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

__device__ __forceinline__ float min3_nan(float a, float b, float c)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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
// the page, and the page's vectors [cells][dim] of each head are a warp's, four loads a lane (two in
// 8 bits) under way.  Every page touched is read once: DRAM bounds it in bf16, in 8 bits the rounds
// of loads, each waited for ahead of its conversions (16 prompts of 1056 tokens, 32 heads, 31 us, of which some 7 are
// instructions; with eight loads under way, and the registers that takes, 45).
template <int DIM, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_bounds(const __grid_constant__ BoundsParams p, int rows)
{
    constexpr int E = FMT == kKvBf16 ? 8 : 16;       // elements of a lane's 16 bytes
    constexpr int L = DIM / E, CW = 32 / L;          // lanes of a cell, cells a warp's load
    constexpr int U = FMT == kKvBf16 ? 4 : 2;
    __shared__ int pages[kThreads], filled[kThreads], n_pages;
    const KvView &kv = p.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x == 0)
        n_pages = 0;
    __syncthreads();
    // the last CTA's rows may go past 2^31
    const unsigned at_row = blockIdx.x * unsigned(rows) + threadIdx.x;
    if (int(threadIdx.x) < rows && at_row < unsigned(p.b.n_rows)) {
        const int row = int(at_row);
        int s = row;
        const bool may = row < p.b.n_seqs;
        const int start = may ? p.b.starts[row] : -1, end = may ? p.b.starts[row + 1] : -1, len = may ? p.b.lens[row] : 0;
        const bool hit = start == row && end == row + 1;
        if (!hit) {
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
        const SeqInfo q = hit ? checked_seq(p.b, start, end, len, p.status) : seq_info(p.b, s, p.status);
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
            for (int u = 0; u < U; u += 2) {
                if (FMT == kKvBf16) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x[u + v]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            lo2[e] = __hmin2_nan(lo2[e], h[e]);
                            hi2[e] = __hmax2_nan(hi2[e], h[e]);
                        }
                    }
                } else {
                    // two cells at once: instructions that take the least of three
                    float f[2][E];
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint32_t w[4] = {x[u + v].x, x[u + v].y, x[u + v].z, x[u + v].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint2 y = widen4<FMT == kKvFp8 ? kKvFp8 : kKvInt8>(w[i]);
                            float *at = f[v] + 4 * i % E;
                            at[0] = __uint_as_float(y.x << 16) * sc[u + v], at[1] = __uint_as_float(y.x & 0xffff0000u) * sc[u + v];
                            at[2] = __uint_as_float(y.y << 16) * sc[u + v], at[3] = __uint_as_float(y.y & 0xffff0000u) * sc[u + v];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        lo[e] = min3_nan(lo[e], f[0][e], f[1][e]);
                        hi[e] = max3_nan(hi[e], f[0][e], f[1][e]);
                    }
                }
            }
        }
        int8_t *dst = kv.bounds + (page * kv.heads + head) * 2 * DIM;
        float top = 0.f, inverse, unit;
        if constexpr (FMT == kKvBf16) {
            // every lane has all lanes' bounds of its elements, the first ones of each write them
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[2 * e] = __low2float(lo2[e]), lo[2 * e + 1] = __high2float(lo2[e]);
                hi[2 * e] = __low2float(hi2[e]), hi[2 * e + 1] = __high2float(hi2[e]);
            }
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
            unit = unit_for(top, inverse);
            if (off == 0) {
                uint32_t c[2][2] = {};
                if (unit == unit)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        c[0][e / 4] |= uint32_t(code_of(lo[e], inverse) & 0xff) << (e % 4 * 8);
                        c[1][e / 4] |= uint32_t(code_of(hi[e], inverse) & 0xff) << (e % 4 * 8);
                    }
                dst += sub * E;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0][0], c[0][1]);
                *reinterpret_cast<uint2 *>(dst + DIM) = make_uint2(c[1][0], c[1][1]);
            }
        } else {
            // Lanes with the same 16 elements join by halves: at each step a lane keeps one half of what
            // it has, its partner the other, until each has N of them.  (In bf16, where there is
            // less to join, this takes a quarter longer.)
            constexpr int N = DIM / 32;
            int first = sub * E;
#pragma unroll
            for (int o = L, half = E / 2; o < 32; o <<= 1, half >>= 1) {
                const bool upper = lane & o;
                first += upper ? half : 0;
#pragma unroll
                for (int e = 0; e < half; ++e) {
                    const float lo_give = upper ? lo[e] : lo[e + half], hi_give = upper ? hi[e] : hi[e + half];
                    lo[e] = min_nan(upper ? lo[e + half] : lo[e], __shfl_xor_sync(0xffffffffu, lo_give, o));
                    hi[e] = max_nan(upper ? hi[e + half] : hi[e], __shfl_xor_sync(0xffffffffu, hi_give, o));
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
                top = max_nan(top, max_nan(fabsf(lo[e]), fabsf(hi[e])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            unit = unit_for(top, inverse);
            uint32_t below = 0, above = 0;
            if (unit == unit)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    below |= uint32_t(code_of(lo[e], inverse) & 0xff) << (8 * e);
                    above |= uint32_t(code_of(hi[e], inverse) & 0xff) << (8 * e);
                }
            dst += first;
            if (N == 4) {
                *reinterpret_cast<uint32_t *>(dst) = below;
                *reinterpret_cast<uint32_t *>(dst + DIM) = above;
            } else {
                *reinterpret_cast<uint16_t *>(dst) = uint16_t(below);
                *reinterpret_cast<uint16_t *>(dst + DIM) = uint16_t(above);
            }
        }
        // (asked for as `lane == 0`, this leaves the compiler at 32 registers in bf16 instead of 40, with
        // fewer loads under way, and 16 prompts' bounds take a fifth longer)
        if (off == 0 && sub == 0)
            kv.unit[page * kv.heads + head] = unit;
    }
}

template <int DIM, int FMT>
cudaError_t launch(const BoundsParams &p, int sms, cudaStream_t stream)
{
    // A CTA has about one page: its rows of a prompt, one row where sequences have few each.
    const int64_t n = p.b.n_rows, touched = n / p.kv.page_size + p.b.n_seqs;
    const int rows = int(std::max<int64_t>(1, std::min<int64_t>(kThreads, n / std::max<int64_t>(1, touched))));
    // The heads too are dealt out to CTAs while these are fewer than twelve a SM.
    const int64_t ctas = (n + rows - 1) / rows;
    const int parts = int(std::max<int64_t>(1, std::min<int64_t>((p.kv.heads + kWarps - 1) / kWarps, 12 * int64_t(sms) / ctas)));
    const dim3 grid{unsigned(ctas), unsigned(parts)};
    return start(k_kv_bounds<DIM, FMT>, grid, kThreads, 0, 0, stream, p, rows);
}

// ---------------------------------------------------------------- select

constexpr int kMaxCluster = 8;
constexpr int kSelThreads = 256;
constexpr int kSelCtas = 3;                  // a SM
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;                   // of a pass over eight bits of the keys
constexpr int kTile = 16;                    // pages a warp scores at once

// Scores are compared as integers: the sign, nine bits of exponent and the sum's 20 bits behind its
// first one, in the places of an fp32 number shifted down by one (its last three bits are zeros), the
// exponent counted from 1 at |sum| = 1 and two units of the least exponent.
constexpr int kNoSay = INT_MIN;              // of a query head that is not finite: below every score

// Bits of a unit, 2^-106 to 2^121, in that place.
__device__ __forceinline__ int unit_bits(float unit) { return __float_as_int(unit) >> 1; }

// The score of a sum; `page` is unit_bits less the exponents' offset, `query` unit_bits or kNoSay (whose
// codes are zeros).
__device__ __forceinline__ int score_of(int sum, int page, int query)
{
    const int size = int((__float_as_uint(float(abs(sum))) >> 1) + uint32_t(page) + uint32_t(query));
    return sum == 0 ? query & kNoSay : sum < 0 ? -size : size;
}
constexpr int kExponents = (127 + 2 * (127 - 106) - 1) << 22;

constexpr uint32_t kNotThere = 0, kLowest = 1, kAbove = ~0u;     // keys of pages: a score's order, from kLowest up
__device__ __forceinline__ uint32_t key_of(int score) { return max(uint32_t(score) ^ 0x80000000u, kLowest); }

// 16 pages' bounds by 8 query heads' codes, 32 of the 2 * DIM products at once.
__device__ __forceinline__ void mma_s8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A query head's codes in shared memory: 16 bytes more than they need, so that two heads' pieces
// lie in different banks.
template <int DIM>
constexpr int kQueryBytes = 2 * DIM + 16;

// 32 bytes (on a boundary of as many) at once: four lanes have a 128-byte line of a page.
__device__ __forceinline__ void load32(const void *src, uint32_t x[8])
{
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                 : "l"(src) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t *local, int rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_cluster(smem_u32(local), uint32_t(rank))), "r"(v) : "memory");
}

// One (row, key head) a cluster of n_cta CTAs: they share the scoring of its pages, and the first
// one, which gets all scores in its shared memory, chooses.
//
// Scores: the 2 * DIM bytes of a page's bounds (lo, then hi) are one row of the products' left side,
// the codes of a query head (those below zero, then those above) one column of the right.  The
// order of the 2 * DIM is free as long as both sides have the same, so a lane takes 32-byte pieces
// of its two pages straight from memory.  (Drafts' 19 us are 28 with dp4a, and 23 with fp16 products of the
// widened codes, which take a third more registers; a cluster's own passes over all scores, instead of one
// CTA's, cost 3 us more for one row.)
template <int DIM>
__global__ void __launch_bounds__(kSelThreads, kSelCtas) k_block_select(const __grid_constant__ SelectParams p, int n_cta)
{
    constexpr int J = 2 * DIM / 128;                 // 128-byte lines of a page: a 32-byte piece for each of four lanes
    extern __shared__ __align__(16) uint8_t smem[];
    const int heads8 = (p.group + 7) & ~7;
    uint8_t *q_codes = smem;
    int *q_unit = reinterpret_cast<int *>(smem + heads8 * kQueryBytes<DIM>);      // [heads8]
    int *hist = reinterpret_cast<int *>(q_unit + heads8);                         // one for each of four passes
    uint32_t *keys = reinterpret_cast<uint32_t *>(hist + 4 * kBins);
    __shared__ int sums[2 * kSelWarps];
    const KvView &kv = p.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = int(cluster_ctarank()), c = lane & 3, g = lane >> 2;
    const int64_t work = int64_t(blockIdx.x) / n_cta;
    const int row = int(work / kv.heads), head = int(work - int64_t(row) * kv.heads);
    grid_dep_wait();
    grid_dep_launch();

    // the queries are on their way while the row's place is looked up, and so are the first pages
    // of the sequence that a decode batch's row belongs to
    constexpr int N = DIM / 32;
    constexpr int kStep = kSelWarps * kTile;
    const uint16_t *q = p.q + row * p.ldq + int64_t(head) * p.group * DIM + lane * N;
    uint2 mine = make_uint2(0, 0);
    auto query = [&](int h) {
        return N == 4 ? *reinterpret_cast<const uint2 *>(q + h * DIM) : make_uint2(*reinterpret_cast<const uint32_t *>(q + h * DIM), 0u);
    };
    if (warp < p.group)
        mine = query(warp);
    int base = warp * kTile, page[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int col = p.first + base + 8 * r + g;
        page[r] = row < p.b.n_seqs && col < p.n_cols ? p.b.pages[row * p.b.ld_pages + col] : -1;
    }
    for (int i = threadIdx.x; i < 4 * kBins; i += kSelThreads)
        hist[i] = 0;
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
            for (int i = threadIdx.x; i < p.blocks; i += kSelThreads)
                out[i] = i >= cols ? -1 : cols <= p.blocks || i < p.first ? table[i] : table[cols - p.blocks + i];
        return;
    }
    // the scores go to the first CTA's shared memory, which has to have started by then
    if (n_cta > 1) {
        __syncwarp();
        cluster_arrive_relaxed();
    }
    // the columns to choose from, [lo, hi) of them this CTA's
    const int n = cols - p.first - p.last, share = (n + n_cta - 1) / n_cta;
    const int lo = min(n, rank * share), hi = min(n, lo + share);
    table += p.first;

    // Two pages of a tile a lane: the first tile's bounds too are on their way while the queries become codes.
    uint32_t a[2][J][8];
    float unit[2];
    auto look_up = [&](int at) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            page[r] = at + 8 * r + g < hi ? table[at + 8 * r + g] : 0;
    };
    auto load = [&]() {                              // and the next tile's pages
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool there = page[r] >= 0 && page[r] < kv.n_pages;
            const int64_t where = int64_t(there ? page[r] : 0) * kv.heads + head;
            const int8_t *src = kv.bounds + where * 2 * DIM + c * 32;
#pragma unroll
            for (int j = 0; j < J; ++j)
                load32(src + 128 * j, a[r][j]);
            unit[r] = there ? kv.unit[where] : -1.f;
        }
        look_up(base + kStep);
    };
    base += lo;
    if (base < hi) {
        if (at.s != row || lo != 0)
            look_up(base);
        load();
    }
    for (int h = warp; h < heads8; h += kSelWarps) {
        const bool on = h < p.group;
        const uint2 x = !on ? make_uint2(0, 0) : h == warp ? mine : query(h);
        const float f[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u)};
        float top = 0.f, inverse;
#pragma unroll
        for (int e = 0; e < N; ++e)
            top = max_nan(top, fabsf(f[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float u = unit_for(top, inverse);
        uint32_t above = 0, below = 0;               // the lane's N codes
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int code = u == u ? code_of(f[e], inverse) : 0;
            above |= uint32_t(max(code, 0) & 0xff) << (8 * e);
            below |= uint32_t(min(code, 0) & 0xff) << (8 * e);
        }
        uint8_t *dst = q_codes + h * kQueryBytes<DIM> + lane * N;
        if (N == 4) {
            *reinterpret_cast<uint32_t *>(dst) = below;
            *reinterpret_cast<uint32_t *>(dst + DIM) = above;
        } else {
            *reinterpret_cast<uint16_t *>(dst) = uint16_t(below);
            *reinterpret_cast<uint16_t *>(dst + DIM) = uint16_t(above);
        }
        if (lane == 0)
            q_unit[h] = on && u == u ? unit_bits(u) : kNoSay;    // no head: no say
    }
    __syncthreads();

    while (base < hi) {
        int best[2] = {kNoSay, kNoSay};
        const int page_unit[2] = {unit_bits(unit[0]) - kExponents, unit_bits(unit[1]) - kExponents};
#pragma unroll 1
        for (int h = 0; h < heads8; h += 8) {
            const uint4 *b = reinterpret_cast<const uint4 *>(q_codes + (h + g) * kQueryBytes<DIM>) + 2 * c;
            int s[2][4] = {};                        // two chains of products
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 y = b[8 * j + e];
                    const uint32_t *x0 = a[0][j] + 4 * e, *x1 = a[1][j] + 4 * e;
                    mma_s8(s[0], x0[0], x1[0], x0[1], x1[1], y.x, y.y);
                    mma_s8(s[1], x0[2], x1[2], x0[3], x1[3], y.z, y.w);
                }
            // pages g and g + 8, heads 2c and 2c + 1; a query that is not finite has no say
            const int2 u = *reinterpret_cast<const int2 *>(q_unit + h + 2 * c);
#pragma unroll
            for (int r = 0; r < 2; ++r)
                best[r] = max(best[r], max(score_of(s[0][2 * r] + s[1][2 * r], page_unit[r], u.x), score_of(s[0][2 * r + 1] + s[1][2 * r + 1], page_unit[r], u.y)));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = max(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = max(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
            const int i = base + 8 * r + g;
            if (c == 0 && i < hi) {
                // a page that is not there comes last; one that is not finite is looked at: its keys
                // reach the result as they would
                if (unit[r] < 0.f)
                    raise_status(p.status, kDevBadPage);
                keys[i] = unit[r] < 0.f ? kNotThere : unit[r] != unit[r] ? kAbove : key_of(best[r]);
            }
        }
        base += kStep;
        if (base < hi)
            load();
    }
    __syncthreads();
    if (n_cta > 1) {
        __syncwarp();
        cluster_wait_acquire();
        if (rank != 0)
            for (int i = lo + int(threadIdx.x); i < hi; i += kSelThreads)
                st_cluster(keys + i, 0, keys[i]);
        __syncwarp();
        cluster_sync();
        if (rank != 0)
            return;
    }

    // The choose-th largest key, eight bits at a time.  Every warp looks through the counts itself:
    // one barrier a pass.
    uint32_t prefix = 0;
    int want = choose;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        int *h = hist + pass * kBins;
        const int shift = 24 - 8 * pass;
        const uint32_t above = pass == 0 ? 0u : ~0u << (shift + 8);
        for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {
            const uint32_t key = i0 + lane < n ? keys[i0 + lane] : 0u;
            const bool in = i0 + lane < n && (key & above) == prefix;
            const int digit = in ? int(key >> shift & (kBins - 1)) : -1;
            // most keys have the same first digit: one addition for each digit of a warp
            const unsigned same = pass == 0 ? __match_any_sync(0xffffffffu, digit) : 1u << lane;
            if (in && __ffs(same) - 1 == lane)
                atomicAdd(&h[digit], __popc(same));
        }
        __syncthreads();
        // lane l has eight bins, from 255 - 8 l down
        const int low = kBins - 8 - 8 * lane;
        const int4 x = *reinterpret_cast<const int4 *>(h + low), y = *reinterpret_cast<const int4 *>(h + low + 4);
        const int bin[8] = {y.w, y.z, y.y, y.x, x.w, x.z, x.y, x.x};
        int all = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b)
            all += bin[b];
        int upto = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d)
                upto += y;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, upto >= want)) - 1;
        int rest = want - (upto - all), digit = 0, count = 0;
        bool done = false;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            if (!done) {
                digit = low + 7 - b;
                count = bin[b];
                done = rest <= bin[b];
                rest -= done ? 0 : bin[b];
            }
        }
        prefix |= uint32_t(__shfl_sync(0xffffffffu, digit, src)) << shift;
        want = __shfl_sync(0xffffffffu, rest, src);  // of the keys equal so far
        if (want == __shfl_sync(0xffffffffu, count, src) && prefix) {
            prefix -= 1;                             // all of them: no need to tell them apart
            want = 0;
            break;
        }
    }

    // All keys above prefix, and the first `want` of those equal to it, in the order of their
    // columns: a warp has a run of them.
    const int run = (n + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32, i1 = min(n, (warp + 1) * run);
    int gt = 0, eq = 0;
    for (int i0 = warp * run; i0 < i1; i0 += 32) {
        const uint32_t key = i0 + lane < i1 ? keys[i0 + lane] : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i0 + lane < i1 && key > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i0 + lane < i1 && key == prefix));
    }
    if (lane == 0)
        sums[warp] = gt, sums[kSelWarps + warp] = eq;
    __syncthreads();
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? sums[kSelWarps + lane] : 0);
    const unsigned below = (1u << lane) - 1;
    for (int i0 = warp * run; i0 < i1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < i1 ? keys[i] : 0u;
        const bool more = i < i1 && key > prefix, same = i < i1 && key == prefix;
        const unsigned mg = __ballot_sync(0xffffffffu, more), me = __ballot_sync(0xffffffffu, same);
        const int ahead = gt + __popc(mg & below), e = eq + __popc(me & below);
        if (more || (same && e < want))
            out[p.first + ahead + min(e, want)] = table[i];
        gt += __popc(mg);
        eq += __popc(me);
    }
    // the first ones, and the last ones behind the n to choose from
    for (int i = threadIdx.x; i < p.first + p.last; i += kSelThreads)
        out[i < p.first ? i : i + choose] = table[i < p.first ? i - p.first : i - p.first + n];
}

template <int DIM>
cudaError_t launch(const SelectParams &p, int sms, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, k_block_select<DIM>, 226 * 1024);
    if (e != cudaSuccess)
        return e;
    // A CTA scores 128 pages in about 2 us: more are shared as far as the GPU has room for the CTAs at
    // once, and more than a thousand in any case, for their balance (32 rows of up to 4125 pages, 8 key heads, 60 us
    // with a CTA each and 47 with shares of a thousand).
    const int64_t units = int64_t(p.b.n_rows) * p.kv.heads;
    int c = 1;
    while (c < kMaxCluster && ((units * c * 2 <= kSelCtas * sms && p.n_cols / c > 128) || p.n_cols / c > 1024))
        c *= 2;
    const size_t heads8 = size_t((p.group + 7) & ~7);
    return start(k_block_select<DIM>, dim3(unsigned(units * c)), kSelThreads,
                 heads8 * (kQueryBytes<DIM> + 4) + (4 * kBins + size_t(p.n_cols)) * 4, c, stream, p, c);
}

}  // namespace

cudaError_t launch_kv_bounds(const BoundsParams &p, int sms, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    switch (p.kv.format) {
    case kKvBf16: return wide ? launch<128, kKvBf16>(p, sms, stream) : launch<64, kKvBf16>(p, sms, stream);
    case kKvInt8: return wide ? launch<128, kKvInt8>(p, sms, stream) : launch<64, kKvInt8>(p, sms, stream);
    default: return wide ? launch<128, kKvFp8>(p, sms, stream) : launch<64, kKvFp8>(p, sms, stream);
    }
}

cudaError_t launch_block_select(const SelectParams &p, int sms, cudaStream_t stream)
{
    return p.kv.dim == 128 ? launch<128>(p, sms, stream) : launch<64>(p, sms, stream);
}

}  // namespace lora
