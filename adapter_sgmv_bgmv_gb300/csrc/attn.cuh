// What the two attention kernels share: the spans of keys a tile of query rows reads,
// the even split of all spans over the CTAs, and the rule for rows with a result that
// is not finite.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv.cuh"
#include "ptx.cuh"

namespace lora {

// A unit is one tile of query rows of one (sequence, key head): the `group` query heads
// that share the key head, token by token, so rho = token * group + head in the group,
// rho in [r * ROWS, (r + 1) * ROWS).  It reads the keys [0, sink) and [lo, hi) in tiles
// of TOK keys: the window's union over its tokens and the first tokens ahead of it.
struct Span {
    int p0;                   // position of the tile's first token (may be negative)
    int lo, hi, sink;
    int n_sink, n;            // tiles of the first tokens, and in all (at least one)
};

template <int ROWS, int TOK>
__device__ __forceinline__ Span span_of(const SeqInfo &q, int r, int group, int window, int sinks)
{
    Span s;
    const int rho1 = min((r + 1) * ROWS, q.n_new * group) - 1;
    const int base = q.len - q.n_new;
    s.p0 = base + r * ROWS / group;
    const int p1 = base + rho1 / group;
    s.hi = max(p1 + 1, 0);
    s.lo = window ? min(max(s.p0 - window + 1, 0), s.hi) : 0;
    s.sink = min(sinks, s.lo);
    s.n_sink = (s.sink + TOK - 1) / TOK;
    s.n = max(1, s.n_sink + (s.hi - s.lo + TOK - 1) / TOK);
    return s;
}

__device__ __forceinline__ int row_tiles(int n_new, int group, int rows)
{
    return int((int64_t(n_new) * group + rows - 1) / rows);
}

// The even split.  All units, one after another (sequence, then row tile, then key head),
// are laid on a line: a unit is as long as its tiles and OV more, for what a unit costs
// besides them.  The line is cut into equal pieces, one per worker; a worker finds its own
// piece from the lengths in device memory, so no plan is made ahead and nothing is read on
// the host.  A piece [x0, x1) holds the tiles [x0 - at - OV, x1 - at - OV) of the unit at
// `at`, as far as it has them.  Only sequences with min_rows <= rows < max_rows (rows =
// new tokens * group) take part: the rest are another kernel's.
static __device__ __noinline__ int64_t wide_quotient(int64_t a, int64_t b) { return a / b; }

// a / b for a >= 0, b > 0; most of a launch's instructions run once, and a 64-bit division
// is a hundred of them to fetch.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((a | b) >> 31) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : wide_quotient(a, b);
}

struct Unit {
    int s, r, h;              // sequence, row tile, key head
    SeqInfo q;
};
struct Cursor : Unit {
    int64_t at;               // where the unit starts on the line
    Span span;
};

template <int ROWS, int TOK, int OV>
struct Split {
    static __device__ __forceinline__ bool mine(const AttnParams &p, const SeqInfo &q)
    {
        const int64_t rows = int64_t(q.n_new) * p.group;
        return rows >= p.min_rows && rows < p.max_rows;
    }

    // Sequence s's length on the line.  `longest` (in shared memory) is raised to the
    // mean length of its units.
    static __device__ int64_t cost(const AttnParams &p, int s, int *longest)
    {
        if (s >= p.b.n_seqs)
            return 0;
        const SeqInfo q = seq_info(p.b, s, blockIdx.x == 0 ? p.status : nullptr);
        if (!mine(p, q))
            return 0;
        int64_t n = 0;
        const int tiles = row_tiles(q.n_new, p.group, ROWS);
#pragma unroll 1
        for (int r = 0; r < tiles; ++r)
            n += span_of<ROWS, TOK>(q, r, p.group, p.window, p.sinks).n + OV;
        if (tiles)
            atomicMax(longest, int(quotient(n, tiles)));
        return n * p.kv.heads;
    }

    // Inclusive scan over the block; `sums` holds one entry per warp.
    template <int THREADS>
    static __device__ int64_t scan(int64_t v, int64_t *sums, int64_t &total)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        long long x = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d)
                x += y;
        }
        __syncthreads();
        if (lane == 31)
            sums[warp] = x;
        __syncthreads();
        int64_t before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp)
                before += sums[w];
            total += sums[w];
        }
        return before + x;
    }

    // The pieces of this CTA's N workers: worker i of CTA c has [(c * N + i) * piece, + piece)
    // cut at `total`; found[i].s is the sequence that holds its start and found[i].at where
    // that sequence begins, where the start is before `total`.  Every thread of the block
    // calls it, then locate() each worker.  `join_pace` is b / (N a) of the kernel (below).
    template <int THREADS, int N>
    static __device__ void find(const AttnParams &p, int64_t *sums, Cursor *found, int64_t &piece,
                                int64_t &total, int *longest, float join_pace)
    {
        const int tid = threadIdx.x;
        // Once over the sequences for the total, once more for the units (without a second
        // look where one round of the block's threads has all of them).
        int64_t c = 0, upto = 0, x0 = 0;
        total = 0;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            int64_t before = 0;
#pragma unroll 1
            for (int base = 0; base < p.b.n_seqs; base += THREADS) {
                int64_t t = 0;
                if (pass == 0 || p.b.n_seqs > THREADS) {
                    c = cost(p, base + tid, longest);
                    upto = before + scan<THREADS>(c, sums, t);
                    before += t;
                }
                if (pass == 0)
                    continue;
#pragma unroll 1
                for (int i = 0; i < N; ++i) {
                    const int64_t x = x0 + i * piece;
                    if (upto > x && upto - c <= x) {
                        found[i].s = base + tid;
                        found[i].at = upto - c;
                    }
                }
                if (p.b.n_seqs > THREADS && before >= x0 + N * piece)
                    break;
            }
            if (pass == 0) {
                total = before;
                const int64_t workers = int64_t(gridDim.x) * N;
                piece = quotient(total + workers - 1, workers);
                // A unit in many parts is soon read but long joined (by one CTA): pieces of k
                // tiles take k a, and the n / (k N) parts of `rows` rows b each to join; the sum is
                // least at k = sqrt(n rows b / (N a)).
                const float rows = float(min(int64_t(ROWS), int64_t(p.b.max_new) * p.group));
                piece = max(piece, int64_t(sqrtf(float(*longest) * rows * join_pace)));
                x0 = piece * N * blockIdx.x;
                if (x0 >= total)
                    return;
            }
        }
        __syncthreads();
    }

    // From the sequence that holds x to its unit that does.
    static __device__ __forceinline__ void locate(const AttnParams &p, int64_t x, Cursor &u)
    {
        u.q = seq_info(p.b, u.s, nullptr);
        u.r = 0;
#pragma unroll 1
        while (true) {
            u.span = span_of<ROWS, TOK>(u.q, u.r, p.group, p.window, p.sinks);
            const int64_t w = int64_t(u.span.n + OV) * p.kv.heads;
            if (u.at + w > x)
                break;
            u.at += w;
            ++u.r;
        }
        u.h = int(quotient(x - u.at, u.span.n + OV));
        u.at += int64_t(u.h) * (u.span.n + OV);
    }

    // The unit after `u` (the caller knows that there is one).
    static __device__ void next(const AttnParams &p, Cursor &u)
    {
        u.at += u.span.n + OV;
        if (++u.h < p.kv.heads)
            return;
        u.h = 0;
        ++u.r;
        if (u.r >= row_tiles(u.q.n_new, p.group, ROWS)) {
            u.r = 0;
            do {
                ++u.s;
                u.q = seq_info(p.b, u.s, nullptr);
            } while (!mine(p, u.q) && u.s + 1 < p.b.n_seqs);
        }
        u.span = span_of<ROWS, TOK>(u.q, u.r, p.group, p.window, p.sinks);
    }
};

// Where row `row` of unit u is: its token among the call's rows and the first column of
// its query head.
template <int ROWS, int DIM>
__device__ __forceinline__ void row_place(const AttnParams &p, const Unit &u, int row, int64_t &token,
                                          int64_t &col, int &pos)
{
    const int rho = u.r * ROWS + row, t = rho / p.group;
    token = u.q.start + t;
    col = int64_t(u.h * p.group + rho - t * p.group) * DIM;
    pos = u.q.len - u.q.n_new + t;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One row computed on its own, key by key, with no product for a key it does not see:
// for a row whose tile gave a result that is not finite.  There the keys other rows of
// the tile see may hold an infinity or a NaN, which a zero weight does not take out of
// the tile's product; here they are never multiplied.  `q` is the row's query, `pos` its
// position; a whole warp, lane l holds the DIM / 32 elements from l * DIM / 32; returns them in o.
// A chain of latencies (page, keys, sum over the warp, exponential): four keys take 2.4 us
// with eight warps of an SM at it.
template <int DIM, int FMT>
__device__ __noinline__ void careful_row(const AttnParams &p, const SeqInfo &s, int seq, int head, int pos,
                            const uint16_t *q, float o[DIM / 32])
{
    constexpr int N = DIM / 32;
    const int lane = threadIdx.x & 31;
    float qf[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        qf[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(q)[lane * N + e]);
        o[e] = 0.f;
    }
    constexpr int B = 4;                    // keys under way at once
#pragma unroll 1
    for (int j0 = 0; j0 <= pos; j0 += B) {
        if (p.window && j0 >= p.sinks && j0 <= pos - p.window)
            j0 = pos - p.window + 1;        // past what the window hides
        float kf[B][N], vf[B][N], dot[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int j = j0 + b;
            bool there = j <= pos && sees(pos, j, p.window, p.sinks);
            const int jp = there ? page_of(p.kv, j) : 0;
            const int page = there ? p.b.pages[int64_t(seq) * p.b.ld_pages + jp] : -1;
            there = page >= 0 && page < p.kv.n_pages;
            const int cell = j - jp * p.kv.page_size;
            const int64_t at = there ? page * p.kv.page_stride + cell * p.kv.cell_stride + head * p.kv.head_stride : 0;
            const int64_t sat = there ? page * p.kv.s_page + cell * p.kv.s_cell + head * p.kv.s_head : 0;
            const float ks = FMT == kKvBf16 ? 1.f : p.kv.k_scale[sat], vs = FMT == kKvBf16 ? 1.f : p.kv.v_scale[sat];
            dot[b] = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int d = lane * N + e;
                float x, y;
                if (FMT == kKvBf16) {
                    x = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.kv.k + at)[d]);
                    y = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.kv.v + at)[d]);
                } else if (FMT == kKvInt8) {
                    x = float(reinterpret_cast<const int8_t *>(p.kv.k + at)[d]) * ks;
                    y = float(reinterpret_cast<const int8_t *>(p.kv.v + at)[d]) * vs;
                } else {
                    x = float(reinterpret_cast<const __nv_fp8_e4m3 *>(p.kv.k + at)[d]) * ks;
                    y = float(reinterpret_cast<const __nv_fp8_e4m3 *>(p.kv.v + at)[d]) * vs;
                }
                kf[b][e] = there ? x : 0.f;
                vf[b][e] = there ? y : 0.f;
                dot[b] = fmaf(qf[e], kf[b][e], dot[b]);
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            dot[b] = warp_sum(dot[b]);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (j0 + b > pos || !sees(pos, j0 + b, p.window, p.sinks))
                continue;
            const float sc = dot[b] * p.scale;
            const float mn = fmaxf(m, sc), ref = mn == -INFINITY ? 0.f : mn;
            const float a = expf(m - ref), w = sc == INFINITY ? __int_as_float(0x7fffffff) : expf(sc - ref);
            m = mn;
            l = l * a + w;
#pragma unroll
            for (int e = 0; e < N; ++e)
                o[e] = o[e] * a + w * vf[b][e];
        }
        if (l != l)                         // every element is a NaN from here on
            break;
    }
    const float inv = l > 0.f ? 1.f / l : l;            // no key: 0; a NaN stays one
#pragma unroll
    for (int e = 0; e < N; ++e)
        o[e] = l == 0.f ? 0.f : o[e] * inv;
}

// Adds `n` partials (the i-th's row at o(i), its maximum and sum ml(i)) of one row in order;
// a whole warp, lane l the DIM / 32 elements from l * DIM / 32.
template <int DIM, int UNROLL, typename O, typename ML>
__device__ __forceinline__ void join(int n, O &&o, ML &&ml, float acc[DIM / 32], float &m, float &l)
{
    constexpr int N = DIM / 32;
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    l = 0.f;
    for (int i = lane; i < n; i += 32)
        m = fmaxf(m, ml(i).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int e = 0; e < N; ++e)
        acc[e] = 0.f;
#pragma unroll UNROLL
    for (int i = 0; i < n; ++i) {
        const float2 t = ml(i);
        const float a = exp2_fast(t.x - ref);
        float v[N];
        o(i, v);
        l += t.y * a;
#pragma unroll
        for (int e = 0; e < N; ++e)
            acc[e] = fmaf(a, v[e], acc[e]);
    }
}

template <int N>
__device__ __forceinline__ void load_vec(float v[N], const float *src)
{
    if (N == 4) {
        const float4 t = __ldcg(reinterpret_cast<const float4 *>(src));
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
        v[0] = t.x, v[1] = t.y;
    }
}

// The end of one row, by a whole warp: its sums o (lane l has the DIM / 32 elements from
// l * DIM / 32) over the sum of its weights l, as bf16.  Where that is not finite the row
// takes careful_row, which may walk a long context: at once, or LATER by a caller whom
// others wait for now.  Such a row is left as NaNs, which no finished one begins with, and
// true is returned.
template <int ROWS, int DIM, int FMT, bool LATER = false>
__device__ __noinline__ bool finish_row(const AttnParams &p, const Unit &u, int row,
                                        const float o[DIM / 32], float l)
{
    constexpr int N = DIM / 32;
    const int lane = threadIdx.x & 31;
    int64_t token, col;
    int pos;
    row_place<ROWS, DIM>(p, u, row, token, col, pos);
    float f[N];
    bool ok = true;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        f[e] = l == 0.f ? 0.f : o[e] / l;
        ok = ok && fabsf(f[e]) < INFINITY;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
        if (LATER) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                f[e] = __int_as_float(0x7fffffff);
        } else {
            careful_row<DIM, FMT>(p, u.q, u.s, u.h, pos, p.q + token * p.ldq + col, f);
        }
    }
    uint16_t *dst = p.out + token * p.ldo + col + lane * N;
    __nv_bfloat162 w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        w[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    if (N == 4)
        *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(w);
    else
        *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<uint32_t *>(w);
    return !ok;
}

}  // namespace lora
