// Attention of a few new tokens over the paged cache: decode batches and short chunks.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - m),  m = the running maximum
//
// over the keys a row sees.  Every key and value is read from DRAM once per unit of 8 (or
// 16) query rows: the query heads that share a key head, and a few tokens.  At one new
// token the bytes of the cache bound it, and the arithmetic has to hide behind them: S^T = K Q^T
// and O^T += V^T W on m16n8k16 tensor-core products (bf16 in, fp32 sums) with the keys and
// the values' columns on the side of 16 and the query rows on the side of 8, so that a unit
// of at most 8 rows wastes nothing of a product on rows that are not there.  W^T comes out
// of the first product as the second one's operand but for a transposition within the
// warp (movmatrix).
//
// Layout.  All (sequence, key head, rows) units are cut into tiles of BT keys and laid
// on a line that is split evenly over the warps of the grid (attn.cuh).  A warp goes
// through its piece alone: its own ring of ST stages in shared memory, filled by 16-byte
// cp.async (any page size, any strides: each row of a stage has its own address), its own
// running maximum, sum and output.  A unit inside one piece goes straight to the output;
// the parts of one that crosses pieces are joined when the CTA's warps are done: first
// within the CTA in shared memory, then over CTAs by the one that arrives last, always in
// the order of the pieces, so the result does not depend on the order of arrival.
//
// 8-bit keys and values become bf16 in registers between ldmatrix and the product (every
// code is exact in bf16).  A key's scale multiplies its column of scores, a value's scale
// its weight.  The second product takes each weight as two bf16 terms (the rounded weight
// and what the rounding left), about 16 significant bits: the tensor cores have the time,
// and one bf16 term was measured to add up to a bf16 step to an output.
//
// Measured (dim 128): 64 sequences of 17 to 4095 keys, 32 key heads, bf16: 167 us, 6.0 TB/s,
// 0.90 of a copy's rate: the bytes.  128 sequences of 500 to 4001 keys, 64 query heads on 8 key
// heads, int8: 133 us, 3.5 TB/s: the instructions around each code.  One sequence of 777
// keys: 17 us, a chain of latencies (lengths, pages, keys, three levels of joining).
#include <cuda_runtime.h>

#include "attn.cuh"
#include "once.h"
#include "tc.cuh"

namespace lora {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnitCost = 3;   // a unit's start and end, in tiles
constexpr int kMaxRows = 16;   // of a unit
// 20 ns for a row of a part (eight parts' loads under way in four warps) to four times
// 0.6 us for a tile: see Split::find.
constexpr float kJoinPace = 8e-3f;
constexpr int kMaxCtas = 2;    // a SM

// NR: groups of 8 query rows of a unit.
template <int DIM, int FMT, int NR>
struct Shape {
    static constexpr int ROWS = 8 * NR;
    static constexpr int ES = FMT == kKvBf16 ? 2 : 1;
    static constexpr int RB = DIM * ES;                    // bytes of a key row
    static constexpr int CTAS = 2;
    static constexpr int BT = FMT == kKvBf16 && DIM == 128 ? 16 : 32;
    static constexpr int SCALES = FMT == kKvBf16 ? 0 : BT * 8;
    static constexpr int STAGE = 2 * BT * RB + SCALES;
    static constexpr int ST = 3;
    static constexpr int SMEM = kWarps * ST * STAGE + 128;
    static_assert(ST * STAGE >= ROWS * DIM * 4, "a warp's partial takes the place of its ring");
};

// Byte offset of 16-byte chunk c of row r: rows of RB bytes, chunks exchanged so that
// eight rows' same chunk lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t cell_at(uint32_t r, uint32_t c)
{
    if (RB >= 128)
        return r * RB + ((c ^ (r & 7u)) << 4);
    return r * RB + ((c ^ ((r >> 1) & 3u)) << 4);          // 64-byte rows: two share 128 bytes
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t r[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t r[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 block of bf16 held a row a four lanes, transposed.
__device__ __forceinline__ uint32_t flip(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Four codes (bytes b0..b3) to the bf16 pairs (b0, b2) and (b1, b3), times kCodeUnit.
template <int FMT>
__device__ __forceinline__ void widen(uint32_t r, uint32_t &even, uint32_t &odd)
{
    if (FMT == kKvInt8) {
        // code + 128 as a byte is a bf16 of (code + 128) 2^-133; times 2^127, less 2, it is
        // code 2^-6, exact, in one operation that does not load the integer pipe
        const uint32_t e = (r & 0x00ff00ffu) ^ 0x00800080u, o = ((r >> 8) & 0x00ff00ffu) ^ 0x00800080u;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(even) : "r"(e), "r"(0x7f007f00u), "r"(0xc000c000u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(odd) : "r"(o), "r"(0x7f007f00u), "r"(0xc000c000u));
    } else {
        const uint32_t s = __byte_perm(r, 0, 0x3120);      // b0 b2 b1 b3
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(s & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(s >> 16), __NV_E4M3);
        const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
        even = bf2(fa.x, fa.y);
        odd = bf2(fb.x, fb.y);
    }
}


// The order of partial results on the line: for each warp the unit it found begun and saw
// the end of (its head), then the unit its piece ended in (its tail).
struct Part {
    bool there, begins;       // begins: holds the unit's first tile
    int m_rows;
    Cursor u;
};

template <int DIM, int FMT, int NR>
__global__ void __launch_bounds__(kThreads, Shape<DIM, FMT, NR>::CTAS) k_attn_rows(const __grid_constant__ AttnParams p)
{
    using S = Shape<DIM, FMT, NR>;
    constexpr int kRows = S::ROWS;
    using Cut = Split<kRows, S::BT, kUnitCost>;
    constexpr int BT = S::BT, ST = S::ST, RB = S::RB, N = DIM / 32;
    constexpr int MT = BT / 16;                            // 16-key tiles of scores
    constexpr int KS = DIM / 16;                           // k-steps of q.k
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ int64_t sums[kWarps];
    __shared__ Cursor found[kWarps];
    __shared__ Part parts[2 * kWarps];
    __shared__ float2 tail_ml[kWarps][kMaxRows];
    __shared__ int last_flag, longest;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, g = lane >> 2;
    const KvView &kv = p.kv;
    const BatchView &b = p.b;

    if (!p.behind) {
        grid_dep_wait();
        grid_dep_launch();
    }

    int64_t piece, total;
    if (threadIdx.x == 0)
        longest = 0;
    __syncthreads();
    Cut::template find<kThreads, kWarps>(p, sums, found, piece, total, &longest, kJoinPace);
    const int64_t share = piece * kWarps;
    if (share * blockIdx.x >= total) {
        if (p.behind)
            grid_dep_wait();
        return;
    }
    const int worker = int(blockIdx.x) * kWarps + warp;
    int64_t x = worker * piece;
    const int64_t x1 = min(x + piece, total);
    uint8_t *mine = smem + warp * ST * S::STAGE;
    const uint32_t ring = smem_u32(mine);
    const float sl = p.scale * 1.4426950408889634f;        // scores in powers of two
    if (lane < 2)
        parts[2 * warp + lane].there = false;
    __syncwarp();

    Cursor u;
    if (x < x1) {
        u.s = found[warp].s;
        u.at = found[warp].at;
        Cut::locate(p, x, u);
    }
    while (x < x1) {
        const int64_t first = u.at + kUnitCost, end = first + u.span.n;
        const int t0 = int(max(x - first, int64_t(0)));
        const int t1 = int(max(min(x1, end) - first, int64_t(0)));
        x = end;
        if (t1 <= t0) {                                    // only the unit's own cost is here
            if (x < x1)
                Cut::next(p, u);
            continue;
        }
        const int n_rows = min(kRows, u.q.n_new * p.group - u.r * kRows);
        const int base = u.q.len - u.q.n_new;
        const uint8_t *kp = kv.k + u.h * kv.head_stride, *vp = kv.v + u.h * kv.head_stride;
        const int32_t *pages = b.pages + int64_t(u.s) * b.ld_pages;

        // first position of tile t's keys, and the end of the keys to read
        auto keys = [&](int t, int &j0, int &j1) {
            if (t < u.span.n_sink) {
                j0 = t * BT;
                j1 = u.span.sink;
            } else {
                j0 = u.span.lo + (t - u.span.n_sink) * BT;
                j1 = u.span.hi;
            }
        };
        auto page_at = [&](int t) -> int {                 // page id of this lane's key of tile t
            int j0, j1;
            keys(t, j0, j1);
            const int j = j0 + lane;
            if (t >= t1 || lane >= BT || j >= j1)
                return -1;
            const int page = pages[page_of(kv, j)];
            if (page < 0 || page >= kv.n_pages) {
                raise_status(p.status, kDevBadPage);
                return -1;
            }
            return page;
        };
        auto issue = [&](int t, int page) {                // copies of tile t into its stage
            if (t < t1) {
                int j0, j1;
                keys(t, j0, j1);
                const int cell = j0 + lane - page_of(kv, j0 + lane) * kv.page_size;
                const int64_t at = page < 0 ? -1 : page * kv.page_stride + cell * kv.cell_stride;
                const uint32_t st = ring + uint32_t(t % ST) * S::STAGE;
                constexpr int CH = RB / 16, RPI = 32 / CH; // chunks a row, rows an instruction
#pragma unroll
                for (int i = 0; i < BT / RPI; ++i) {
                    const int r = i * RPI + lane / CH, ch = lane % CH;
                    const int64_t a = __shfl_sync(0xffffffffu, (long long)at, r);
                    const uint32_t n = a < 0 ? 0u : 16u;
                    const int64_t off = a < 0 ? 0 : a + ch * 16;
                    tc::cp_async16(st + cell_at<RB>(r, ch), kp + off, n);
                    tc::cp_async16(st + BT * RB + cell_at<RB>(r, ch), vp + off, n);
                }
                if (FMT != kKvBf16 && lane < BT) {
                    const int64_t sa = page < 0 ? 0 : page * kv.s_page + cell * kv.s_cell + u.h * kv.s_head;
                    const uint32_t n = page < 0 ? 0u : 4u;
                    const uint32_t d = st + 2 * BT * RB + lane * 4;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(kv.k_scale + sa), "r"(n) : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + BT * 4), "l"(kv.v_scale + sa), "r"(n) : "memory");
                }
            }
            tc::cp_async_commit();
        };

        int page_next = page_at(t0);

        // The queries of rows 8r + g, as the products want them, and the positions of this
        // thread's rows of the scores, 8r + 2c and 8r + 2c + 1.
        int pos[NR][2];
        uint32_t qf[NR][KS][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * r + 2 * c + e;
                pos[r][e] = row < n_rows ? base + (u.r * kRows + row) / p.group : -1;
            }
            const int row = 8 * r + g;
            const bool on = row < n_rows;
            int64_t token, col;
            int unused;
            row_place<kRows, DIM>(p, u, on ? row : 0, token, col, unused);
            const uint16_t *src = p.q + token * p.ldq + col;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (FMT == kKvBf16) {
                    qf[r][k][0] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * c) : 0u;
                    qf[r][k][1] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 8 + 2 * c) : 0u;
                } else {
                    // the codes of d = 4c .. 4c + 3 arrive as pairs (0, 2) and (1, 3)
                    const uint2 w = on ? *reinterpret_cast<const uint2 *>(src + 16 * k + 4 * c) : make_uint2(0, 0);
                    qf[r][k][0] = __byte_perm(w.x, w.y, 0x5410);
                    qf[r][k][1] = __byte_perm(w.x, w.y, 0x7632);
                }
            }
        }
        float o[DIM / 16][NR][4], m[NR][2], l[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r][0] = m[r][1] = -INFINITY;
            l[r][0] = l[r][1] = 0.f;
#pragma unroll
            for (int i = 0; i < DIM / 16; ++i)
                o[i][r][0] = o[i][r][1] = o[i][r][2] = o[i][r][3] = 0.f;
        }

        // The first ST - 1 rounds only issue copies: one copy of that code.
#pragma unroll 1
        for (int t = t0 - (ST - 1); t < t1; ++t) {
            int j0 = 0, j1 = 0;
            if (t >= t0) {
                tc::cp_async_wait<ST - 2>();
                __syncwarp();
                keys(t, j0, j1);
            }
            if (j0 < j1) {
                const uint32_t st = ring + uint32_t(t % ST) * S::STAGE;
                // scores: this thread has keys 16i + g and 16i + g + 8, rows 8r + 2c and + 1
                float s[MT][NR][4];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float s2[NR][4];                       // every other step's: half the chain
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[i][r][e] = s2[r][e] = 0.f;
                    const uint32_t row = i * 16 + (lane & 15);
                    if (FMT == kKvBf16) {
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            uint32_t f[4];
                            ldsm4(st + cell_at<RB>(row, 2 * k + (lane >> 4)), f);
#pragma unroll
                            for (int r = 0; r < NR; ++r)
                                mma(k & 1 ? s2[r] : s[i][r], f, qf[r][k][0], qf[r][k][1]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < KS; k += 2) {  // two 16-element chunks
                            uint32_t f[4], a[2][4];
                            ldsm4(st + cell_at<RB>(row, k + (lane >> 4)), f);
                            widen<FMT>(f[0], a[0][0], a[0][2]);
                            widen<FMT>(f[1], a[0][1], a[0][3]);
                            widen<FMT>(f[2], a[1][0], a[1][2]);
                            widen<FMT>(f[3], a[1][1], a[1][3]);
#pragma unroll
                            for (int r = 0; r < NR; ++r) {
                                mma(s[i][r], a[0], qf[r][k][0], qf[r][k][1]);
                                mma(s2[r], a[1], qf[r][k + 1][0], qf[r][k + 1][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[i][r][e] += s2[r][e];
                }
                // scale, mask, running maximum
                const float *sc = reinterpret_cast<const float *>(mine + (t % ST) * S::STAGE + 2 * BT * RB);
                const int je = min(j0 + BT, j1);
                const bool all = je - 1 <= u.span.p0 && je - j0 == BT &&
                                 (p.window == 0 || t < u.span.n_sink || j0 > base + (u.r * kRows + n_rows - 1) / p.group - p.window);
                float mx[NR][2];
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    mx[r][0] = m[r][0], mx[r][1] = m[r][1];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = 16 * i + 8 * h + g, j = j0 + k;
                        const float ks = FMT == kKvBf16 ? sl : sl / kCodeUnit<FMT> * sc[k];
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float v = s[i][r][2 * h + e] * ks;
                                if (!all && (j >= j1 || !sees(pos[r][e], j, p.window, p.sinks)))
                                    v = -INFINITY;
                                s[i][r][2 * h + e] = v;
                                mx[r][e] = fmaxf(mx[r][e], v);
                            }
                    }
                float ref[NR][2];
                bool moved = false;
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            mx[r][e] = fmaxf(mx[r][e], __shfl_xor_sync(0xffffffffu, mx[r][e], d));
                        ref[r][e] = mx[r][e] == -INFINITY ? 0.f : mx[r][e];
                        moved = moved || mx[r][e] != m[r][e];
                    }
                // most tiles of a long sequence leave every maximum as it was
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float a = exp2_fast(m[r][e] - ref[r][e]);
                            m[r][e] = mx[r][e];
                            l[r][e] *= a;
#pragma unroll
                            for (int d = 0; d < DIM / 16; ++d) {
                                o[d][r][e] *= a;
                                o[d][r][2 + e] *= a;
                            }
                        }
                }
                // weights, as the right operand of the second product
                uint32_t w[MT][NR][2], wl[MT][NR][2];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float vs = FMT == kKvBf16 ? 1.f : sc[BT + 16 * i + 8 * h + g] / kCodeUnit<FMT>;
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            float q[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = s[i][r][2 * h + e], v = exp2_fast(x - ref[r][e]);
                                l[r][e] += v;
                                // a key that is not seen has weight 0 whatever its scale is
                                q[e] = FMT == kKvBf16 ? v : x == -INFINITY ? 0.f : v * vs;
                            }
                            const uint32_t hi = bf2(q[0], q[1]);
                            w[i][r][h] = flip(hi);
                            wl[i][r][h] = flip(bf2(q[0] - __uint_as_float(hi << 16), q[1] - __uint_as_float(hi & 0xffff0000u)));
                        }
                    }
                // o^T += v^T w: this thread has columns of v (d) and rows 8r + 2c, + 1
                const uint32_t sv = st + BT * RB;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (FMT == kKvBf16) {
                        const uint32_t row = i * 16 + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                        for (int d = 0; d < DIM / 16; ++d) {
                            uint32_t f[4];
                            ldsm4t(sv + cell_at<RB>(row, 2 * d + (lane >> 3 & 1)), f);
#pragma unroll
                            for (int r = 0; r < NR; ++r) {
                                mma(o[d][r], f, w[i][r][0], w[i][r][1]);
                                mma(o[d][r], f, wl[i][r][0], wl[i][r][1]);
                            }
                        }
                    } else {
                        const uint32_t row = i * 16 + (lane & 15);
#pragma unroll
                        for (int d = 0; d < DIM / 16; d += 2) {   // 16-element chunks d, d + 1
                            uint32_t f[4], a[2][4];
                            ldsm4t(sv + cell_at<RB>(row, d + (lane >> 4)), f);
                            widen<FMT>(f[0], a[0][0], a[0][1]);
                            widen<FMT>(f[1], a[0][2], a[0][3]);
                            widen<FMT>(f[2], a[1][0], a[1][1]);
                            widen<FMT>(f[3], a[1][2], a[1][3]);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int r = 0; r < NR; ++r) {
                                    mma(o[d + e][r], a[e], w[i][r][0], w[i][r][1]);
                                    mma(o[d + e][r], a[e], wl[i][r][0], wl[i][r][1]);
                                }
                        }
                    }
                }
            }
            __syncwarp();
            const int ahead = page_at(t + ST);             // on its way during the next round
            issue(t + ST - 1, page_next);
            page_next = ahead;
        }
        tc::cp_async_wait<0>();
        __syncwarp();
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], d);

        // Where the rows go: the unit's end, or a partial.  o[i][r][e] is row 8r + 2c + (e & 1)
        // and element d = 16i + g + 8 (e / 2) for bf16 pools, 16i + 2g + e / 2 for 8-bit ones
        // (their chunks come apart into even and odd elements).
        const bool begins = t0 == 0, ends = t1 == u.span.n;
        const bool head = ends && !begins;
        float *dst = head ? p.part.warp_o + int64_t(worker) * kMaxRows * DIM : reinterpret_cast<float *>(mine);
        float2 *dml = head ? p.part.warp_ml + int64_t(worker) * kMaxRows : tail_ml[warp];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * r + 2 * c + e;
                if (row >= n_rows)
                    continue;
                if (g == 0)
                    dml[row] = make_float2(m[r][e], l[r][e]);
#pragma unroll
                for (int i = 0; i < DIM / 16; ++i) {
                    float *at = dst + row * DIM + 16 * i;
                    if (FMT == kKvBf16) {
                        at[g] = o[i][r][e];
                        at[g + 8] = o[i][r][2 + e];
                    } else {
                        *reinterpret_cast<float2 *>(at + 2 * g) = make_float2(o[i][r][e], o[i][r][2 + e]);
                    }
                }
            }
        __syncwarp();
        if (begins && ends) {
#pragma unroll 1
            for (int row = 0; row < n_rows; ++row) {
                float f[N];
#pragma unroll
                for (int e = 0; e < N; ++e)
                    f[e] = dst[row * DIM + lane * N + e];
                finish_row<kRows, DIM, FMT>(p, u, row, f, dml[row].y);
            }
            __syncwarp();                                  // the ring is free again
        } else if (lane == 0) {
            Part &pt = parts[2 * warp + (head ? 0 : 1)];
            pt.there = true;
            pt.begins = begins;
            pt.m_rows = n_rows;
            pt.u = u;
        }
        if (x < x1)
            Cut::next(p, u);
    }

    // Units that crossed the warps of this CTA: runs of `parts` with the same unit.  Each
    // run is one warp's; those that reach beyond the CTA become its partials.
    __threadfence_block();
    __syncthreads();
    int cross[2] = {-1, -1};                               // parts of the runs that came in / go on
    int run = 0;
#pragma unroll 1
    for (int i = 0; i < 2 * kWarps;) {
        if (!parts[i].there) {
            ++i;
            continue;
        }
        const int64_t at = parts[i].u.at;
        int idx[2 * kWarps], n = 0, j = i;
#pragma unroll 1
        for (; j < 2 * kWarps; ++j) {
            if (!parts[j].there)
                continue;
            if (parts[j].u.at != at)
                break;
            idx[n++] = j;
        }
        const bool begins = parts[i].begins, ends = (idx[n - 1] & 1) == 0;
        if (!begins)
            cross[0] = i;
        else if (!ends)
            cross[1] = i;
        if (run++ % kWarps == warp) {
#pragma unroll 1
            for (int row = 0; row < parts[i].m_rows; ++row) {
                float acc[N], m, l;
                auto ml = [&](int k) {
                    const int w = idx[k] >> 1;
                    return (idx[k] & 1) ? tail_ml[w][row] : __ldcg(&p.part.warp_ml[(int64_t(blockIdx.x) * kWarps + w) * kMaxRows + row]);
                };
                auto o = [&](int k, float *v) {
                    const int w = idx[k] >> 1;
                    if (idx[k] & 1) {
                        const float *src = reinterpret_cast<const float *>(smem + w * ST * S::STAGE) + row * DIM + lane * N;
#pragma unroll
                        for (int e = 0; e < N; ++e)
                            v[e] = src[e];
                    } else {
                        load_vec<N>(v, p.part.warp_o + ((int64_t(blockIdx.x) * kWarps + w) * kMaxRows + row) * DIM + lane * N);
                    }
                };
                join<DIM, 2>(n, o, ml, acc, m, l);
                if (begins && ends) {
                    finish_row<kRows, DIM, FMT>(p, parts[i].u, row, acc, l);
                } else {
                    const int64_t at2 = (int64_t(blockIdx.x) * 2 + begins) * kMaxRows + row;
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        p.part.cta_o[at2 * DIM + lane * N + e] = acc[e];
                    if (lane == 0)
                        p.part.cta_ml[at2] = make_float2(m, l);
                }
            }
        }
        i = j;
    }
    // Units that cross CTAs: the last to arrive adds the CTAs' partials, all its warps.
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (cross[k] < 0)
            continue;
        const Part &pt = parts[cross[k]];
        const int64_t first = quotient(pt.u.at + kUnitCost, share), final_ = quotient(pt.u.at + kUnitCost + pt.u.span.n - 1, share);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            last_flag = atomicAdd(&p.part.arrived[first], 1) == int(final_ - first);
            if (last_flag)
                p.part.arrived[first] = 0;
        }
        __syncthreads();
        if (!last_flag)
            continue;
        __threadfence();
#pragma unroll 1
        for (int row = warp; row < pt.m_rows; row += kWarps) {
            float acc[N], m, l;
            auto at = [&](int i) { return ((first + i) * 2 + (i == 0)) * kMaxRows + row; };
            join<DIM, 8>(int(final_ - first) + 1,
                      [&](int i, float *v) { load_vec<N>(v, p.part.cta_o + at(i) * DIM + lane * N); },
                      [&](int i) { return __ldcg(&p.part.cta_ml[at(i)]); }, acc, m, l);
            finish_row<kRows, DIM, FMT>(p, pt.u, row, acc, l);
        }
    }
    // whoever comes next may take this kernel's end for the whole call's
    if (p.behind)
        grid_dep_wait();
}

template <int DIM, int FMT, int NR>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream)
{
    using S = Shape<DIM, FMT, NR>;
    static OncePerDevice once;
    const cudaError_t e = once([] {
        return cudaFuncSetAttribute(k_attn_rows<DIM, FMT, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    });
    if (e != cudaSuccess)
        return e;
    static_assert(S::CTAS <= kMaxCtas, "the scratch has room for every CTA");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(S::CTAS * sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_rows<DIM, FMT, NR>, p);
}

// Units of 8 rows where no sequence can have more; else of 16.
template <int FMT>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    if (int64_t(p.b.max_new) * p.group <= 8)
        return wide ? launch<128, FMT, 1>(p, sms, stream) : launch<64, FMT, 1>(p, sms, stream);
    return wide ? launch<128, FMT, 2>(p, sms, stream) : launch<64, FMT, 2>(p, sms, stream);
}

}  // namespace

size_t attn_rows_scratch(uint8_t *base, int sms, AttnScratch *s)
{
    const size_t ctas = size_t(sms) * kMaxCtas, warps = ctas * kWarps;
    const size_t row = 128 * sizeof(float);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *p = base + at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    AttnScratch t;
    t.cta_o = reinterpret_cast<float *>(take(ctas * 2 * kMaxRows * row));
    t.cta_ml = reinterpret_cast<float2 *>(take(ctas * 2 * kMaxRows * sizeof(float2)));
    t.warp_o = reinterpret_cast<float *>(take(warps * kMaxRows * row));
    t.warp_ml = reinterpret_cast<float2 *>(take(warps * kMaxRows * sizeof(float2)));
    t.arrived = reinterpret_cast<int *>(take(ctas * sizeof(int)));
    if (s)
        *s = t;
    return at;
}

cudaError_t launch_attn_rows(const AttnParams &p, int sms, cudaStream_t stream)
{
    switch (p.kv.format) {
    case kKvBf16: return launch<kKvBf16>(p, sms, stream);
    case kKvInt8: return launch<kKvInt8>(p, sms, stream);
    default: return launch<kKvFp8>(p, sms, stream);
    }
}

}  // namespace lora
