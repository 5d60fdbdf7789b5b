// Attention of single rows over page lists of their own, one for each key head: what the choice of
// pages (blocks.cu) leaves of a long context.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - m),  m = the running maximum
//
// A unit is one row and key head: the group of query heads that share the key head, 8 or 16 at a
// time, over at most `blocks` pages, so units are of nearly one length and need no plan: each is a
// cluster of up to eight CTAs, every warp takes an equal run of its tiles of 16 keys (two of them at
// once in 8 bits), and the warps' parts are joined through the cluster's shared memory in the order
// of the warps.
//
// Keys and values go from memory to registers in the order in which the tensor cores take them;
// nothing is staged.  In S = Q K^T (m16n8k16, bf16 in, fp32 sums) the order of the head's elements
// is free as long as both sides have the same, so lane (g, c) takes 16-byte pieces of keys g and
// g + 8.  Its weights come out as the right operand of O^T += V^T W as it wants them: row g, keys 2c, 2c + 1
// and 8 more.  For the left one the lane takes the values of those four keys, 16-byte pieces again,
// and pairs neighbouring keys' elements by a byte permutation.  The next tile's keys are on their way
// while this one's weights are made, its values during the next one's scores; three CTAs a SM hide
// the rest.  Weights are taken as two bf16 terms (about 16 significant bits).
//
// 8-bit codes become bf16 in registers (exact); a key's scale multiplies its scores, a value's
// scale its weight.
//
// Bound: the bytes of the chosen pages in the end; now the chain of one tile (scores, maximum,
// weights, products: 2900 cycles for 16 keys in bf16, 3600 for 32 in 8 bits, with two or three warps on a
// scheduler), and where units are few that of start, tiles and joining.  Measured (dim 128): one row of 32
// pages of 64, 32 heads on 8, bf16 9.2 us; 39 rows of 128 pages of 16, 28 heads on 4, 31 us (164 MB, most
// of it from L2); 32 rows of 48 pages of 64, 64 heads on 8, int8 55 us, 3.8 TB/s, and
// with 128 heads on 8, 16 to a key head, 64 us (bf16 75).  The few-rows kernel over the first
// three's lists takes 16.7, 45 and 67 us.  Registers decide: int8 with three CTAs a SM instead of two, spilling 170
// bytes, 124 us; with one tile at once and six warps a CTA 57; bf16 with two CTAs a SM 40 us, with four 44.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn.cuh"
#include "launch.cuh"

namespace lora {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;               // with a lane for each warp's part
static_assert(kMaxCluster * kWarps <= 32);

__device__ __forceinline__ void mma(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// 16 (or 8) bytes that no other warp reads; zeros where they are not there.  In program order:
// the loads go out ahead of the arithmetic that follows them.
__device__ __forceinline__ uint4 load16(const uint8_t *src, bool there)
{
    uint4 x = make_uint4(0, 0, 0, 0);
    if (there)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(src) : "memory");
    return x;
}

__device__ __forceinline__ uint2 load8(const uint8_t *src, bool there)
{
    uint2 x = make_uint2(0, 0);
    if (there)
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(src) : "memory");
    return x;
}

__device__ __forceinline__ float4 ld_cluster(const float *local, int rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(map_cluster(smem_u32(local), uint32_t(rank))) : "memory");
    return v;
}

// Four codes (bytes b0..b3) to the bf16 pairs (b0, b2) and (b1, b3), times kCodeUnit.
template <int FMT>
__device__ __forceinline__ void widen(uint32_t r, uint32_t &even, uint32_t &odd)
{
    if (FMT == kKvInt8) {
        const uint32_t e = (r & 0x00ff00ffu) ^ 0x00800080u, o = ((r >> 8) & 0x00ff00ffu) ^ 0x00800080u;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(even) : "r"(e), "r"(0x7f007f00u), "r"(0xc000c000u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(odd) : "r"(o), "r"(0x7f007f00u), "r"(0xc000c000u));
    } else {
        const uint2 w = widen4<FMT>(__byte_perm(r, 0, 0x3120));      // b0 b2 b1 b3
        even = w.x;
        odd = w.y;
    }
}

// NR: groups of 8 query rows.  EVEN: pages of a multiple of 16 cells, so that a tile lies in one.
template <int DIM, int FMT, int NR>
struct Shape {
    static constexpr int ES = FMT == kKvBf16 ? 2 : 1;
    static constexpr int SUB = FMT == kKvBf16 ? 1 : 2;     // tiles of 16 keys at once
    static constexpr int KEYS = 16 * SUB;
    static constexpr int J = DIM * ES / 64;                // 16-byte pieces of a key a lane
    static constexpr int MT = DIM / 16;                    // 16-element tiles of values
    static constexpr int ROWS = 8 * NR;
    static constexpr int LD = DIM + 4;                     // floats of a part's row
    static constexpr int CTAS = NR == 1 && FMT == kKvBf16 ? 3 : 2;       // a SM
};

template <int DIM, int FMT, int NR, bool EVEN>
__global__ void __launch_bounds__(kThreads, Shape<DIM, FMT, NR>::CTAS) k_attn_blocks(const __grid_constant__ AttnParams p, int n_cta, int row_tiles)
{
    using S = Shape<DIM, FMT, NR>;
    constexpr int SUB = S::SUB, J = S::J, MT = S::MT, N = DIM / 32;
    constexpr bool kWide = FMT != kKvBf16;
    __shared__ __align__(16) float part[kWarps][S::ROWS * S::LD];
    __shared__ __align__(16) float4 part_ml[kWarps][S::ROWS];        // maximum and sum
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, g = lane >> 2, rank = int(cluster_ctarank());
    const KvView &kv = p.kv;
    int64_t work = int64_t(blockIdx.x) / n_cta;
    Unit u;
    u.r = int(work % row_tiles);
    work /= row_tiles;
    u.h = int(work % kv.heads);
    u.s = int(work / kv.heads);
    grid_dep_wait();
    grid_dep_launch();

    // The queries: element pairs of rows g and g + 8 in the order in which the keys' come.
    const int n_rows = min(S::ROWS, p.group - u.r * S::ROWS);
    uint4 qf[NR][DIM / 32];                                // two steps of 16 elements each
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = 8 * r + g;
        const uint16_t *src = p.q + u.s * p.ldq + int64_t(u.h * p.group + u.r * S::ROWS + min(row, n_rows - 1)) * DIM;
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j) {
            uint4 x;
            if (!kWide) {
                x = *reinterpret_cast<const uint4 *>(src + 32 * j + 8 * c);
            } else {
                // words w = 2 (j & 1) and the next of piece j / 2, four codes each
                const uint16_t *at = src + 64 * (j / 2) + 16 * c + 8 * (j & 1);
                const uint4 y = *reinterpret_cast<const uint4 *>(at);
                x = make_uint4(__byte_perm(y.x, y.y, 0x5410), __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x5410), __byte_perm(y.z, y.w, 0x7632));
            }
            qf[r][j] = row < n_rows ? x : make_uint4(0, 0, 0, 0);
        }
    }
    u.q = row_info(p.b, u.s, rank == 0 && u.h == 0 && u.r == 0 ? p.status : nullptr);
    if (u.q.n_new == 0)
        return;                                            // a row of no sequence; the whole cluster
    const int n = u.q.len;
    const int32_t *list = p.b.pages + int64_t(u.s) * p.b.ld_pages + u.h * p.b.head_pages;
    const uint8_t *kp = kv.k + u.h * kv.head_stride + c * 16;
    const uint8_t *vp = kv.v + u.h * kv.head_stride + g * (DIM == 128 || !kWide ? 16 : 8);
    const float *ksp = kWide ? kv.k_scale + u.h * kv.s_head : nullptr, *vsp = kWide ? kv.v_scale + u.h * kv.s_head : nullptr;

    // this warp's tiles
    const int tiles = (n + S::KEYS - 1) / S::KEYS, workers = n_cta * kWarps, w = rank * kWarps + warp;
    const int t0 = int(int64_t(tiles) * w / workers), t1 = int(int64_t(tiles) * (w + 1) / workers);

    // The lane's keys of a tile: g and g + 8 for the scores, 2c, 2c + 1, 8 + 2c, 9 + 2c for the values.
    auto key_of = [&](int i) { return i < 2 ? g + 8 * i : 2 * c + (i - 2 & 1) + (i >= 4 ? 8 : 0); };
    // Where the next tile's cells are, in bytes, and their scales.  A tile of a page of even size has
    // one place for all its cells; else each key's is looked up, and the scales' that the lane fetches.
    struct Place {
        bool there;
        int64_t at, s_at;
    };
    auto cell_place = [&](int j) {
        const int slot = page_of(kv, j);
        const int page = j < n ? list[slot] : -2;
        if (page != -2 && (page < 0 || page >= kv.n_pages))
            raise_status(p.status, kDevBadPage);
        const int cell = j - slot * kv.page_size;
        return Place{page >= 0 && page < kv.n_pages, page * kv.page_stride + cell * kv.cell_stride, page * kv.s_page + cell * kv.s_cell};
    };
    Place at[EVEN ? SUB : 6 * SUB], s_at;
    auto look_up = [&](int t) {
        const int j0 = t * S::KEYS;
        if (EVEN) {
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                const int j = j0 + 16 * b;
                // the next 16 cells of the same page, or another page
                if (t > t0 && j - page_of(kv, j) * kv.page_size >= S::KEYS) {
                    at[b].at += S::KEYS * kv.cell_stride;
                    at[b].s_at += S::KEYS * kv.s_cell;
                } else {
                    at[b] = cell_place(t < t1 ? j : n);
                }
            }
        } else {
#pragma unroll
            for (int b = 0; b < SUB; ++b)
#pragma unroll
                for (int i = 0; i < 6; ++i)
                    at[b * 6 + i] = cell_place(t < t1 ? j0 + 16 * b + key_of(i) : n);
            if (kWide)
                s_at = cell_place(t < t1 && lane < S::KEYS ? j0 + lane : n);
        }
    };
    const int64_t cs = kv.cell_stride;
    const int64_t k_first = EVEN ? g * cs : 0, v_first = EVEN ? 2 * c * cs : 0, s_first = lane % 16 * kv.s_cell;
    kp += k_first;
    vp += v_first;
    // key i of tile b: whether it is there, and its bytes from the first one's
    auto key_at = [&](int t, int b, int i, int64_t &off) {
        if (EVEN) {
            off = at[b].at + (i == 1 ? 8 * cs : i < 3 ? 0 : i == 3 ? cs : i == 4 ? 8 * cs : 9 * cs);
            return at[b].there && t * S::KEYS + 16 * b + key_of(i) < n;
        }
        off = at[EVEN ? 0 : b * 6 + i].at;
        return at[EVEN ? 0 : b * 6 + i].there;
    };
    uint4 kx[SUB][2][J];
    float ks, vs;                                          // of key `lane` of the tile
    auto load_scale = [&](int t, const float *scales) {
        float x = 0.f;
        const Place &pl = EVEN ? at[lane / 16 % SUB] : s_at;
        const int64_t off = EVEN ? (SUB == 2 && lane >= 16 ? at[SUB - 1].s_at : at[0].s_at) + s_first : s_at.s_at;
        const bool there = EVEN ? (SUB == 2 && lane >= 16 ? at[SUB - 1].there : at[0].there) && lane < S::KEYS && t * S::KEYS + lane < n : pl.there;
        if (there)
            asm volatile("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(scales + off) : "memory");
        return x;
    };
    auto load_k = [&](int t) {
        if (kWide)
            ks = load_scale(t, ksp);
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                int64_t off;
                const bool there = key_at(t, b, i, off);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    kx[b][i][j] = load16(kp + off + 64 * j, there);
            }
    };
    constexpr int VW = DIM * S::ES / 32;                   // words of a value a lane
    uint32_t vx[SUB][4][VW];
    auto load_v = [&](int t) {
        if (kWide)
            vs = load_scale(t, vsp);
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t off;
                const bool there = key_at(t, b, 2 + i, off);
                if (VW == 2) {
                    const uint2 x = load8(vp + off, there);
                    vx[b][i][0] = x.x, vx[b][i][1] = x.y;
                } else {
#pragma unroll
                    for (int j = 0; j < VW; j += 4) {
                        const uint4 x = load16(vp + off + 32 * j, there);
                        vx[b][i][j] = x.x, vx[b][i][j + 1 < VW ? j + 1 : 0] = x.y, vx[b][i][j + 2 < VW ? j + 2 : 0] = x.z, vx[b][i][j + 3 < VW ? j + 3 : 0] = x.w;
                    }
                }
            }
    };
    // the scale of key 16b + 8i + 2c + e of a tile
    auto scale_of = [&](float scales, int b, int i, int e) { return __shfl_sync(0xffffffffu, scales, 16 * b + 8 * i + 2 * c + e); };

    const float sl = p.scale * 1.4426950408889634f / kCodeUnit<FMT>;  // scores in powers of two
    float o[MT][NR][4], m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
            o[i][r][0] = o[i][r][1] = o[i][r][2] = o[i][r][3] = 0.f;
    }
    if (t0 < t1) {
        look_up(t0);
        load_k(t0);
        load_v(t0);
        look_up(t0 + 1);
    }
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
        // scores: row g (and g + 8), keys 2c, 2c + 1 and 8 more
        float s[SUB][2][4];
#pragma unroll
        for (int b = 0; b < SUB; ++b) {
            float s2[2][4] = {};                           // every other step's: half the chain
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[b][i][e] = 0.f;
#pragma unroll
            for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 y;
                    if (!kWide) {
                        y = kx[b][i][j];
                    } else {
                        const uint4 x = kx[b][i][j / 2];
                        widen<FMT>(j & 1 ? x.z : x.x, y.x, y.y);
                        widen<FMT>(j & 1 ? x.w : x.y, y.z, y.w);
                    }
                    const uint4 a = qf[0][j], a8 = NR == 2 ? qf[NR - 1][j] : make_uint4(0, 0, 0, 0);
                    mma(s[b][i], a.x, a8.x, a.y, a8.y, y.x, y.y);
                    mma(s2[i], a.z, a8.z, a.w, a8.w, y.z, y.w);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = kWide ? sl * scale_of(ks, b, i, e) : sl;
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        s[b][i][2 * r + e] = (s[b][i][2 * r + e] + s2[i][2 * r + e]) * f;
                }
        }
        if (t + 1 < t1)
            load_k(t + 1);
        if ((t + 1) * S::KEYS > n)
#pragma unroll
            for (int b = 0; b < SUB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t * S::KEYS + 16 * b + 8 * i + 2 * c + (e & 1) >= n)
                            s[b][i][e] = -INFINITY;
        float ref[NR], mx[NR];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            mx[r] = m[r];
#pragma unroll
            for (int b = 0; b < SUB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mx[r] = fmaxf(mx[r], fmaxf(s[b][i][2 * r], s[b][i][2 * r + 1]));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            ref[r] = mx[r] == -INFINITY ? 0.f : mx[r];
            moved = moved || mx[r] != m[r];
        }
        // most tiles of a long list leave every maximum as it was
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float a = exp2_fast(m[r] - ref[r]);
                m[r] = mx[r];
                l[r] *= a;
                // the sums' columns are rows 2c and 2c + 1
                const float a0 = __shfl_sync(0xffffffffu, a, 8 * c), a1 = __shfl_sync(0xffffffffu, a, 8 * c + 4);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][r][0] *= a0, o[i][r][1] *= a1;
                    o[i][r][2] *= a0, o[i][r][3] *= a1;
                }
            }
        }
        // weights, the right operand: row g, keys 2c, 2c + 1 and 8 more
        uint32_t hi[SUB][NR][2], lo[SUB][NR][2];
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float f[2] = {1.f, 1.f};
                if (kWide)
                    f[0] = scale_of(vs, b, i, 0) * (1.f / kCodeUnit<FMT>), f[1] = scale_of(vs, b, i, 1) * (1.f / kCodeUnit<FMT>);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float q[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = s[b][i][2 * r + e], v = exp2_fast(x - ref[r]);
                        l[r] += v;
                        // a key that is not seen has weight 0 whatever its scale is
                        q[e] = !kWide ? v : x == -INFINITY ? 0.f : v * f[e];
                    }
                    hi[b][r][i] = bf2(q[0], q[1]);
                    lo[b][r][i] = bf2(q[0] - __uint_as_float(hi[b][r][i] << 16), q[1] - __uint_as_float(hi[b][r][i] & 0xffff0000u));
                }
            }
        // o^T += v^T w: element tiles of 16, the lane's element i of its first half in row g, of its second in row g + 8
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
            for (int i = 0; i < MT; i += kWide ? 4 : 2) {
                if (!kWide) {
                    // a word has elements i and i + 1
                    const int w0 = i / 2, w1 = w0 + VW / 2;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t sel = e ? 0x7632 : 0x5410;
                        const uint32_t a0 = __byte_perm(vx[b][0][w0], vx[b][1][w0], sel), a1 = __byte_perm(vx[b][0][w1], vx[b][1][w1], sel);
                        const uint32_t a2 = __byte_perm(vx[b][2][w0], vx[b][3][w0], sel), a3 = __byte_perm(vx[b][2][w1], vx[b][3][w1], sel);
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            mma(o[i + e][r], a0, a1, a2, a3, hi[b][r][0], hi[b][r][1]);
                            mma(o[i + e][r], a0, a1, a2, a3, lo[b][r][0], lo[b][r][1]);
                        }
                    }
                } else {
                    // a word has elements i .. i + 3
                    const int w0 = i / 4, w1 = w0 + VW / 2;
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const uint32_t sel = e ? 0x7362 : 0x5140;
                        const uint2 a0 = widen4_unit<FMT>(__byte_perm(vx[b][0][w0], vx[b][1][w0], sel));
                        const uint2 a1 = widen4_unit<FMT>(__byte_perm(vx[b][0][w1], vx[b][1][w1], sel));
                        const uint2 a2 = widen4_unit<FMT>(__byte_perm(vx[b][2][w0], vx[b][3][w0], sel));
                        const uint2 a3 = widen4_unit<FMT>(__byte_perm(vx[b][2][w1], vx[b][3][w1], sel));
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            mma(o[i + e][r], a0.x, a1.x, a2.x, a3.x, hi[b][r][0], hi[b][r][1]);
                            mma(o[i + e][r], a0.x, a1.x, a2.x, a3.x, lo[b][r][0], lo[b][r][1]);
                            mma(o[i + e + 1][r], a0.y, a1.y, a2.y, a3.y, hi[b][r][0], hi[b][r][1]);
                            mma(o[i + e + 1][r], a0.y, a1.y, a2.y, a3.y, lo[b][r][0], lo[b][r][1]);
                        }
                    }
                }
            }
        if (t + 1 < t1) {
            load_v(t + 1);
            look_up(t + 2);
        }
    }

    // The warp's part: o[i][r][e] is row 8r + 2c + (e & 1) and the element that the lane's i-th (or, for
    // e >= 2, its i-th of the second half) stands for.
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (c == 0)
            part_ml[warp][8 * r + g] = make_float4(m[r], l[r], 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = kWide ? MT * 2 * g + i + (e >= 2 ? MT : 0) : DIM == 128 ? 8 * g + i + (e >= 2 ? 64 : 0) : 8 * g + i + (e >= 2 ? 4 : 0);
                part[warp][(8 * r + 2 * c + (e & 1)) * S::LD + d] = o[i][r][e];
            }
    }
    __syncwarp();
    if (n_cta > 1)
        cluster_sync();
    else
        __syncthreads();
    // Rows are dealt out to the cluster's warps.
#pragma unroll 1
    for (int row = w; row < n_rows; row += workers) {
        // lane i has the i-th part's maximum and sum
        float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        if (lane < workers)
            ml = n_cta > 1 ? ld_cluster(&part_ml[lane % kWarps][row].x, lane / kWarps) : part_ml[lane][row];
        float top = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float a = exp2_fast(ml.x - (top == -INFINITY ? 0.f : top));
        const float sum = warp_sum(a * ml.y);
        float f[N] = {};
        auto add = [&](int i, float4 v) {
            const float x = __shfl_sync(0xffffffffu, a, i);
            if (N == 4) {
                f[0] = fmaf(x, v.x, f[0]), f[1] = fmaf(x, v.y, f[1]);
                f[N - 2] = fmaf(x, v.z, f[N - 2]), f[N - 1] = fmaf(x, v.w, f[N - 1]);
            } else {
                f[0] = fmaf(x, lane & 1 ? v.z : v.x, f[0]), f[1] = fmaf(x, lane & 1 ? v.w : v.y, f[1]);
            }
        };
        const int piece = row * S::LD + (lane * N & ~3);
        if (n_cta == 1) {
#pragma unroll
            for (int i = 0; i < kWarps; ++i)
                add(i, *reinterpret_cast<const float4 *>(&part[i][piece]));
        } else {
            // eight parts' loads under way at once
#pragma unroll 1
            for (int i0 = 0; i0 < workers; i0 += 8) {
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = min(i0 + i, workers - 1);
                    v[i] = ld_cluster(&part[k % kWarps][piece], k / kWarps);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < workers)
                        add(i0 + i, v[i]);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;    // no key: zeros
        bool ok = true;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            f[e] *= inv;
            ok = ok && fabsf(f[e]) < INFINITY;
        }
        const int64_t col = int64_t(u.h * p.group + u.r * S::ROWS + row) * DIM;
        if (!__all_sync(0xffffffffu, ok))
            careful_row<DIM, FMT>(p, u.q, u.s, u.h, n - 1, p.q + u.s * p.ldq + col, f);
        uint16_t *dst = p.out + u.s * p.ldo + col + lane * N;
        if (N == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(bf2(f[0], f[1]), bf2(f[N - 2], f[N - 1]));
        else
            *reinterpret_cast<uint32_t *>(dst) = bf2(f[0], f[1]);
    }
    if (n_cta > 1) {
        __syncwarp();
        cluster_sync();                                    // others may still read this CTA's parts
    }
}

template <int DIM, int FMT, int NR>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream)
{
    using S = Shape<DIM, FMT, NR>;
    // CTAs of a unit: the fewest rounds of CTAs times what one takes, its tiles a warp and about
    // eight tiles' time for its start and the joining.
    const int row_tiles = (p.group + S::ROWS - 1) / S::ROWS;
    const int64_t units = int64_t(p.b.n_rows) * p.kv.heads * row_tiles, slots = int64_t(sms) * S::CTAS;
    const int tiles = (p.b.capacity + S::KEYS - 1) / S::KEYS;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int c = 1; c <= kMaxCluster; ++c) {
        const int64_t cost = (units * c + slots - 1) / slots * (8 + (tiles + c * kWarps - 1) / (c * kWarps));
        if (cost < least)
            least = cost, best = c;
    }
    const dim3 grid(unsigned(units * best));
    return p.kv.page_size % 16 == 0 ? start(k_attn_blocks<DIM, FMT, NR, true>, grid, kThreads, 0, best, stream, p, best, row_tiles)
                                    : start(k_attn_blocks<DIM, FMT, NR, false>, grid, kThreads, 0, best, stream, p, best, row_tiles);
}

template <int FMT>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    if (p.group <= 8)
        return wide ? launch<128, FMT, 1>(p, sms, stream) : launch<64, FMT, 1>(p, sms, stream);
    return wide ? launch<128, FMT, 2>(p, sms, stream) : launch<64, FMT, 2>(p, sms, stream);
}

}  // namespace

cudaError_t launch_attn_blocks(const AttnParams &p, int sms, cudaStream_t stream)
{
    switch (p.kv.format) {
    case kKvBf16: return launch<kKvBf16>(p, sms, stream);
    case kKvInt8: return launch<kKvInt8>(p, sms, stream);
    default: return launch<kKvFp8>(p, sms, stream);
    }
}

}  // namespace lora
