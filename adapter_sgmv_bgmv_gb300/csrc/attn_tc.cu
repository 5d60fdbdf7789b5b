// Attention of many new tokens over the paged cache: prefill, and chunks of a prompt.
//
// The same sums as in attn_rows.cu, with the products on the tensor cores at full width.
// A unit is 256 query rows (two tiles A and B of 128) of one (sequence, key head); it goes
// through its keys in tiles of 128.  Per key tile and row tile, two products of
// 128 x 128 x dim: S = Q K^T, then O += W V with W = exp2(S - reference).  Two products of
// 128^3 take 1024 cycles of the tensor cores an SM has, and W takes 128 exponentials a row:
// both row tiles share every key tile, and while one is at its weights the tensor cores
// work for the other.
//
//   warps 0-3, 4-7   weights of tile A / B: one thread a row, S read from TMEM, W written
//                    back over it as bf16 (the left operand of the second product).  The
//                    reference is the running maximum, but it is moved (and O rescaled in
//                    TMEM) only when the maximum passes it by 2^8: weights stay below 2^8,
//                    and the sums are divided out at the end all the same.
//   then 4 or 8      loads: cells of the pages to 128-byte-swizzled tiles, each row with its
//                    own address (any page size, any strides); bf16 by cp.async, 8-bit codes
//                    through registers, where they become bf16 (exact).
//   then two         one thread each issues the products of tile A / B: an issue holds its
//                    thread until the tensor cores have taken it, so with one thread for both
//                    they stood still while it waited for barriers (2 400 of 5 400 cycles a
//                    key tile).  The two take turns: left to themselves the tiles fall into
//                    step, both at their weights and then both at their products.
//   then one         one thread goes along the CTA's piece ahead of the others and leaves
//                    them what they need of each unit (the only copy of that code: see below
//                    on code size).
//
// TMEM (512 columns): S of A and B (128 each, W in their first half), O of A and B (dim).
// The products of one thread run in the order of their issue, so the next S may be issued
// behind the second product that reads the weights it will overwrite.
// Shared memory (dim 128): Q 64 KB, a ring of four 32 KB tiles (keys, values by turns).
//
// The units lie on a line that is split evenly over one CTA per SM (attn.cuh), each CTA
// going through its piece without a break: the loads of the next unit run while the
// last one ends.  A unit cut by the ends of pieces leaves its parts in scratch, and the CTA
// that arrives last joins them in the order of the CTAs.
//
// Rows whose result is not finite (attn.cuh) are only marked on the way, and redone when the
// piece is done: each walks its whole context again, and the other roles' waits are bounded.
//
// Code size.  The four kinds of warps run different programs on one instruction cache: with
// bodies unrolled to a thousand instructions each waited longer for instructions than for
// anything else (1909 -> 592 us for the 8191-token prompt below went with short loops, one
// copy of each, and one warp for what all need to know of a unit).
//
// Measured (bf16, dim 128, 32 query heads on 8 key heads, one 8191-token prompt in pages of
// one token): 555 us, 0.99 PFLOP/s, 0.52 of a cuBLAS bf16 product's rate; what bounds it is the
// chain of one row tile (scores, maximum, weights, products: 4,200 cycles for 1,024 of
// products), of which two run side by side.  16 prompts of 1056 tokens, a key head for each
// query head: 325 us, 0.45 PFLOP/s; a unit there is nine key tiles long at most, and its start
// and end take as long as three.
#include <cuda_runtime.h>

#include <climits>

#include "attn.cuh"
#include "once.h"
#include "tc.cuh"

namespace lora {

namespace {

constexpr int kM = 128;              // rows of a row tile
constexpr int kRows = 2 * kM;
constexpr int kKeys = 128;           // keys of a key tile
constexpr int kUnitCost = 2;         // a unit's start and end, in key tiles
constexpr int kScaleSlots = 4;
// 5 ns for a row of a part (loads of four rows of four parts under way in eight warps) to
// 2.5 us for a key tile: see Split::find.
constexpr float kJoinPace = 2e-3f;
// Warps: 8 of the weights, LOADS of the loads (8-bit codes pass through their registers:
// twice as many), two of the products, one of the parts, one there for its registers, of
// which these two kinds give some to the weights.
template <int FMT>
struct Crew {
    static constexpr int LOADS = FMT == kKvBf16 ? 4 : 8;
    static constexpr int ROWS = 128 / LOADS;             // of a tile, for a load warp
    static constexpr int WARPS = 12 + LOADS;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int launch = FMT == kKvBf16 ? 128 : 96;
    static constexpr int more = FMT == kKvBf16 ? 152 : 144, load = FMT == kKvBf16 ? 120 : 64, few = FMT == kKvBf16 ? 88 : 64;
    static_assert(8 * more + LOADS * load + 4 * few == WARPS * launch, "the registers of the block");
};

template <int DIM>
struct TcShape {
    static constexpr int HALVES = DIM / 64;
    static constexpr uint32_t HALF = 128 * 128;              // 128 rows x 64 elements
    static constexpr uint32_t TILE = HALVES * HALF;
    static constexpr int STAGES = DIM == 128 ? 4 : 6;
    static constexpr uint32_t RING = 2 * TILE;               // after the two Q tiles
    static constexpr uint32_t SCALES = RING + STAGES * TILE; // [slot][k, v][128] floats
    static constexpr uint32_t BARS = SCALES + kScaleSlots * 2 * kKeys * 4;
    static constexpr uint32_t BYTES = BARS + 512;
    static constexpr uint32_t SMEM = BYTES + 1024;
};

// Barriers, 8 bytes each from BARS.
enum Bar : uint32_t {
    kFull = 0, kEmpty = 8, kQFull = 16, kQEmpty = 18, kSFull = 20, kPvDone = 24,
    kPartFull = 26, kPartEmpty = 30, kJoin = 34, kTurn = 35,
    kWReady = 37                  // of A's first and second half of the keys, then B's
};

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t r[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16_raw(uint32_t a, uint32_t r[16])
{
    float v[16];
    tc::tmem_ld16(a, v);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        r[i] = __float_as_uint(v[i]);
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Bounded wait of a role: after one that ran out (here or in another warp) every wait of
// the block gives up at once, and the roles leave their loops.
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, volatile int *dead, unsigned *status, unsigned code)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (!*dead) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            raise_status(status, code);
            *dead = 1;
        }
    }
    return false;
}

// One row tile of a unit: its rows, and the positions of its first and last token.
struct Side {
    int rows, p_first, p_last;
};

__device__ __forceinline__ Side side_of(const AttnParams &p, const Unit &u, int tile)
{
    Side s;
    const int rho = u.r * kRows + tile * kM, all = u.q.n_new * p.group;
    s.rows = max(0, min(kM, all - rho));
    const int base = u.q.len - u.q.n_new;
    s.p_first = base + rho / p.group;
    s.p_last = base + (rho + max(s.rows, 1) - 1) / p.group;
    return s;
}

// The key tiles in which any row of a row tile sees a key: those before `behind` and from
// `from` on, short of `to`.  The products of the others are left out.
struct Active {
    int from, to, behind;
    __device__ __forceinline__ bool operator()(int t) const { return t < to && (t >= from || t < behind); }
};

__device__ __forceinline__ Active active(const AttnParams &p, const Cursor &u, const Side &s)
{
    const Span &k = u.span;
    Active a{0, 0, 0};
    if (s.rows == 0 || s.p_last < 0)
        return a;
    a.to = k.n_sink + (s.p_last >= k.lo ? (s.p_last - k.lo) / kKeys + 1 : 0);
    if (p.window) {
        a.from = k.n_sink + max(0, s.p_first - p.window + 1 - k.lo) / kKeys;
        a.behind = k.n_sink + (p.sinks > k.lo ? (p.sinks - k.lo + kKeys - 1) / kKeys : 0);
    }
    return a;
}

// What a CTA has of one unit: key tiles [t0, t1), of which the first n_sink hold the first
// tokens, [0, sink), and the others [lo, hi).
struct Part : Unit {
    int t0, t1, n_sink, lo, hi, sink;
    int more;                 // 0: past the last part
    int begins, ends;         // holds the unit's first / last tile
    int first, last;          // the CTAs that have parts of the unit
    Side side[2];
    Active act[2];
};
constexpr int kParts = 4;     // parts under way at once

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// The two passes over this thread's row of S (128 columns from tS), 32 columns at a time and
// in short loops: the warps of a CTA run four different programs, and straight code of a
// thousand instructions for each was measured to wait for instruction fetches most of
// the time.  SCALED: times the keys' scales ks (in shared memory, the same for every row).

template <bool SCALED>
__device__ __forceinline__ float maximum(uint32_t tS, const float *ks)
{
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    uint32_t r[64];
    tc::tmem_ld32_nowait(tS, r);
    tc::tmem_wait_ld();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // the other half's columns are on their way during this half's
            if (b == 0 || h == 0)
                tc::tmem_ld32_nowait(tS + 64 * h + 32 * b + 32, r + 32 * (1 - b));
            float *s = reinterpret_cast<float *>(r + 32 * b);
            if (SCALED) {
                const float4 *k4 = reinterpret_cast<const float4 *>(ks + 64 * h + 32 * b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 k = k4[i];
                    const float2 x = mul2(make_float2(s[4 * i], s[4 * i + 1]), make_float2(k.x, k.y));
                    const float2 y = mul2(make_float2(s[4 * i + 2], s[4 * i + 3]), make_float2(k.z, k.w));
                    mx[0] = max3(mx[0], x.x, x.y);
                    mx[1] = max3(mx[1], y.x, y.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = max3(mx[e], s[i + e], s[i + e + 4]);
            }
            tc::tmem_wait_ld();
        }
    }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// The weights exp2(s * f - m), written as bf16 (times the values' scales, ks + kKeys) over
// the columns of S they came from; returns their sum.  Each half of the keys is handed
// over as it is written (`ready`, and the next barrier), so that the products with the
// first half run during the second.
template <int FMT, bool SCALED>
__device__ __forceinline__ float weights(uint32_t tS, const float *ks, float f, float m, uint32_t ready)
{
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 ff = make_float2(f, f), less = make_float2(-m, -m);
    uint32_t r[64];
    tc::tmem_ld32_nowait(tS, r);
    tc::tmem_wait_ld();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (b == 0 || h == 0)
                tc::tmem_ld32_nowait(tS + 64 * h + 32 * b + 32, r + 32 * (1 - b));
            const float *s = reinterpret_cast<const float *>(r + 32 * b);
            const float4 *k4 = reinterpret_cast<const float4 *>(ks + 64 * h + 32 * b);
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float2 k0 = ff, k1 = ff;
                if (SCALED) {
                    const float4 k = k4[i];
                    k0 = make_float2(k.x, k.y), k1 = make_float2(k.z, k.w);
                }
                float2 x = fma2(make_float2(s[4 * i], s[4 * i + 1]), k0, less);
                float2 y = fma2(make_float2(s[4 * i + 2], s[4 * i + 3]), k1, less);
                x.x = exp2_fast(x.x), x.y = exp2_fast(x.y), y.x = exp2_fast(y.x), y.y = exp2_fast(y.y);
                sum[0] = add2(sum[0], x);
                sum[1] = add2(sum[1], y);
                if (FMT != kKvBf16) {
                    const float4 v = k4[kKeys / 4 + i];
                    x = mul2(x, make_float2(v.x, v.y));
                    y = mul2(y, make_float2(v.z, v.w));
                }
                pk[2 * i] = pack2(x.x, x.y);
                pk[2 * i + 1] = pack2(y.x, y.y);
            }
            tc::tmem_wait_ld();
            tmem_st16(tS + 32 * h + 16 * b, pk);
        }
        tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(ready + 8 * h);
    }
    return (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
}

// Joins the parts that the CTAs [first, last] left of unit u's rows, by the eight warps of
// the weights; true in a warp that left a row to redo_rows.
template <int DIM, int FMT>
__device__ __noinline__ bool join_unit(const AttnParams &p, const Part &u)
{
    bool odd = false;
    constexpr int N = DIM / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_rows = min(kRows, u.q.n_new * p.group - u.r * kRows), n = u.last - u.first + 1;
    auto at = [&](int i, int row) { return int64_t((u.first + i) * 2 + (i == 0)) * kRows + min(row, n_rows - 1); };
    // four rows at a time: one by one, the loads' latency was most of a short chunk's time
    constexpr int B = 4;
#pragma unroll 1
    for (int row = warp * B; row < n_rows; row += 8 * B) {
        float acc[B][N], m[B], l[B];
#pragma unroll
        for (int r = 0; r < B; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e)
                acc[r][e] = 0.f;
        }
        for (int i = lane; i < n; i += 32)
#pragma unroll
            for (int r = 0; r < B; ++r)
                m[r] = fmaxf(m[r], __ldcg(&p.part.cta_ml[at(i, row + r)]).x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1)
#pragma unroll
            for (int r = 0; r < B; ++r)
                m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], k));
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            float2 t[B];
            float v[B][N];
#pragma unroll
            for (int r = 0; r < B; ++r) {
                t[r] = __ldcg(&p.part.cta_ml[at(i, row + r)]);
                load_vec<N>(v[r], p.part.cta_o + at(i, row + r) * DIM + lane * N);
            }
#pragma unroll
            for (int r = 0; r < B; ++r) {
                const float a = exp2_fast(t[r].x - (m[r] == -INFINITY ? 0.f : m[r]));
                l[r] += t[r].y * a;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    acc[r][e] = fmaf(a, v[r][e], acc[r][e]);
            }
        }
#pragma unroll
        for (int r = 0; r < B; ++r)
            if (row + r < n_rows)
                odd |= finish_row<kRows, DIM, FMT, true>(p, u, row + r, acc[r], l[r]);
    }
    return odd;
}

// A CTA's piece [x, x1) and what it ended of it, for redo_rows.
struct Piece {
    int64_t x, x1;
    int64_t at;               // where the sequence that holds x, s, begins
    int s;
    int odd;                  // some row was left
    int joined;               // units cut by the piece's ends that were joined here: bit 1 the
                              // one that begins in the piece, bit 0 the one that does not
};

// The rows whose result was not finite, each on its own.  They may take seconds over a long
// context, so the eight warps of the weights come here once every part is done and nobody
// waits for them within a bounded wait.
template <int DIM, int FMT>
__device__ __noinline__ void redo_rows(const AttnParams &p, const Piece &piece)
{
    using Cut = Split<kRows, kKeys, kUnitCost>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = piece.x;
    const int64_t x1 = piece.x1;
    Cursor u;
    u.s = piece.s;
    u.at = piece.at;
    Cut::locate(p, x, u);
#pragma unroll 1
    while (true) {
        const int64_t first = u.at + kUnitCost, end = first + u.span.n;
        const int t0 = int(max(x - first, int64_t(0))), t1 = int(max(min(x1, end) - first, int64_t(0)));
        const bool begins = t0 == 0, ends = t1 == u.span.n;
        if (t1 > t0 && ((begins && ends) || (piece.joined >> int(begins) & 1))) {
            // a warp looks at every eighth row, so that only it sees what it writes
            const int row = 8 * lane + warp;
            bool odd = false;
            if (row < min(kRows, u.q.n_new * p.group - u.r * kRows)) {
                int64_t token, col;
                int pos;
                row_place<kRows, DIM>(p, u, row, token, col, pos);
                odd = (p.out[token * p.ldo + col] & 0x7fffu) > 0x7f80u;
            }
            unsigned rows = __ballot_sync(0xffffffffu, odd);
            const float o[DIM / 32] = {};
#pragma unroll 1
            while (rows) {
                finish_row<kRows, DIM, FMT>(p, u, 8 * (__ffs(rows) - 1) + warp, o, __int_as_float(0x7fffffff));
                rows &= rows - 1;
            }
        }
        x = end;
        if (x >= x1)
            break;
        Cut::next(p, u);
    }
}

template <int DIM, int FMT>
__global__ void __launch_bounds__(Crew<FMT>::THREADS, 1) k_attn_tc(const __grid_constant__ AttnParams p)
{
    using S = TcShape<DIM>;
    using Cut = Split<kRows, kKeys, kUnitCost>;
    constexpr int ST = S::STAGES;
    constexpr int kThreads = Crew<FMT>::THREADS, LW = Crew<FMT>::LOADS, LR = Crew<FMT>::ROWS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sm = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sm - raw);
    __shared__ int64_t sums[kThreads / 32];
    __shared__ Cursor cursor;                              // the parts' warp's
    __shared__ Part parts[kParts];
    __shared__ uint32_t poison[kScaleSlots * 4];           // per slot: keys whose value's scale is not finite
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_flag, last_flag, longest;
    __shared__ Piece whole;
    volatile int *dead = &dead_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const KvView &kv = p.kv;
    auto bar = [&](uint32_t i) { return sm + S::BARS + 8 * i; };

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            // the load warps' lanes as their copies end, or the warps as they have stored
            mbar_init(bar(kFull + i), FMT == kKvBf16 ? 32 * LW : LW);
            mbar_init(bar(kEmpty + i), 2);         // a commit of each row tile's products
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kQFull + i), 32 * LW);
            mbar_init(bar(kQEmpty + i), 1);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kWReady + 2 * i), 4);    // the warps of one row tile
            mbar_init(bar(kWReady + 2 * i + 1), 4);
            mbar_init(bar(kPvDone + i), 1);
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(bar(kPartFull + i), 1);
            mbar_init(bar(kPartEmpty + i), 10 + LW);   // every warp that reads the parts
        }
        mbar_init(bar(kJoin), 8);
        mbar_init(bar(kTurn + 0), 1);
        mbar_init(bar(kTurn + 1), 1);
        fence_mbar_init();
        dead_flag = 0;
        longest = 0;
        whole.odd = whole.joined = 0;
    }
    if (warp == 8 + LW)
        tc::tmem_alloc(smem_u32(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    grid_dep_wait();
    grid_dep_launch();

    int64_t piece, total;
    Cut::template find<kThreads, 1>(p, sums, &cursor, piece, total, &longest, kJoinPace);

    // The parts in order, for the warps that read them: `part()` waits for the next and is null
    // past the last (or when the block has given up); `part_done()` lets go of it.
    uint32_t part_no = 0;
    auto part = [&]() -> const Part * {
        const bool there = await(bar(kPartFull + part_no % kParts), part_no / kParts & 1, dead, p.status, kDevTimeoutPipe);
        const Part *q = &parts[part_no % kParts];
        return there && q->more ? q : nullptr;
    };
    auto part_done = [&]() {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(kPartEmpty + part_no % kParts));
        ++part_no;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ weights
        setmaxnreg_inc<Crew<FMT>::more>();
        const int T = warp >> 2, row = tid & 127;
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + T * 128u, tO = tmem + lanes + 256u + T * uint32_t(DIM);
        const float sl = p.scale * 1.4426950408889634f;
        uint32_t n_s = 0, n_end = 0, n_join = 0;           // S tiles taken so far, parts ended, joins
        int tile_no = 0;                                   // key tiles of the CTA so far
        bool alive = true;
        auto wait = [&](uint32_t b, uint32_t parity) {
            alive = __all_sync(0xffffffffu, alive && await(bar(b), parity, dead, p.status, kDevTimeoutMma));
            tc::fence_after_sync();
            return alive;
        };
        auto meet = [&]() {                                // the eight warps of the weights
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(kJoin));
            return wait(kJoin, n_join++ & 1);
        };
        while (alive) {
            const Part *pt = part();
            if (!__all_sync(0xffffffffu, pt != nullptr))
                break;
            const int t0 = pt->t0, t1 = pt->t1, n_sink = pt->n_sink, lo = pt->lo, sink_end = pt->sink;
            const Side sd = pt->side[T];
            const Active act = pt->act[T];
            const bool on = row < sd.rows;
            int pos = -1;
            if (on)
                pos = pt->q.len - pt->q.n_new + (pt->r * kRows + T * kM + row) / p.group;
            float ref = -INFINITY, l = 0.f;
            bool begun = false;
#pragma unroll 1
            for (int t = t0; t < t1; ++t, ++tile_no) {
                if (!act(t))
                    continue;
                const bool sink = t < n_sink;
                const int j0 = sink ? t * kKeys : lo + (t - n_sink) * kKeys;
                const bool masked = j0 + kKeys - 1 > sd.p_first || (sink && j0 + kKeys > sink_end) ||
                                    (p.window && !sink && j0 <= sd.p_last - p.window);
                const float *ks = reinterpret_cast<const float *>(smem + S::SCALES) + (tile_no % kScaleSlots) * 2 * kKeys;
                if (!wait(kSFull + T, n_s & 1))
                    break;
                const uint32_t *odd = poison + (tile_no % kScaleSlots) * 4;
                const bool rework = masked || (FMT == kKvBf16 ? sl <= 0.f : (odd[0] | odd[1] | odd[2] | odd[3]) != 0);
                if (rework) {
                    // the few tiles at an edge of what the rows see: scores scaled and hidden
                    // in place, so that the passes below have one form
                    const int hi = (sink ? min(pos, sink_end - 1) : pos) - j0;     // last key seen
                    const int behind = p.window && !sink ? pos - p.window - j0 : -1;
                    const int kept = p.sinks - j0;
#pragma unroll 1
                    for (int i = 0; i < 128; i += 16) {
                        uint32_t v[16];
                        tmem_ld16_raw(tS + i, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int k = i + e;
                            float x = __uint_as_float(v[e]);
                            if (FMT != kKvBf16) {
                                x *= ks[k];
                                // a value's scale that is not finite makes the row's sum a NaN
                                if (odd[k >> 5] >> (k & 31) & 1)
                                    x = __int_as_float(0x7fffffff);
                            } else if (sl <= 0.f) {
                                x *= sl;
                            }
                            if (k > hi || (k <= behind && k >= kept))
                                x = -INFINITY;
                            v[e] = __float_as_uint(x);
                        }
                        tmem_st16(tS + i, v);
                    }
                    tmem_wait_st();
                }
                const bool plain = FMT == kKvBf16 || rework;   // no scales of the keys to apply
                const float f = FMT == kKvBf16 && sl > 0.f ? sl : 1.f;
                const float top = (plain ? maximum<false>(tS, ks) : maximum<true>(tS, ks)) * f;
                const bool move = top > ref + 8.f;         // the first tile's always does
                if (__any_sync(0xffffffffu, move)) {
                    const float a = move ? exp2_fast(ref - top) : 1.f;
                    if (move)
                        ref = top;
                    l *= a;
                    if (begun) {                           // S here says that the products so far are at rest
#pragma unroll 1
                        for (int i = 0; i < DIM; i += 16) {
                            uint32_t v[16];
                            tmem_ld16_raw(tO + i, v);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
                            tmem_st16(tO + i, v);
                        }
                    }
                }
                const float m = ref == -INFINITY ? 0.f : ref;
                const uint32_t ready = bar(kWReady + 2 * T);
                l += plain ? weights<FMT, false>(tS, ks, f, m, ready) : weights<FMT, true>(tS, ks, f, m, ready);
                begun = true;
                ++n_s;
            }
            // the part's end
            if (begun)
                wait(kPvDone + T, n_end++ & 1);
            if (!alive)
                break;
            if (pt->begins && pt->ends) {
                int64_t token, col;
                row_place<kRows, DIM>(p, *pt, on ? T * kM + row : 0, token, col, pos);
                const float inv = l == 0.f || !begun ? 0.f : 1.f / l;
                bool fine = true;
                uint16_t *dst = p.out + token * p.ldo + col;
#pragma unroll 1
                for (int i = 0; i < DIM; i += 16) {
                    uint32_t v[16];
                    tmem_ld16_raw(tO + i, v);
                    uint4 y[2];
                    uint32_t *yw = reinterpret_cast<uint32_t *>(y);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float a = inv == 0.f ? 0.f : __uint_as_float(v[e]) * inv;
                        const float b = inv == 0.f ? 0.f : __uint_as_float(v[e + 1]) * inv;
                        fine = fine && fabsf(a) < INFINITY && fabsf(b) < INFINITY;
                        yw[e / 2] = pack2(a, b);
                    }
                    if (on) {
                        *reinterpret_cast<uint4 *>(dst + i) = y[0];
                        *reinterpret_cast<uint4 *>(dst + i + 8) = y[1];
                    }
                }
                // a sum of weights that overflowed gives zeros above; it is not finite either
                if (on && !(fine && l < INFINITY)) {
                    *dst = 0x7fff;
                    whole.odd = 1;
                }
            } else {
                const int64_t at = (int64_t(blockIdx.x) * 2 + pt->begins) * kRows + T * kM + row;
                if (on)
                    p.part.cta_ml[at] = make_float2(ref, l);
#pragma unroll 1
                for (int i = 0; i < DIM; i += 16) {
                    uint32_t v[16];
                    tmem_ld16_raw(tO + i, v);
                    if (on)
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<uint4 *>(p.part.cta_o + at * DIM + i + e) =
                                begun ? make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_uint4(0, 0, 0, 0);
                }
                __threadfence();
                if (!meet())
                    break;
                if (warp == 0 && lane == 0) {
                    last_flag = atomicAdd(&p.part.arrived[pt->first], 1) == pt->last - pt->first;
                    if (last_flag) {
                        p.part.arrived[pt->first] = 0;
                        whole.joined |= 1 << pt->begins;
                    }
                }
                if (!meet())
                    break;
                if (last_flag) {
                    __threadfence();
                    if (join_unit<DIM, FMT>(p, *pt))
                        whole.odd = 1;
                }
                if (!meet())                               // last_flag is free again
                    break;
            }
            tc::fence_before_sync();
            part_done();
        }
        if (alive && meet() && whole.odd)
            redo_rows<DIM, FMT>(p, whole);
    } else if (warp < 8 + LW) {
        // ------------------------------------------------------------ loads
        setmaxnreg_dec<Crew<FMT>::load>();
        const int lw = warp - 8;                           // this warp has LR keys (or rows) of a tile,
        const int mine = lw * LR + lane;                   // this lane one of them (of the lanes below LR)
        bool alive = true;
        uint32_t entry = 0, slot = 0, phase = 1;           // ring entries: keys 2j, values 2j + 1
        int tile_no = 0;
        auto wait = [&](uint32_t b, uint32_t parity) {
            alive = __all_sync(0xffffffffu, alive && await(bar(b), parity, dead, p.status, kDevTimeoutPipe));
            return alive;
        };
        auto wait_slot = [&]() { return entry < uint32_t(ST) || wait(kEmpty + slot, phase); };
        auto advance = [&]() {
            ++entry;
            if (++slot == uint32_t(ST))
                slot = 0, phase ^= 1;
        };
        // The part in hand, by what a lane needs of it: its key of tile t is key0 + (t - t0) *
        // kKeys (a part's first tokens and its window are runs of their own).
        const Part *pt = nullptr;
        int t = 0;
        auto enter = [&]() {
            pt = part();
            if (!__all_sync(0xffffffffu, pt != nullptr))
                pt = nullptr;
            t = pt ? pt->t0 : 0;
        };
        auto page_id = [&]() -> int {                      // INT_MIN: no key
            if (!pt)
                return INT_MIN;
            const bool sink = t < pt->n_sink;
            const int j = (sink ? t * kKeys : pt->lo + (t - pt->n_sink) * kKeys) + mine;
            return lane < LR && j < (sink ? pt->sink : pt->hi) ? p.b.pages[int64_t(pt->s) * p.b.ld_pages + page_of(kv, j)] : INT_MIN;
        };
        auto place = [&](int page, int64_t &at, int64_t &s_at) {
            at = -1;
            s_at = 0;
            if (page == INT_MIN)
                return;
            if (page < 0 || page >= kv.n_pages) {
                raise_status(p.status, kDevBadPage);
                return;
            }
            const int j = (t < pt->n_sink ? t * kKeys : pt->lo + (t - pt->n_sink) * kKeys) + mine;
            const int cell = j - page_of(kv, j) * kv.page_size;
            at = page * kv.page_stride + cell * kv.cell_stride + pt->h * kv.head_stride;
            s_at = page * kv.s_page + cell * kv.s_cell + pt->h * kv.s_head;
        };
        auto q_place = [&](int T) -> int64_t {             // this lane's row of the queries, bytes
            const int row = T * kM + mine;
            if (lane >= LR || pt->r * kRows + row >= pt->q.n_new * p.group)
                return -1;
            int64_t token, col;
            int pos;
            row_place<kRows, DIM>(p, *pt, row, token, col, pos);
            return (token * p.ldq + col) * 2;
        };
        constexpr int CH = DIM / 8, RPI = 32 / CH;         // 16-byte chunks of a bf16 row, rows an instruction
        // The copies arrive on `done` by themselves, lane by lane, as they end; the warp that
        // reads them by the tensor cores makes them visible to those.
        auto copy_rows = [&](uint32_t dst, const uint8_t *src, int64_t at, uint32_t done) {
#pragma unroll 4
            for (int i = 0; i < LR / RPI; ++i) {
                const int rr = i * RPI + lane / CH, ch = lane % CH, row = lw * LR + rr;
                const int64_t a = __shfl_sync(0xffffffffu, (long long)at, rr);
                tc::cp_async16(dst + (ch / 8) * S::HALF + tc::sw128(row, ch % 8), src + (a < 0 ? 0 : a + ch * 16), a < 0 ? 0u : 16u);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(done)) : "memory");
        };
        enter();
        int page = page_id();
        int64_t at = -1, s_at = 0;
        if (FMT == kKvBf16) {
            // per tile: keys, then the queries of a new part, then values
            while (pt && alive) {
                place(page, at, s_at);
                const bool fresh = t == pt->t0;
                const uint32_t no = part_no;
                const int64_t qa = fresh ? q_place(0) : -1, qb = fresh ? q_place(1) : -1;
                if (++t == pt->t1) {
                    part_done();
                    enter();
                }
                page = page_id();                          // on its way during this tile
#pragma unroll 1
                for (int job = 0; job < 4; ++job) {
                    const bool ring = job == 0 || job == 3;
                    if (!ring && !fresh)
                        continue;
                    if (!(ring ? wait_slot() : no == 0 || wait(kQEmpty + job - 1, (no - 1) & 1)))
                        break;
                    copy_rows(ring ? sm + S::RING + slot * S::TILE : sm + (job - 1) * S::TILE,
                              job == 0 ? kv.k : job == 3 ? kv.v : reinterpret_cast<const uint8_t *>(p.q),
                              ring ? at : job == 1 ? qa : qb, ring ? kFull + slot : kQFull + job - 1);
                    if (ring)
                        advance();
                }
            }
        } else {
            constexpr int C8 = DIM / 16, R8 = 32 / C8;     // 16-byte chunks of a row of codes, rows an instruction
            constexpr int XN = LR / R8;
            auto fetch = [&](uint4 x[XN], const uint8_t *src, int64_t at) {
#pragma unroll
                for (int i = 0; i < XN; ++i) {
                    const int64_t a = __shfl_sync(0xffffffffu, (long long)at, i * R8 + lane / C8);
                    x[i] = a < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(src + a + (lane % C8) * 16);
                }
            };
            auto store = [&](const uint4 x[XN]) {          // into the ring's next slot
#pragma unroll
                for (int i = 0; i < XN; ++i) {
                    const int row = lw * LR + i * R8 + lane / C8, ch = 2 * (lane % C8);
                    const uint2 a = widen4_unit<FMT>(x[i].x), b = widen4_unit<FMT>(x[i].y), c = widen4_unit<FMT>(x[i].z), d = widen4_unit<FMT>(x[i].w);
                    uint8_t *base = smem + S::RING + slot * S::TILE + (ch / 8) * S::HALF;
                    *reinterpret_cast<uint4 *>(base + tc::sw128(row, ch % 8)) = make_uint4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<uint4 *>(base + tc::sw128(row, ch % 8 + 1)) = make_uint4(c.x, c.y, d.x, d.y);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(kFull + slot));
                advance();
            };
            const float sl = p.scale * 1.4426950408889634f;
            // x holds the tile that is stored next, y the one after it on its way
            uint4 x[XN], y[XN];
            float ks = 0.f, vs = 0.f;
            auto begin = [&]() {
                place(page, at, s_at);
                fetch(x, kv.k, at);
                ks = at < 0 ? 0.f : kv.k_scale[s_at] * (sl / kCodeUnit<FMT>);
                vs = at < 0 ? 0.f : kv.v_scale[s_at] * (1.f / kCodeUnit<FMT>);
            };
            if (pt)
                begin();
            while (pt && alive) {
                const bool fresh = t == pt->t0;
                const uint32_t no = part_no;
                fetch(y, kv.v, at);
                const int64_t qa = fresh ? q_place(0) : -1, qb = fresh ? q_place(1) : -1;
                if (++t == pt->t1) {
                    part_done();
                    enter();
                }
                page = page_id();
                if (!wait_slot())
                    break;
                float *sc = reinterpret_cast<float *>(smem + S::SCALES) + (tile_no % kScaleSlots) * 2 * kKeys + mine;
                const bool fine = fabsf(vs) < INFINITY;
                if (lane < LR) {
                    sc[0] = ks;
                    sc[kKeys] = fine ? vs : 0.f;
                }
                const unsigned bad = __ballot_sync(0xffffffffu, !fine);
                if (lane == 0)
                    reinterpret_cast<uint16_t *>(poison)[(tile_no % kScaleSlots) * 8 + lw] = uint16_t(bad);
                store(x);
                if (fresh) {
#pragma unroll 1
                    for (int T = 0; T < 2; ++T) {
                        if (no > 0 && !wait(kQEmpty + T, (no - 1) & 1))
                            break;
                        copy_rows(sm + T * S::TILE, reinterpret_cast<const uint8_t *>(p.q), T ? qb : qa, kQFull + T);
                    }
                }
                if (pt)
                    begin();
                if (!wait_slot())
                    break;
                store(y);
                ++tile_no;
            }
        }
    } else if (warp < 10 + LW) {
        // ------------------------------------------------------------ products
        setmaxnreg_dec<Crew<FMT>::few>();
        const int T = warp - 8 - LW;
        if (lane == 0) {
            constexpr uint32_t iqk = tc::idesc_bf16(kM, kKeys, 0, 0), ipv = tc::idesc_bf16(kM, DIM, 0, 1);
            constexpr uint32_t kTile16 = S::TILE / 16, kHalf16 = S::HALF / 16;   // descriptor units
            const uint64_t q = tc::smem_desc_sw128(sm + T * S::TILE, 16u, 1024u),
                           k_desc = tc::smem_desc_sw128(sm + S::RING, 16u, 1024u),
                           v_desc = tc::smem_desc_sw128(sm + S::RING, S::HALF, 1024u);
            const uint32_t tS = tmem + T * 128u, tO = tmem + 256u + T * uint32_t(DIM);
            // ring slots of the keys and values in turn: keys 2j, values 2j + 1
            uint32_t k_slot = 0, k_phase = 0, v_slot = 1, v_phase = 0, w_phase = 0;
            uint32_t turn = 0;                             // rounds so far
            auto next_slot = [&](uint32_t &slot, uint32_t &phase) {
                slot += 2;
                if (slot >= uint32_t(ST))
                    slot -= ST, phase ^= 1;
            };
            bool alive = true;
            auto wait = [&](uint32_t b, uint32_t parity) {
                alive = alive && await(bar(b), parity, dead, p.status, kDevTimeoutPipe);
                return alive;
            };
            while (alive) {
                const Part *pt = part();
                if (!pt)
                    break;
                const Active act = pt->act[T];
                const int t0 = pt->t0, t1 = pt->t1;
                mbar_arrive(bar(kPartEmpty + part_no % kParts));
                uint32_t started = 0;
                // Round t: the values of tile t - 1 and the scores of tile t, one behind the
                // other; what they need besides the weights is waited for ahead.
#pragma unroll 1
                for (int t = t0; t <= t1; ++t) {
                    const bool with_v = t > t0, with_s = t < t1;
                    if (with_v && !wait(kFull + v_slot, v_phase))
                        break;
                    if (with_s && !wait(kFull + k_slot, k_phase))
                        break;
                    if (t == t0 && !wait(kQFull + T, part_no & 1))
                        break;
                    tc::fence_proxy_async_smem();          // the copies that were waited for
                    const bool values = with_v && act(t - 1);
                    if (values && !wait(kWReady + 2 * T, w_phase))
                        break;
                    // A's round, then B's, by turns: A's first needs no leave, B's n-th and A's
                    // next have the other's
                    if ((T == 1 || turn > 0) && !wait(kTurn + T, (turn - (T == 0)) & 1))
                        break;
                    ++turn;
                    tc::fence_after_sync();
                    if (values) {
                        const uint64_t v = v_desc + v_slot * kTile16;
                        mma_tmem_a(tO, tS, v, ipv, started);
#pragma unroll
                        for (int i = 1; i < kKeys / 32; ++i)
                            mma_tmem_a(tO, tS + 8 * i, v + 128 * i, ipv, 1);
                        if (!wait(kWReady + 2 * T + 1, w_phase))
                            break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int i = kKeys / 32; i < kKeys / 16; ++i)
                            mma_tmem_a(tO, tS + 8 * i, v + 128 * i, ipv, 1);
                        w_phase ^= 1;
                        started = 1;
                    }
                    if (with_s && act(t)) {
                        const uint64_t k = k_desc + k_slot * kTile16;
#pragma unroll
                        for (int i = 0; i < DIM / 16; ++i)
                            tc::mma_bf16(tS, q + (i / 4) * kHalf16 + 2 * (i % 4), k + (i / 4) * kHalf16 + 2 * (i % 4), iqk, i > 0);
                        // says that every product so far has ended, the values' among them
                        tc::mma_commit(bar(kSFull + T));
                    }
                    mbar_arrive(bar(kTurn + 1 - T));
                    if (t == t1 && started)
                        tc::mma_commit(bar(kPvDone + T));
                    if (with_v) {
                        tc::mma_commit(bar(kEmpty + v_slot));
                        next_slot(v_slot, v_phase);
                    }
                    if (with_s) {
                        tc::mma_commit(bar(kEmpty + k_slot));
                        next_slot(k_slot, k_phase);
                        if (t + 1 == t1)
                            tc::mma_commit(bar(kQEmpty + T));
                    }
                }
                ++part_no;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ parts
        setmaxnreg_dec<Crew<FMT>::few>();
        if (warp == 10 + LW && lane == 0) {
            int64_t x = piece * blockIdx.x;
            const int64_t x1 = min(x + piece, total);
            if (x < x1) {
                whole.x = x, whole.x1 = x1;
                whole.s = cursor.s, whole.at = cursor.at;
                Cut::locate(p, x, cursor);
            }
            bool more = true;
            while (more) {
                int t0 = 0, t1 = 0;
                while (x < x1) {                           // the next unit that has tiles here
                    const int64_t first = cursor.at + kUnitCost, end = first + cursor.span.n;
                    t0 = int(max(x - first, int64_t(0)));
                    t1 = int(max(min(x1, end) - first, int64_t(0)));
                    x = end;
                    if (t1 > t0)
                        break;
                    if (x < x1)
                        Cut::next(p, cursor);
                }
                more = t1 > t0;
                const uint32_t slot = part_no % kParts;
                if (part_no >= kParts &&
                    !await(bar(kPartEmpty + slot), (part_no / kParts - 1) & 1, dead, p.status, kDevTimeoutPipe))
                    break;
                Part &q = parts[slot];
                q.more = more;
                if (more) {
                    q.s = cursor.s, q.r = cursor.r, q.h = cursor.h, q.q = cursor.q;
                    q.t0 = t0, q.t1 = t1;
                    q.n_sink = cursor.span.n_sink, q.lo = cursor.span.lo, q.hi = cursor.span.hi, q.sink = cursor.span.sink;
                    q.begins = t0 == 0;
                    q.ends = t1 == cursor.span.n;
                    q.first = int(quotient(cursor.at + kUnitCost, piece));
                    q.last = int(quotient(cursor.at + kUnitCost + cursor.span.n - 1, piece));
                    for (int T = 0; T < 2; ++T) {
                        q.side[T] = side_of(p, cursor, T);
                        q.act[T] = active(p, cursor, q.side[T]);
                    }
                }
                mbar_arrive(bar(kPartFull + slot));
                ++part_no;
                if (more && x < x1)
                    Cut::next(p, cursor);
            }
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // Every product has ended: the weights' warps waited for each tile's last.  Where the
    // roles gave up, those under way get the time that they can take at most.
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 8 + LW) {
        if (dead_flag) {
            const uint64_t t = globaltimer_ns();
            while (globaltimer_ns() - t < 1000000ull) {
            }
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int DIM, int FMT>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = once([] {
        return cudaFuncSetAttribute(k_attn_tc<DIM, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    TcShape<DIM>::SMEM);
    });
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(sms));
    cfg.blockDim = dim3(Crew<FMT>::THREADS);
    cfg.dynamicSmemBytes = TcShape<DIM>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_tc<DIM, FMT>, p);
}

}  // namespace

size_t attn_tc_scratch(uint8_t *base, int sms, AttnScratch *s)
{
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *p = base + at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    AttnScratch t{};
    t.cta_o = reinterpret_cast<float *>(take(size_t(sms) * 2 * kRows * 128 * sizeof(float)));
    t.cta_ml = reinterpret_cast<float2 *>(take(size_t(sms) * 2 * kRows * sizeof(float2)));
    t.arrived = reinterpret_cast<int *>(take(size_t(sms) * sizeof(int)));
    if (s)
        *s = t;
    return at;
}

cudaError_t launch_attn_tc(const AttnParams &p, int sms, cudaStream_t stream)
{
    const bool wide = p.kv.dim == 128;
    switch (p.kv.format) {
    case kKvBf16: return wide ? launch<128, kKvBf16>(p, sms, stream) : launch<64, kKvBf16>(p, sms, stream);
    case kKvInt8: return wide ? launch<128, kKvInt8>(p, sms, stream) : launch<64, kKvInt8>(p, sms, stream);
    default: return wide ? launch<128, kKvFp8>(p, sms, stream) : launch<64, kKvFp8>(p, sms, stream);
    }
}

}  // namespace lora
