// Norms of each head's queries and keys, then the rotation of their pairs by position, in one
// pass; on request keys and values go straight to their cells in the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w                      (per head, where there is a w)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),      t = position * freqs[j]
//
// over the pairs (j, j + half) or (2j, 2j + 1) of a head's first 2 half elements.  All in fp32,
// rounded once: to bf16, or to the cache's 8-bit codes straight from fp32.
//
// Angles.  position * frequency has more bits than fp32, and near 32,768 an fp32 product is off
// by 2e-3.  Whole turns do not matter, so the frequency is taken as a 64-bit binary fraction of
// a turn (from a double-double product with 1 / 2 pi, once a CTA), and position times it modulo
// 2^64 is the angle: off by at most 2^-34 turns at any position, by one integer product.  Its cosine and
// sine are taken of 32 of these bits in fp32, whose 24 are within 2^-26 turns: fp32's own step.
//
// A vector is one (row, head), 16 elements a lane: eight and eight that are turned with one
// another (a lane's own pairs, so nothing is exchanged), or 16 side by side.  An item is as many
// vectors of one row as a warp holds; a CTA serves up to eight rows, whose items its warps take
// in turn, two under way at once.  Bound: DRAM at prefill sizes (each vector read and written
// once; norms add an exchange over the vector's lanes to each item's chain), the chain launch,
// lengths, angles for a decode batch.
//
// Measured: 16,896 rows of 32 + 32 heads of 128 without norms 86 us, 6.4 TB/s (0.95 of a copy's
// rate); 8191 rows of 32 + 8 heads with norms and the store into a bf16 cache 41 us (36 without the
// norms), 4.9 TB/s, into int8 45.5 and e4m3 46.6 us.  Eight elements a lane, pairs in two lanes and
// exchanged, took 173 and 58 us, bound by instructions; three CTAs a SM instead of four 89 and 41, five 91 and 53.
#include <cuda_fp8.h>
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
constexpr int kMaxRows = kWarps;             // rows a CTA: a warp looks up each
constexpr int kCtas = 4;                     // a SM
constexpr int kMaxHalf = 128;                // pairs of a head
constexpr int kNone = -1;                    // FMT: nothing goes to a cache
constexpr float kMaxFreq = 1048576.f;        // radians a token: the fraction's low part fits

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// f / 2 pi modulo 1, in units of 2^-64.  Of |f|, whose whole turns come off without a rounding (next to
// -0 the remainder would have to be rounded to 2^-54, 2^-24 turns at position 2^30).
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    // 1 / 2 pi to 106 bits
    const double c0 = 0x1.45f306dc9c883p-3, c1 = -0x1.6b01ec5417056p-57;
    const double x = fabsf(f), hi = x * c0, lo = fma(x, c0, -hi) + x * c1;
    const uint64_t t = uint64_t(__double2ull_rn((hi - floor(hi)) * 0x1p64)) + uint64_t(__double2ll_rn(lo * 0x1p64));
    return f < 0.f ? 0 - t : t;
}

// The codes of one vector held 16 elements (fp32) a lane by LANES consecutive lanes, and its
// scale, by the rule of encode16 (kv.cuh).  Every lane of the warp calls it.
template <int FMT, int LANES>
__device__ __forceinline__ uint4 encode_wide(const float f[16], float &scale)
{
    constexpr float T = code_top<FMT>();
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e)
        top = max_nan(top, fabsf(f[e]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!(top < INFINITY)) {
        scale = __int_as_float(0x7fffffff);
        return make_uint4(0, 0, 0, 0);
    }
    scale = __fdiv_rn(top, T);
    const float d = scale > 0.f ? scale : 1.f;
    // the quotient lies between the products with 1 / d taken 2^-21 too small and too large
    const float r = __fdividef(1.f, d), r0 = r * (1.f - 0x1p-21f), r1 = r * (1.f + 0x1p-21f);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float *v = f + 4 * w;
        auto four = [&](float q) {
            if (FMT == kKvInt8) {
                // added to 1.5 * 2^23, a number rounds to an integer that the low bits hold
                uint32_t a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a[e] = __float_as_uint(fmaf(v[e], q, 12582912.f));
                return __byte_perm(__byte_perm(a[0], a[1], 0x0040), __byte_perm(a[2], a[3], 0x0040), 0x5410);
            }
            return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(v[0] * q, v[1] * q), __NV_SATFINITE, __NV_E4M3)) |
                   uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(v[2] * q, v[3] * q), __NV_SATFINITE, __NV_E4M3)) << 16;
        };
        lo[w] = four(r0);
        hi[w] = four(r1);
    }
    const uint32_t differ = (lo[0] ^ hi[0]) | (lo[1] ^ hi[1]) | (lo[2] ^ hi[2]) | (lo[3] ^ hi[3]);
    if (differ || !(d > 1e-30f && d < 1e30f)) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            hi[w] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // a scale that was rounded down puts the largest element past the top
                const float z = fminf(fmaxf(__fdiv_rn(f[4 * w + e], d), -T), T);
                const uint32_t code = FMT == kKvInt8 ? uint32_t(__float2int_rn(z)) & 0xffu
                                                     : uint32_t(__nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3));
                hi[w] |= code << (8 * e);
            }
        }
    }
    return make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// A row's queries, keys and values: where they come from and go.
struct RowSides {
    const uint16_t *src[3];
    uint8_t *dst[3];
    int64_t scale_at;
    int pos;                  // negative: no position
    bool on[3];               // what is written
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(d)) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

__device__ __forceinline__ uint4 pack(const float2 f[4])
{
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = __float22bfloat162_rn(f[e]);
    return u;
}

// G lanes a vector.
template <int G, int FMT>
__global__ void __launch_bounds__(kThreads, kCtas) k_rope(const __grid_constant__ RopeParams p, int rows)
{
    constexpr int kVec = 32 / G;                     // vectors of an item
    constexpr bool kStore = FMT != kNone;
    __shared__ RowSides sides[kMaxRows];
    __shared__ uint64_t fraction[kMaxHalf];
    __shared__ bool fraction_bad[kMaxHalf];
    // angles two by two (both cosines, both sines), and weights, as the lanes read them: [which of a lane's][lane]
    __shared__ float4 turn[kMaxRows][4][G];
    __shared__ float4 weight[2][4][G];
    const int row0 = blockIdx.x * rows, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / G, l = lane % G;
    const int half = p.half, k_at = p.q_heads, v_at = p.q_heads + p.k_heads;
    // Where a lane's elements are: e0 .. e0 + 7 and e1 .. e1 + 7.
    auto places_of = [&](int lane, int &e0, int &e1) {
        const int hl = p.interleaved ? 0 : half / 8;
        e0 = lane < hl ? lane * 8 : 2 * hl * 8 + (lane - hl) * 16;
        e1 = lane < hl ? half + lane * 8 : e0 + 8;
    };
    int e0, e1;
    places_of(l, e0, e1);
    const bool turns = p.interleaved ? l * 16 < 2 * half : l * 8 < half;
    const bool on0 = e0 < p.dim, on1 = e1 < p.dim;
    grid_dep_wait();
    grid_dep_launch();
    const int nvec = kStore ? v_at + p.k_heads : v_at, n_rows = min(rows, p.b.n_rows - row0);
    const int row_items = (nvec + kVec - 1) / kVec, items = n_rows * row_items, stride = gridDim.y * kWarps;
    auto load = [&](int it, uint4 x[2]) {
        const int r = p.per_row.quotient(it), vec = (it - r * row_items) * kVec + sub;
        const int64_t row = row0 + r;
        const uint16_t *src = vec < k_at ? p.q + row * p.ldq + vec * p.dim
                              : !kStore || vec < v_at ? p.k + row * p.ldk + (vec - k_at) * p.dim
                                                      : p.v + row * p.ldv + (vec - v_at) * p.dim;
        const bool on = it < items && vec < nvec;
        x[0] = on && on0 ? *reinterpret_cast<const uint4 *>(src + e0) : uint4{0, 0, 0, 0};
        x[1] = on && on1 ? *reinterpret_cast<const uint4 *>(src + e1) : uint4{0, 0, 0, 0};
    };
    // the first vectors are on their way while the rows' places are looked up
    int it = blockIdx.y * kWarps + warp;
    uint4 x0[2], x1[2];
    load(it, x0);
    load(it + stride, x1);
    const bool norms = p.q_weight || p.k_weight;
    if (norms)
        for (int i = threadIdx.x; i < 8 * G; i += kThreads) {
            const int side = i / (4 * G), which = i / G % 4;
            int a, b;
            places_of(i % G, a, b);
            const int d = (which & 2 ? b : a) + (which & 1) * 4;
            const float *w = side ? p.k_weight : p.q_weight;
            weight[side][which][i % G] = w && d < p.dim ? *reinterpret_cast<const float4 *>(w + d) : make_float4(1.f, 1.f, 1.f, 1.f);
        }
    for (int j = threadIdx.x; j < half; j += kThreads) {
        fraction[j] = turn_fraction(p.freqs[j]);
        fraction_bad[j] = !(fabsf(p.freqs[j]) <= kMaxFreq);
    }
    if (warp < n_rows) {
        const int64_t row = row0 + warp;
        const RowAt at = find_pos(p.b, int(row), p.status);
        Place pl{at.live, false, 0, 0};
        if (kStore)
            pl = place_of(p.kv, p.b, at, p.status);
        if (lane == 0) {
            RowSides &s = sides[warp];
            s.src[0] = p.q + row * p.ldq;
            s.src[1] = p.k + row * p.ldk;
            s.src[2] = p.v + row * p.ldv;
            s.dst[0] = reinterpret_cast<uint8_t *>(p.q_out + row * p.ldqo);
            s.dst[1] = kStore ? p.kv.k + pl.at : reinterpret_cast<uint8_t *>(p.k_out + row * p.ldko);
            s.dst[2] = p.kv.v + pl.at;
            s.scale_at = pl.s_at;
            s.pos = at.live ? at.pos : -1;
            s.on[0] = pl.live;
            s.on[1] = s.on[2] = kStore ? pl.stored : pl.live;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_rows * half; i += kThreads) {
        const int r = int(unsigned(i) / unsigned(half)), j = i - r * half;
        const uint64_t t = fraction[j] * uint64_t(max(sides[r].pos, 0)) + 0x80000000ull;
        float s, c;
        sincospif(float(int(t >> 32)) * 0x1p-31f, &s, &c);
        if (fraction_bad[j])
            s = c = __int_as_float(0x7fffffff);
        float *at = reinterpret_cast<float *>(&turn[r][j / 2 % 4][j / 8]) + (j & 1);
        at[0] = c;
        at[2] = s;
    }
    __syncthreads();
    const float mean = 1.f / float(p.dim);
    const int64_t kv_stride = kStore ? p.kv.head_stride : p.dim * 2;
    auto work = [&](int it, uint4 x[2]) {
        const int r = p.per_row.quotient(it), vec = (it - r * row_items) * kVec + sub;
        const int side = vec < k_at ? 0 : kStore && vec >= v_at ? 2 : 1;
        const RowSides &row = sides[r];
        const bool put = vec < nvec && row.on[side];
        float2 f[8];                                 // elements two by two
        unpack8(x[0], reinterpret_cast<float *>(f));
        unpack8(x[1], reinterpret_cast<float *>(f + 4));
        if (norms) {
            float2 ss = mul2(f[0], f[0]), st = mul2(f[4], f[4]);
#pragma unroll
            for (int e = 1; e < 4; ++e) {
                ss = fma2(f[e], f[e], ss);
                st = fma2(f[4 + e], f[4 + e], st);
            }
            float sum = (ss.x + ss.y) + (st.x + st.y);
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (side != 2 && (side ? p.k_weight : p.q_weight)) {
                const float inv = rsqrtf(fmaf(sum, mean, p.eps));
                const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = weight[side][e][l];
                    f[2 * e] = mul2(mul2(f[2 * e], inv2), make_float2(w.x, w.y));
                    f[2 * e + 1] = mul2(mul2(f[2 * e + 1], inv2), make_float2(w.z, w.w));
                }
            }
        }
        if (side != 2 && turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 cs = turn[r][e][l];
                if (p.interleaved) {
                    auto pair = [&](float2 &x, float c, float s) { x = make_float2(x.x * c - x.y * s, x.x * s + x.y * c); };
                    pair(f[2 * e], cs.x, cs.z);
                    pair(f[2 * e + 1], cs.y, cs.w);
                } else {
                    const float2 c = make_float2(cs.x, cs.y), s = make_float2(cs.z, cs.w), a = f[e], b = f[4 + e];
                    f[e] = fma2(a, c, mul2(b, make_float2(-s.x, -s.y)));
                    f[4 + e] = fma2(a, s, mul2(b, c));
                }
            }
        }
        uint8_t *dst = row.dst[side];
        if (side == 0)
            dst += vec * p.dim * 2;
        else
            dst += (vec - (side == 2 ? v_at : k_at)) * kv_stride;
        if (!kStore || side == 0 || FMT == kKvBf16) {
            // a row without a position becomes zeros (it has no cell)
            const bool zero = row.pos < 0;
            uint4 y0 = pack(f), y1 = pack(f + 4);
            if (zero)
                y0 = y1 = uint4{0, 0, 0, 0};
            if (put && on0)
                *reinterpret_cast<uint4 *>(dst + e0 * 2) = y0;
            if (put && on1)
                *reinterpret_cast<uint4 *>(dst + e1 * 2) = y1;
        }
        if constexpr (FMT == kKvInt8 || FMT == kKvFp8) {
            if (__any_sync(0xffffffffu, put && side)) {
                float scale;
                const uint4 code = encode_wide<FMT, G>(reinterpret_cast<const float *>(f), scale);
                if (put && side) {
                    *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(code.x, code.y);
                    *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(code.z, code.w);
                    if (l == 0)
                        (side == 2 ? p.kv.v_scale : p.kv.k_scale)[row.scale_at + (vec - (side == 2 ? v_at : k_at)) * p.kv.s_head] = scale;
                }
            }
        }
    };
    // behind the look-ups an item's vectors are found in `sides`
    auto load_next = [&](int it, uint4 x[2]) {
        if (it >= items)
            return;
        const int r = p.per_row.quotient(it), vec = (it - r * row_items) * kVec + sub;
        const int side = vec < k_at ? 0 : kStore && vec >= v_at ? 2 : 1;
        const uint16_t *src = sides[r].src[side] + (vec - (side == 2 ? v_at : side ? k_at : 0)) * p.dim;
        if (vec < nvec && on0)
            x[0] = *reinterpret_cast<const uint4 *>(src + e0);
        if (vec < nvec && on1)
            x[1] = *reinterpret_cast<const uint4 *>(src + e1);
    };
    while (it < items) {
        work(it, x0);
        load_next(it + 2 * stride, x0);
        it += stride;
        if (it >= items)
            break;
        work(it, x1);
        load_next(it + 2 * stride, x1);
        it += stride;
    }
}

template <int G, int FMT>
cudaError_t launch(RopeParams p, int sms, cudaStream_t stream)
{
    // Several rows a CTA, so that whole waves of them are on the GPU; a row cut into parts where
    // there are not enough.
    const int64_t wave = int64_t(sms) * kCtas;
    const int64_t n = p.b.n_rows, waves = std::max<int64_t>(1, (n + wave * kMaxRows - 1) / (wave * kMaxRows));
    const int rows = int(std::max<int64_t>(1, n / wave < 1 ? 1 : (n + wave * waves - 1) / (wave * waves)));
    const int nvec = p.q_heads + (FMT != kNone ? 2 : 1) * p.k_heads, row_items = (nvec + 32 / G - 1) / (32 / G);
    p.per_row = Divider(row_items);
    const int64_t parts = rows > 1 ? 1 : std::max<int64_t>(1, std::min<int64_t>((row_items + kWarps - 1) / kWarps, wave / std::max<int64_t>(n, 1)));
    const dim3 grid{unsigned((n + rows - 1) / rows), unsigned(parts)};
    return start(k_rope<G, FMT>, grid, kThreads, 0, 0, stream, p, rows);
}

template <int FMT>
cudaError_t launch(const RopeParams &p, int sms, cudaStream_t stream)
{
    if constexpr (FMT == kNone)                      // a cache has heads of 64 or 128
        if (p.dim > 128)
            return launch<16, FMT>(p, sms, stream);
    return p.dim <= 64 ? launch<4, FMT>(p, sms, stream) : launch<8, FMT>(p, sms, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool store, int sms, cudaStream_t stream)
{
    if (!store)
        return launch<kNone>(p, sms, stream);
    switch (p.kv.format) {
    case kKvBf16: return launch<kKvBf16>(p, sms, stream);
    case kKvInt8: return launch<kKvInt8>(p, sms, stream);
    default: return launch<kKvFp8>(p, sms, stream);
    }
}

}  // namespace lora
