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
// 2^64 is the angle: off by at most 2^-34 turns at any position, by one integer product.
//
// A vector is one (row, head), eight elements a lane (16 bytes of bf16); a CTA serves up to
// eight rows.  A pair's other half is another lane's: a shuffle.  Bound: DRAM at prefill sizes
// (each vector read and written once), the chain launch, lengths, angles for a decode batch.
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
constexpr int kMaxRows = kThreads / 32;      // rows a CTA: a warp looks up each
constexpr int kMaxHalf = 128;                // pairs of a head
constexpr int kNone = -1;                    // FMT: nothing goes to a cache
constexpr float kMaxFreq = 1048576.f;        // radians a token: the fraction's low part fits

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// f / 2 pi modulo 1, in units of 2^-64.
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    // 1 / 2 pi to 106 bits
    const double c0 = 0x1.45f306dc9c883p-3, c1 = -0x1.6b01ec5417056p-57;
    const double x = f, hi = x * c0, lo = fma(x, c0, -hi) + x * c1;
    return uint64_t(__double2ull_rn((hi - floor(hi)) * 0x1p64)) + uint64_t(__double2ll_rn(lo * 0x1p64));
}

// The codes of one vector held 8 elements (fp32) a lane by LANES consecutive lanes, and its
// scale, by the rule of encode16 (kv.cuh).  Every lane of the warp calls it.
template <int FMT, int LANES>
__device__ __forceinline__ uint2 encode8(const float f[8], float &scale)
{
    constexpr float T = code_top<FMT>();
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = max_nan(top, fabsf(f[e]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!(top < INFINITY)) {
        scale = __int_as_float(0x7fffffff);
        return make_uint2(0, 0);
    }
    scale = __fdiv_rn(top, T);
    const float d = scale > 0.f ? scale : 1.f;
    auto pack = [&](float r) {
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (FMT == kKvInt8)
                c[e] = __float_as_uint(fmaf(f[e], r, 12582912.f)) & 0xffu;
            else
                c[e] = uint32_t(__nv_cvt_float_to_fp8(f[e] * r, __NV_SATFINITE, __NV_E4M3));
        return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    };
    // the quotient lies between the products with 1 / d taken 2^-21 too small and too large
    const float r = __fdividef(1.f, d);
    const uint2 lo = pack(r * (1.f - 0x1p-21f));
    uint2 hi = pack(r * (1.f + 0x1p-21f));
    if (lo.x != hi.x || lo.y != hi.y || !(d > 1e-30f && d < 1e30f)) {
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // a scale that was rounded down puts the largest element past the top
            const float z = fminf(fmaxf(__fdiv_rn(f[e], d), -T), T);
            const uint32_t code = FMT == kKvInt8 ? uint32_t(__float2int_rn(z)) & 0xffu
                                                 : uint32_t(__nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3));
            c[e / 4] |= code << (8 * (e % 4));
        }
        hi = make_uint2(c[0], c[1]);
    }
    return hi;
}

// G lanes a vector.
template <int G, int FMT>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeParams p, int rows)
{
    constexpr int kPer = kThreads / G;               // vectors per pass of the CTA
    constexpr int U = 4;
    constexpr bool kStore = FMT != kNone;
    __shared__ Place places[kMaxRows];
    __shared__ int row_pos[kMaxRows];
    __shared__ uint64_t fraction[kMaxHalf];
    __shared__ __align__(16) float2 turn[kMaxRows][kMaxHalf];
    const int row0 = blockIdx.x * rows, sub = threadIdx.x / G, l = threadIdx.x % G, warp = threadIdx.x >> 5;
    const int d0 = l * 8, half = p.half, kv_at = p.q_heads;
    const bool lane_on = d0 < p.dim;
    grid_dep_wait();
    grid_dep_launch();
    const int nvec = p.q_heads + (kStore ? 2 : 1) * p.k_heads, all = min(rows, p.b.n_rows - row0) * nvec;
    const int stride = gridDim.y * kPer * U;
    uint4 x[U];
    auto load = [&](int v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = v0 + u * kPer + sub, r = p.per_row.quotient(i), row = row0 + r, vec = i - r * nvec;
            const uint16_t *src = vec < kv_at ? p.q + int64_t(row) * p.ldq + vec * p.dim
                                  : vec < kv_at + p.k_heads ? p.k + int64_t(row) * p.ldk + (vec - kv_at) * p.dim
                                                            : p.v + int64_t(row) * p.ldv + (vec - kv_at - p.k_heads) * p.dim;
            x[u] = i < all && lane_on ? *reinterpret_cast<const uint4 *>(src + d0) : uint4{0, 0, 0, 0};
        }
    };
    // the first vectors are on their way while the rows' places are looked up
    int v0 = blockIdx.y * kPer * U;
    load(v0);
    float qw[8], kw[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 a = p.q_weight && lane_on ? *reinterpret_cast<const float4 *>(p.q_weight + d0 + e) : one;
        const float4 b = p.k_weight && lane_on ? *reinterpret_cast<const float4 *>(p.k_weight + d0 + e) : one;
        qw[e] = a.x, qw[e + 1] = a.y, qw[e + 2] = a.z, qw[e + 3] = a.w;
        kw[e] = b.x, kw[e + 1] = b.y, kw[e + 2] = b.z, kw[e + 3] = b.w;
    }
    for (int j = threadIdx.x; j < half; j += kThreads)
        fraction[j] = turn_fraction(p.freqs[j]);
    if (warp < rows && row0 + warp < p.b.n_rows) {
        const RowAt at = find_pos(p.b, row0 + warp, p.status);
        Place pl{at.live, false, 0, 0};
        if (kStore)
            pl = place_of(p.kv, p.b, at, p.status);
        if ((threadIdx.x & 31) == 0) {
            places[warp] = pl;
            row_pos[warp] = at.live ? at.pos : -1;
        }
    }
    __syncthreads();
    for (int r = 0; r < min(rows, p.b.n_rows - row0); ++r)
        for (int j = threadIdx.x; j < half; j += kThreads) {
            const uint64_t t = fraction[j] * uint64_t(max(row_pos[r], 0)) + 0x80000000ull;
            float s, c;
            sincospif(float(int(t >> 32)) * 0x1p-31f, &s, &c);
            if (!(fabsf(p.freqs[j]) <= kMaxFreq))
                s = c = __int_as_float(0x7fffffff);
            turn[r][j] = make_float2(c, s);
        }
    __syncthreads();
    const int hl = half / 8;                         // lanes of a half
    const int other = l < hl ? l + hl : l < 2 * hl ? l - hl : l;
    const float mean = 1.f / float(p.dim);
    for (; v0 < all; v0 += stride) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = v0 + u * kPer + sub, r = min(p.per_row.quotient(i), rows - 1), vec = i - r * nvec;
            const bool is_q = vec < kv_at, is_v = kStore && vec >= kv_at + p.k_heads;
            const bool here = i < all && lane_on && places[r].live, at = row_pos[r] >= 0;
            float f[8];
            unpack8(x[u], f);
            if (p.q_weight || p.k_weight) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss = fmaf(f[e], f[e], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!is_v && (is_q ? p.q_weight : p.k_weight)) {
                    const float inv = rsqrtf(fmaf(ss, mean, p.eps));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] *= inv * (is_q ? qw[e] : kw[e]);
                }
            }
            if (p.interleaved) {
                if (!is_v && d0 < 2 * half)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 t = turn[r][l * 4 + e];
                        const float a = f[2 * e], b = f[2 * e + 1];
                        f[2 * e] = a * t.x - b * t.y;
                        f[2 * e + 1] = a * t.y + b * t.x;
                    }
            } else if (half) {
                float g[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    g[e] = __shfl_sync(0xffffffffu, f[e], other, G);
                if (!is_v && l < 2 * hl) {
                    const float2 *t = turn[r] + (l < hl ? l : l - hl) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = f[e] * t[e].x + g[e] * (l < hl ? -t[e].y : t[e].y);
                }
            }
            if (kStore && !is_q) {
                // stored below
            } else if (here) {
                const int64_t row = row0 + r;
                uint16_t *dst = is_q ? p.q_out + row * p.ldqo + vec * p.dim : p.k_out + row * p.ldko + (vec - kv_at) * p.dim;
                *reinterpret_cast<uint4 *>(dst + d0) = at ? pack8(f) : uint4{0, 0, 0, 0};
            }
            if (kStore) {
                const Place &pl = places[r];
                const int head = is_v ? vec - kv_at - p.k_heads : vec - kv_at;
                const bool put = here && !is_q && pl.stored;
                uint8_t *dst = (is_v ? p.kv.v : p.kv.k) + (put ? pl.at + head * p.kv.head_stride : 0);
                if (FMT == kKvBf16) {
                    if (put)
                        *reinterpret_cast<uint4 *>(dst + d0 * 2) = pack8(f);
                } else if (__any_sync(0xffffffffu, put)) {
                    float scale;
                    const uint2 code = encode8<FMT == kKvFp8 ? kKvFp8 : kKvInt8, G>(f, scale);
                    if (put) {
                        *reinterpret_cast<uint2 *>(dst + d0) = code;
                        if (l == 0)
                            (is_v ? p.kv.v_scale : p.kv.k_scale)[pl.s_at + head * p.kv.s_head] = scale;
                    }
                }
            }
        }
        if (v0 + stride < all)
            load(v0 + stride);
    }
}

template <int G, int FMT>
cudaError_t launch(RopeParams p, cudaStream_t stream)
{
    // as in kv.cu: several rows a CTA where that leaves two CTAs for each SM, a row cut into
    // parts where rows are few
    const int rows = int(std::min<int64_t>(kMaxRows, std::max<int64_t>(1, p.b.n_rows / 304)));
    const int nvec = p.q_heads + (FMT != kNone ? 2 : 1) * p.k_heads, per = kThreads / G * 4;
    p.per_row = Divider(nvec);
    const dim3 grid(unsigned((p.b.n_rows + rows - 1) / rows), unsigned(rows == 1 ? (nvec + per - 1) / per : 1));
    return start(k_rope<G, FMT>, grid, kThreads, 0, 0, stream, p, rows);
}

template <int FMT>
cudaError_t launch(const RopeParams &p, cudaStream_t stream)
{
    if constexpr (FMT == kNone)                      // a cache has heads of 64 or 128
        if (p.dim > 128)
            return launch<32, FMT>(p, stream);
    return p.dim <= 64 ? launch<8, FMT>(p, stream) : launch<16, FMT>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool store, cudaStream_t stream)
{
    if (!store)
        return launch<kNone>(p, stream);
    switch (p.kv.format) {
    case kKvBf16: return launch<kKvBf16>(p, stream);
    case kKvInt8: return launch<kKvInt8>(p, stream);
    default: return launch<kKvFp8>(p, stream);
    }
}

}  // namespace lora
