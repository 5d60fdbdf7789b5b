// 8-bit codes of the key/value cache.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv.h"
#include "ptx.cuh"

namespace lora {

template <int FMT>
__device__ __forceinline__ constexpr float code_top()
{
    return FMT == kKvInt8 ? 127.f : 448.f;
}

// The codes of one vector held 16 elements (bf16) a lane by LANES consecutive lanes, and
// its scale (the same in all of them).  Every lane of the warp calls it.
template <int FMT, int LANES>
__device__ __forceinline__ uint4 encode16(const uint4 x[2], float &scale)
{
    constexpr float T = code_top<FMT>();
    const uint32_t *xw = reinterpret_cast<const uint32_t *>(x);
    __nv_bfloat162 m;
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(x);
        m = __habs2(h[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e)
            m = __hmax2_nan(m, __habs2(h[e]));
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        const uint32_t t = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t *>(&m), o);
        m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162 *>(&t));
    }
    const float top = __bfloat162float(__hmax_nan(m.x, m.y));
    uint32_t lo[4], hi[4];
    if (!(top < INFINITY)) {
        scale = __int_as_float(0x7fffffff);
        return make_uint4(0, 0, 0, 0);
    }
    scale = __fdiv_rn(top, T);
    const float d = scale > 0.f ? scale : 1.f;
    // The code is that of the quotient f / d (rounded to fp32).  Products with 1 / d taken
    // 2^-21 too small and too large lie on both sides of it, so where they give the same
    // code it is the code; only a lane with an element next to the middle between two codes
    // (or with a scale near the ends of fp32) takes the divisions.
    const float r = __fdividef(1.f, d), r0 = r * (1.f - 0x1p-21f), r1 = r * (1.f + 0x1p-21f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f[2 * e] = __uint_as_float(xw[2 * w + e] << 16);
            f[2 * e + 1] = __uint_as_float(xw[2 * w + e] & 0xffff0000u);
        }
        if (FMT == kKvInt8) {
            // added to 1.5 * 2^23, a number rounds to an integer that the low bits hold
            uint32_t a[4], b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = __float_as_uint(fmaf(f[e], r0, 12582912.f));
                b[e] = __float_as_uint(fmaf(f[e], r1, 12582912.f));
            }
            lo[w] = __byte_perm(__byte_perm(a[0], a[1], 0x0040), __byte_perm(a[2], a[3], 0x0040), 0x5410);
            hi[w] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        } else {
            auto two = [&](int e, float q) {
                return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(f[e] * q, f[e + 1] * q), __NV_SATFINITE, __NV_E4M3));
            };
            lo[w] = two(0, r0) | two(2, r0) << 16;
            hi[w] = two(0, r1) | two(2, r1) << 16;
        }
    }
    const uint32_t differ = (lo[0] ^ hi[0]) | (lo[1] ^ hi[1]) | (lo[2] ^ hi[2]) | (lo[3] ^ hi[3]);
    if (differ || !(d > 1e-30f && d < 1e30f)) {
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
            uint32_t c = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t pair = w == 0 ? xw[e / 2] : w == 1 ? xw[2 + e / 2] : w == 2 ? xw[4 + e / 2] : xw[6 + e / 2];
                const float f = __uint_as_float(e & 1 ? pair & 0xffff0000u : pair << 16);
                // a scale that was rounded down puts the largest element past the top
                const float z = fminf(fmaxf(__fdiv_rn(f, d), -T), T);
                const uint32_t code = FMT == kKvInt8 ? uint32_t(__float2int_rn(z)) & 0xffu
                                                     : uint32_t(__nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3));
                c |= code << (8 * e);
            }
            hi[0] = w == 0 ? c : hi[0], hi[1] = w == 1 ? c : hi[1], hi[2] = w == 2 ? c : hi[2], hi[3] = w == 3 ? c : hi[3];
        }
    }
    return make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// Four codes (bytes 0..3) as bf16, in order; exact.
template <int FMT>
__device__ __forceinline__ uint2 widen4(uint32_t r)
{
    uint2 y;
    if (FMT == kKvInt8) {
        // 128 + the low seven bits, less 128 or (sign bit) 256
        const uint32_t a = __byte_perm(r, 0, 0x4140), b = __byte_perm(r, 0, 0x4342);
        const uint32_t a1 = (a & 0x007f007fu) | 0x43004300u, a0 = (a & 0x00800080u) | 0x43004300u;
        const uint32_t b1 = (b & 0x007f007fu) | 0x43004300u, b0 = (b & 0x00800080u) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y.x) : "r"(a1), "r"(a0));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y.y) : "r"(b1), "r"(b0));
    } else {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(r & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(r >> 16), __NV_E4M3);
        const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
        const __nv_bfloat162 ya = __floats2bfloat162_rn(fa.x, fa.y), yb = __floats2bfloat162_rn(fb.x, fb.y);
        y.x = *reinterpret_cast<const uint32_t *>(&ya);
        y.y = *reinterpret_cast<const uint32_t *>(&yb);
    }
    return y;
}

// What the attention kernels' products take of a code: kCodeUnit times it.
template <int FMT>
constexpr float kCodeUnit = FMT == kKvInt8 ? 0x1p-6f : 1.f;

// Four codes (bytes 0..3) as bf16, in order, times kCodeUnit; exact.
template <int FMT>
__device__ __forceinline__ uint2 widen4_unit(uint32_t r)
{
    if (FMT != kKvInt8)
        return widen4<FMT>(r);
    // code + 128 as a byte is a bf16 of (code + 128) 2^-133; times 2^127, less 2, it is
    // code 2^-6, in one operation that does not load the integer pipe
    const uint32_t t = r ^ 0x80808080u, a = __byte_perm(t, 0, 0x4140), b = __byte_perm(t, 0, 0x4342);
    uint2 y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y.x) : "r"(a), "r"(0x7f007f00u), "r"(0xc000c000u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y.y) : "r"(b), "r"(0x7f007f00u), "r"(0xc000c000u));
    return y;
}

// scale times 16 codes, rounded to bf16 once.
template <int FMT>
__device__ __forceinline__ void decode16(uint4 c, float scale, uint4 y[2])
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 v = widen4<FMT>(w[i]);
        h[2 * i] = __floats2bfloat162_rn(__uint_as_float(v.x << 16) * scale, __uint_as_float(v.x & 0xffff0000u) * scale);
        h[2 * i + 1] = __floats2bfloat162_rn(__uint_as_float(v.y << 16) * scale, __uint_as_float(v.y & 0xffff0000u) * scale);
    }
}

}  // namespace lora
