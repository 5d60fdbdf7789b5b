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

// The codes of one vector held 8 elements (bf16) a lane by LANES consecutive lanes, and
// its scale (the same in all of them).  Every lane of the warp calls it.
template <int FMT, int LANES>
__device__ __forceinline__ uint2 encode8(uint4 x, float &scale)
{
    constexpr float T = code_top<FMT>();
    __nv_bfloat162 m;
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x);
        m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        const uint32_t t = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t *>(&m), o);
        m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162 *>(&t));
    }
    const float top = __bfloat162float(__hmax_nan(m.x, m.y));
    if (!(top < INFINITY)) {
        scale = __int_as_float(0x7fffffff);
        return make_uint2(0, 0);
    }
    scale = __fdiv_rn(top, T);
    const float d = scale > 0.f ? scale : 1.f;
    float f[8];
    unpack8(x, f);
    // The code is that of the quotient f / d (rounded to fp32).  A product with 1 / d is
    // within 2^-21 of it, so where both ends of that range give the same code it is the
    // code; only a lane with an element next to the middle between two codes (or with a
    // scale near the ends of fp32) takes the divisions.
    const float r = __fdividef(1.f, d);
    uint32_t lo[2], hi[2];
    if (FMT == kKvInt8) {
        // added to 1.5 * 2^23, a number rounds to an integer that the low bits hold
        uint32_t a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = f[e] * r;
            a[e] = __float_as_uint(fmaf(z, 1.f - 0x1p-21f, 12582912.f));
            b[e] = __float_as_uint(fmaf(z, 1.f + 0x1p-21f, 12582912.f));
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            lo[w] = __byte_perm(__byte_perm(a[4 * w], a[4 * w + 1], 0x0040), __byte_perm(a[4 * w + 2], a[4 * w + 3], 0x0040), 0x5410);
            hi[w] = __byte_perm(__byte_perm(b[4 * w], b[4 * w + 1], 0x0040), __byte_perm(b[4 * w + 2], b[4 * w + 3], 0x0040), 0x5410);
        }
    } else {
        uint16_t a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float z0 = f[2 * e] * r, z1 = f[2 * e + 1] * r;
            a[e] = __nv_cvt_float2_to_fp8x2(make_float2(z0 * (1.f - 0x1p-21f), z1 * (1.f - 0x1p-21f)), __NV_SATFINITE, __NV_E4M3);
            b[e] = __nv_cvt_float2_to_fp8x2(make_float2(z0 * (1.f + 0x1p-21f), z1 * (1.f + 0x1p-21f)), __NV_SATFINITE, __NV_E4M3);
        }
        lo[0] = a[0] | uint32_t(a[1]) << 16, lo[1] = a[2] | uint32_t(a[3]) << 16;
        hi[0] = b[0] | uint32_t(b[1]) << 16, hi[1] = b[2] | uint32_t(b[3]) << 16;
    }
    if (lo[0] != hi[0] || lo[1] != hi[1] || !(d > 1e-30f && d < 1e30f)) {
        hi[0] = hi[1] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // a scale that was rounded down puts the largest element past the top
            const float z = fminf(fmaxf(__fdiv_rn(f[e], d), -T), T);
            const uint32_t c = FMT == kKvInt8 ? uint32_t(__float2int_rn(z)) & 0xffu
                                              : uint32_t(__nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3));
            hi[e / 4] |= c << (8 * (e % 4));
        }
    }
    return make_uint2(hi[0], hi[1]);
}

// The values of 8 codes (without the scale); exact in bf16, fp16 and fp32.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 c, float f[8])
{
    const uint32_t w[2] = {c.x, c.y};
    if (FMT == kKvInt8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = float(int8_t(w[e / 4] >> (8 * (e % 4))));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                __nv_fp8x2_storage_t(w[e / 2] >> (16 * (e % 2))), __NV_E4M3);
            const float2 t = __half22float2(__half2(h));
            f[2 * e] = t.x;
            f[2 * e + 1] = t.y;
        }
    }
}

}  // namespace lora
