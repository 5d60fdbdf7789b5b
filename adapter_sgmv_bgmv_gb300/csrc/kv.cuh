// 8-bit codes of the key/value cache.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv.h"

namespace lora {

template <int FMT>
__device__ __forceinline__ constexpr float code_top()
{
    return FMT == kKvInt8 ? 127.f : 448.f;
}

// The codes of one vector held 8 elements a lane by LANES consecutive lanes, and its
// scale (the same in all of them).  Every lane of the warp calls it.
template <int FMT, int LANES>
__device__ __forceinline__ uint2 encode8(const float f[8], float &scale)
{
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        finite = finite && fabsf(f[e]) < INFINITY;
        top = fmaxf(top, fabsf(f[e]));
    }
    if (!finite)
        top = INFINITY;                     // fmaxf would drop a NaN
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    constexpr float T = code_top<FMT>();
    if (!(top < INFINITY)) {
        scale = __int_as_float(0x7fffffff);
        return make_uint2(0, 0);
    }
    scale = __fdiv_rn(top, T);
    const float d = scale > 0.f ? scale : 1.f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // a scale rounded down can put the largest element past the top
        const float z = fminf(fmaxf(__fdiv_rn(f[e], d), -T), T);
        uint32_t c;
        if (FMT == kKvInt8)
            c = uint32_t(__float2int_rn(z)) & 0xffu;
        else
            c = __nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3);
        w[e / 4] |= c << (8 * (e % 4));
    }
    return make_uint2(w[0], w[1]);
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
