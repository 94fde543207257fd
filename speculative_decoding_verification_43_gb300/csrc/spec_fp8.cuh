// Values in 8 bits (e4m3: sign, four bits of exponent, three of mantissa; largest 448, least 2^-9, no infinity)
// and the scales of a cache that holds them.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace spec {

// The least scale that is set: a block of zeros has it, and so have values below 2^-52.
constexpr int kLeastScaleLog2 = -60;

// Two e4m3 in the lower half of a word (the first in the lower byte) as 16-bit floats; exact.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return h;
}
// The same as fp32.
__device__ __forceinline__ float2 e4m3_to_float2(uint16_t v) {
    const uint32_t h = e4m3_to_half2(v);
    return __half22float2(reinterpret_cast<const __half2 &>(h));
}
__device__ __forceinline__ float4 e4m3_to_float4(uint32_t v) {
    const float2 a = e4m3_to_float2(static_cast<uint16_t>(v)), b = e4m3_to_float2(static_cast<uint16_t>(v >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
}
// Two fp32 rounded to e4m3, `lo` in the lower byte. Beyond the largest: the largest; NaN: NaN.
__device__ __forceinline__ uint16_t to_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The same to e5m2 (three bits, least 2^-16).
__device__ __forceinline__ uint16_t to_e5m2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four weights (16-bit floats' range, below 61440) as sums of three e5m2 each; the words have the first weight in
// the lowest byte. e5m2 is the upper byte of a 16-bit float, so: the weight is rounded to a 16-bit float (11
// bits), its upper byte after rounding is the first part (three bits), what that leaves, which is a multiple of
// the 16-bit float's last place and at most four of the first part's places off, gives the second in the same way
// and the third. Three bits each hold it whole, down to the least e5m2, 2^-16.
__device__ __forceinline__ void split_e5m2(float a, float b, float c, float d, uint32_t (&w)[3]) {
    __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t u = (reinterpret_cast<const uint32_t &>(x) + 0x00800080u) & 0xff00ff00u,
                       v = (reinterpret_cast<const uint32_t &>(y) + 0x00800080u) & 0xff00ff00u;
        w[i] = __byte_perm(u, v, 0x7531);
        if (i < 2) {
            x = __hsub2(x, reinterpret_cast<const __half2 &>(u));
            y = __hsub2(y, reinterpret_cast<const __half2 &>(v));
        }
    }
}
// The same, and what the 16-bit float and its three parts leave of the weight, times 2^SHIFT, in three more.
template <int SHIFT>
__device__ __forceinline__ void split_e5m2_wide(float a, float b, float c, float d, uint32_t (&w)[6]) {
    __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
    const float2 fx = __half22float2(x), fy = __half22float2(y);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t u = (reinterpret_cast<const uint32_t &>(x) + 0x00800080u) & 0xff00ff00u,
                       v = (reinterpret_cast<const uint32_t &>(y) + 0x00800080u) & 0xff00ff00u;
        w[i] = __byte_perm(u, v, 0x7531);
        x = __hsub2(x, reinterpret_cast<const __half2 &>(u));
        y = __hsub2(y, reinterpret_cast<const __half2 &>(v));
    }
    const float2 gx = __half22float2(x), gy = __half22float2(y);  // (0 but for the smallest weights)
    constexpr float times = static_cast<float>(1 << SHIFT);
    uint32_t more[3];
    split_e5m2((a - fx.x + gx.x) * times, (b - fx.y + gx.y) * times, (c - fy.x + gy.x) * times, (d - fy.y + gy.y) * times, more);
#pragma unroll
    for (int i = 0; i < 3; ++i) w[3 + i] = more[i];
}
// An e5m2 in the upper byte of the lower half of a word.
__device__ __forceinline__ float e5m2_to_float(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 8)));
}

// The least power of two s with top <= 448 s, at least 2^kLeastScaleLog2. top is finite and not negative:
// 448 = 1.75 * 2^8, so s = 2^(e-8) for top = f 2^e with 1 <= f <= 1.75, and 2^(e-7) for f above.
__device__ __forceinline__ float e4m3_scale(float top) {
    const uint32_t bits = __float_as_uint(top);
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, kLeastScaleLog2) + 127) << 23);
}

}  // namespace spec
