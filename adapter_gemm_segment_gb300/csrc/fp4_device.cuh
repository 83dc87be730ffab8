// Device code shared by the 4-bit kernels.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace lora {

// Two float32 values to a byte of two e2m1 codes (lo in the low half), round to nearest even,
// saturating.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "cvt.u16.u8 %0, t;\n\t}"
        : "=h"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// The codes of a lane's 8 elements and the scale byte of its block; four neighbouring lanes hold a
// block of 32.  With E the biased float32 exponent of the block's largest |x| the byte is
// max(E - 2, 0): the largest element then lies in [4, 8) times the scale, of which [6, 8) saturates
// at 6.  2^(127 - byte) and the products with it are exact, so the rounding to e2m1 is the only one.
__device__ __forceinline__ uint32_t quantise8(const float (&f)[8], uint32_t& scale) {
    // |x| as an integer orders like |x|, with infinities and NaNs on top
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t E = m >> 23;
    if (E == 255) {
        scale = 255;
        return 0;
    }
    scale = E > 2 ? E - 2 : 0;
    const float k = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale): 2^-125 .. 2^127
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) c |= cvt_e2m1x2(f[2 * e] * k, f[2 * e + 1] * k) << (8 * e);
    return c;
}

// The four scale bytes of a half-warp's 128 columns as one word (every lane of the half gets it).
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, int lane) {
    const int h = lane & 16;
    uint32_t w = __shfl_sync(0xffffffffu, scale, h);
    w |= __shfl_sync(0xffffffffu, scale, h + 4) << 8;
    w |= __shfl_sync(0xffffffffu, scale, h + 8) << 16;
    w |= __shfl_sync(0xffffffffu, scale, h + 12) << 24;
    return w;
}

// Whether any of 8 packed 16-bit values is an infinity or a NaN.
template <typename T> __device__ __forceinline__ bool nonfinite8(const uint4& v);
template <> __device__ __forceinline__ bool nonfinite8<__nv_bfloat16>(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);
    return bad != 0;
}
template <> __device__ __forceinline__ bool nonfinite8<__half>(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= __vcmpeq2(w[i] & 0x7c007c00u, 0x7c007c00u);
    return bad != 0;
}
// The same values with the infinities and NaNs replaced by zeros.
template <typename T> __device__ __forceinline__ uint4 finite8(const uint4& v) {
    const uint32_t mask = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    return make_uint4(v.x & ~__vcmpeq2(v.x & mask, mask), v.y & ~__vcmpeq2(v.y & mask, mask),
                      v.z & ~__vcmpeq2(v.z & mask, mask), v.w & ~__vcmpeq2(v.w & mask, mask));
}
// Sum over the infinities and NaNs among b's 8 values of b times s (the part finite8 leaves out).
template <typename T> __device__ __forceinline__ float nonfinite_dot8(const uint4& b, const uint4& s, float acc) {
    float bf[8], sf[8];
    unpack8<T>(b, bf);
    unpack8<T>(s, sf);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if ((__float_as_uint(bf[e]) & 0x7f800000u) == 0x7f800000u) acc = fmaf(bf[e], sf[e], acc);
    return acc;
}

}  // namespace lora
