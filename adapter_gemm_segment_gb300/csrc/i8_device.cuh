// Device code shared by the 8-bit integer kernels.
#pragma once
#include "common.cuh"

namespace lora {

// a + b = s + e exactly.
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// Two float32 values, worked on by one instruction.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 two_sum2(F2 a, F2 b, F2& e) {
    const F2 s = add2(a, b), bb = sub2(s, a);
    e = add2(sub2(a, sub2(s, bb)), sub2(b, bb));
    return s;
}
// The whole numbers nearest two values of at most 127.5 either way (ties to even): as floats, and as bits whose
// lowest byte is the number (1.5 * 2^23 added: the sum's last bit is 1).
__device__ __forceinline__ F2 nearest2(F2 v, uint32_t& a, uint32_t& b) {
    const F2 magic = f2(12582912.f, 12582912.f), t = add2(v, magic);
    const float2 u = unpack(t);
    a = __float_as_uint(u.x);
    b = __float_as_uint(u.y);
    return sub2(t, magic);
}

// The scale of a row whose largest |x| is amax: the float32 nearest amax / 127.  A row that holds an
// infinity or a NaN has a NaN scale.
__device__ __forceinline__ float i8_scale(float amax) {
    return amax <= 3.402823466e38f ? __fdiv_rn(amax, 127.f) : __uint_as_float(0x7fc00000u);
}

// What a row's elements are divided by: x / s is (x * up) * inv to 2^-23 of itself, where up is a power
// of two that keeps the quotient's parts clear of subnormals; s is then s * up.  inv = 0 gives codes 0
// (a row of zeros, of values too small for a scale, or one that holds an infinity or a NaN).
struct I8Divisor {
    float up, s, inv;
};
__device__ __forceinline__ I8Divisor i8_divisor(float s) {
    I8Divisor d;
    d.up = s < 8.2718e-25f ? 1.2676506e30f : 1.f;  // 2^-80, 2^100
    d.s = s * d.up;
    d.inv = s > 0.f ? __frcp_rn(d.s) : 0.f;
    return d;
}

// The whole number nearest x / s, ties to the even one, where x / s = k + rest is computed to 1.6e-5 (k nearest
// to it) and lies next to the border of two codes: the sign of x - (k +- 1/2) s decides, which one fused
// multiply-add gives exactly, so that the codes are those of the real quotient.
__device__ __forceinline__ int i8_border(float x, float s, int k, float rest) {
    const int side = rest > 0.f ? 1 : -1;
    const float past = fmaf(-(static_cast<float>(k) + 0.5f * side), s, x) * static_cast<float>(side);
    return past > 0.f || (past == 0.f && (k & 1) != 0) ? k + side : k;
}
__device__ __forceinline__ int i8_code(float x, const I8Divisor& d) {
    const float xs = d.inv == 0.f ? 0.f : x * d.up, v = xs * d.inv, k = rintf(v);
    int c = static_cast<int>(k);
    if (fabsf(v - k) > 0.4999f) c = i8_border(xs, d.s, c, v - k);
    return min(max(c, -127), 127);
}

// Four lowest bytes in a word, the first in its lowest.
__device__ __forceinline__ uint32_t i8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Sum of the absolute values of a word's four codes.
__device__ __forceinline__ int i8_abs_sum(uint32_t w) {
    int sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += abs(static_cast<int>(w << (24 - 8 * e)) >> 24);
    return sum;
}

// Four codes of a word as float16, exactly: with the sign bit flipped a byte b stands for b - 128, and
// 0x6400 + b is the float16 1024 + b.
__device__ __forceinline__ uint2 i8_to_f16x4(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A product's value from its whole-number sum: times the scales, one after the other.  The sum is below 2^31, so times
// a scale of up to 2^96 it is a float32 number; of a larger one the other comes first, which then is small or makes an
// infinity that the output is too.  (Downwards nothing is lost: a sum is 0 or at least 1.)
__device__ __forceinline__ bool i8_large(float sx) { return sx > 7.9228163e28f; }
__device__ __forceinline__ float i8_scaled(int sum, float sx, float sw) {
    const bool swap = i8_large(sx);
    return __int2float_rn(sum) * (swap ? sw : sx) * (swap ? sx : sw);
}

// Eight consecutive elements of a row of B (R elements), zeros past R.
template <typename T> __device__ __forceinline__ void load_b8(const T* row, int j, int R, float (&f)[8]);
template <> __device__ __forceinline__ void load_b8<__half>(const __half* row, int j, int R, float (&f)[8]) {
    unpack8<__half>(__ldg(reinterpret_cast<const uint4*>(row + j)), f);
}
template <>
__device__ __forceinline__ void load_b8<__nv_bfloat16>(const __nv_bfloat16* row, int j, int R, float (&f)[8]) {
    unpack8<__nv_bfloat16>(__ldg(reinterpret_cast<const uint4*>(row + j)), f);
}
template <> __device__ __forceinline__ void load_b8<float>(const float* row, int j, int R, float (&f)[8]) {
    if (R % 4 == 0) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + j));
        const float4 b = j + 4 < R ? __ldg(reinterpret_cast<const float4*>(row + j + 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = j + e < R ? __ldg(row + j + e) : 0.f;
    }
}

}  // namespace lora
