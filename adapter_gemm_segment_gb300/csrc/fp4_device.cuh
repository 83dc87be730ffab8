// Device code shared by the 4-bit kernels.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace lora {

// Quantisation of a block of 32 held by four neighbouring lanes, 8 elements each.  With E the biased
// float32 exponent of the block's largest |x| the scale byte is max(E - 2, 0): the largest element
// then lies in [4, 8) times the scale, of which [6, 8) saturates at 6.  Multiplying by the power of
// two 2^(127 - byte) is exact wherever the result does not round to zero anyway, so the rounding to
// e2m1 (to nearest, ties to even) is the only one.  E = 255, an infinity or a NaN, gives the NaN scale
// and codes 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t E) { return E == 255 ? 255u : E > 2 ? E - 2 : 0u; }

// 8 float32 values times 2^(127 - byte), as codes (0 with the NaN scale).
__device__ __forceinline__ uint32_t codes8(const float (&f)[8], uint32_t byte) {
    const float k = __uint_as_float((254u - min(byte, 253u)) << 23);  // 2^-125 .. 2^127
    uint32_t c;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c)
        : "f"(f[0] * k), "f"(f[1] * k), "f"(f[2] * k), "f"(f[3] * k), "f"(f[4] * k), "f"(f[5] * k), "f"(f[6] * k),
          "f"(f[7] * k));
    return byte == 255 ? 0u : c;
}

// A lane's 8 elements of a row: packed for the 16-bit types, as they are for float32.
template <typename T> struct Raw8 {
    uint4 v;
};
template <> struct Raw8<float> {
    float4 a, b;
};
// Largest |x| of two packed pairs (a NaN wins), without and with the absolute values taken.
template <typename T> __device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t max_abs2<__nv_bfloat16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t max_abs2<__half>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.NaN.f16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
template <typename T> __device__ __forceinline__ uint32_t exponent16(uint32_t top);  // biased float32 exponent
template <> __device__ __forceinline__ uint32_t exponent16<__nv_bfloat16>(uint32_t top) { return top >> 7; }
template <> __device__ __forceinline__ uint32_t exponent16<__half>(uint32_t top) {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top)))) >> 23;
}

// 8 packed 16-bit values times 2^(127 - byte), as codes (0 with the NaN scale).
template <typename T> __device__ __forceinline__ uint32_t codes8_packed(const uint4& v, uint32_t byte);
template <> __device__ __forceinline__ uint32_t codes8_packed<__nv_bfloat16>(const uint4& v, uint32_t byte) {
    // bf16 times bf16 to float32 in one instruction each; the addend -0 keeps the sign of -0
    const uint32_t k = (254u - min(byte, 253u)) << 7;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 l, h, k;\n\t"
            "mov.b32 {l, h}, %2;\n\t"
            "cvt.u16.u32 k, %3;\n\t"
            "fma.rn.f32.bf16 %0, l, k, 0f80000000;\n\t"
            "fma.rn.f32.bf16 %1, h, k, 0f80000000;\n\t}"
            : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
            : "r"(w[i]), "r"(k));
    uint32_t c;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return byte == 255 ? 0u : c;
}
template <> __device__ __forceinline__ uint32_t codes8_packed<__half>(const uint4& v, uint32_t byte) {
    // The factor is 2^-13 .. 2^26 (an all-zero block's is not needed), in two that f16 holds.  A
    // product that underflows was far below the smallest code.
    const int K = min(127 - static_cast<int>(byte), 26), k1 = min(K, 14);
    const uint32_t a = static_cast<uint32_t>(k1 + 15) * 0x04000400u, b = static_cast<uint32_t>(K - k1 + 15) * 0x04000400u;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w[i]), *reinterpret_cast<const __half2*>(&a)),
                                  *reinterpret_cast<const __half2*>(&b));
        m[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    uint32_t c;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c)
        : "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3]));
    return byte == 255 ? 0u : c;
}

// Quantises NR (even) rows at once: codes[j] are this lane's 8 codes of row j, words[j] the four scale
// bytes of row j's 128 columns held by this half-warp (the same in each of its lanes).
template <typename T, int NR>
__device__ __forceinline__ void quantise_rows(const Raw8<T> (&x)[NR], uint32_t (&codes)[NR], uint32_t (&words)[NR],
                                              int lane) {
    uint32_t byte[NR];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < NR; j += 2) {
            const uint4 &u = x[j].v, &v = x[j + 1].v;
            const uint32_t a = max_abs2<T>(max_abs2<T>(u.x, u.y), max_abs2<T>(u.z, u.w));
            const uint32_t b = max_abs2<T>(max_abs2<T>(v.x, v.y), max_abs2<T>(v.z, v.w));
            uint32_t m = max_abs2<T>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));  // two rows
            m = max_abs2<T>(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_abs2<T>(m, __shfl_xor_sync(0xffffffffu, m, 2));
            byte[j] = scale_byte(exponent16<T>(m & 0xffffu));
            byte[j + 1] = scale_byte(exponent16<T>(m >> 16));
            codes[j] = codes8_packed<T>(u, byte[j]);
            codes[j + 1] = codes8_packed<T>(v, byte[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const float f[8] = {x[j].a.x, x[j].a.y, x[j].a.z, x[j].a.w, x[j].b.x, x[j].b.y, x[j].b.z, x[j].b.w};
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            byte[j] = scale_byte(m >> 23);
            codes[j] = codes8(f, byte[j]);
        }
    }
    // byte i of a row's word comes from the lanes of block i; two rows travel together
#pragma unroll
    for (int j = 0; j < NR; j += 2) {
        uint32_t w = (byte[j] | byte[j + 1] << 16) << (8 * ((lane >> 2) & 1));
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 8);
        const uint32_t lo = (lane & 8) ? o : w, hi = (lane & 8) ? w : o;
        words[j] = __byte_perm(lo, hi, 0x5410);
        words[j + 1] = __byte_perm(lo, hi, 0x7632);
    }
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
// The largest |s| that a 16-bit part holds: float16 takes 65520 and more for an infinity, bfloat16 has float32's range.
template <typename T> __device__ __forceinline__ bool too_large(float s) { return false; }
template <> __device__ __forceinline__ bool too_large<__half>(float s) {
    const float a = fabsf(s);
    return a >= 65520.f && a <= 3.402823466e38f;
}
// Two float32 values in the 16-bit type, the first in the low half, and back.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Eight shrink values for the tensor cores: s = hi + lo, each of the 16-bit type, which multiply the same
// elements of B.  The two carry s to 2^-16 of itself in bfloat16, 2^-22 (and no nearer than 2^-25) in float16;
// hi alone would lose as much as the rounding of y does.  An infinity or NaN stays in hi.  What float16 does not
// hold is left out (both 0) and the result true: nonfinite_dot8 adds it.
template <typename T> __device__ __forceinline__ bool split8(const float (&s)[8], uint4& hi, uint4& lo) {
    hi = make_uint4(pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]), pack2<T>(s[4], s[5]), pack2<T>(s[6], s[7]));
    float h[8];
    unpack8<T>(hi, h);
    lo = make_uint4(pack2<T>(s[0] - h[0], s[1] - h[1]), pack2<T>(s[2] - h[2], s[3] - h[3]),
                    pack2<T>(s[4] - h[4], s[5] - h[5]), pack2<T>(s[6] - h[6], s[7] - h[7]));
    if (!nonfinite8<T>(hi)) return false;
    lo = finite8<T>(lo);  // (inf - inf, NaN)
    alignas(16) T v[8];
    *reinterpret_cast<uint4*>(v) = hi;
    bool left_out = false;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (too_large<T>(s[e])) {
            v[e] = from_f32<T>(0.f);
            left_out = true;
        }
    hi = *reinterpret_cast<const uint4*>(v);
    return left_out;
}
// Sum over b times s of what the blocks leave out: b an infinity or NaN (finite8), or s too large (split8).
template <typename T> __device__ __forceinline__ float nonfinite_dot8(const uint4& b, const float (&s)[8], float acc) {
    float bf[8];
    unpack8<T>(b, bf);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if ((__float_as_uint(bf[e]) & 0x7f800000u) == 0x7f800000u || too_large<T>(s[e])) acc = fmaf(bf[e], s[e], acc);
    return acc;
}

// Eight shrink values summed over their K parts.
__device__ __forceinline__ void sum_parts8(const float* s, int parts, size_t stride, float (&v)[8]) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int k0 = 0; k0 < parts; k0 += 4) {  // four parts' loads in flight
        float4 c[4], d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4* p = reinterpret_cast<const float4*>(s + min(k0 + k, parts - 1) * stride);
            c[k] = __ldcg(p);
            d[k] = __ldcg(p + 1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k0 + k < parts) {
                a.x += c[k].x, a.y += c[k].y, a.z += c[k].z, a.w += c[k].w;
                b.x += d[k].x, b.y += d[k].y, b.z += d[k].z, b.w += d[k].w;
            }
    }
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

}  // namespace lora
