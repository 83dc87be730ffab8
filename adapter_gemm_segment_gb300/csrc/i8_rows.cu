// Rows of 8-bit integer matrices: quantisation, reading back, and the root-mean-square norm that writes its
// output so.
//
// Stored form (lora.h): a row x becomes codes c and a scale s, s = max|x| / 127 rounded to float32 and c
// the whole number nearest x / s (ties to even).  Codes are those of the real quotient, not of a rounded
// one: a 16384 x 4096 batch has hundreds of elements whose float32 quotient rounds onto the border of two
// codes (and where a bfloat16 row's largest value is even, one element in 200 lies that close), and with
// them equal inputs would not give equal bytes on every path.
//
// Every kernel here moves its rows once and is bound by memory, below a few MB by the launch.  16384 x 4096
// bfloat16, us (at the copy rate): quantise 42 (30), read back 32 (30), norm with residual, y and codes 112 (90).  The
// quantiser's and the norm's instructions fill 66 and 68 % of the issue slots; the float32 quantiser's a third: its
// vectors are 32 bytes, so that a warp's 16-byte accesses lie 32 apart (8191 x 11008: 101 us, 67 at the copy rate).
#include <algorithm>
#include <climits>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "i8_device.cuh"
#include "kernels.h"

namespace lora {

constexpr float kFltMax = 3.402823466e38f;
constexpr int kRowThreads = 512;             // at most, a row
constexpr size_t kRowSmem = 200 * 1024;      // a row is kept in shared memory up to this size

// Eight elements of a row as they are in memory.
template <typename T> struct Raw {
    uint4 v;
};
template <> struct Raw<float> {
    uint4 v, w;
};
template <typename T> __device__ __forceinline__ void to8(const Raw<T>& r, float (&f)[8]) { unpack8<T>(r.v, f); }
template <> __device__ __forceinline__ void to8<float>(const Raw<float>& r, float (&f)[8]) {
    f[0] = __uint_as_float(r.v.x), f[1] = __uint_as_float(r.v.y), f[2] = __uint_as_float(r.v.z), f[3] = __uint_as_float(r.v.w);
    f[4] = __uint_as_float(r.w.x), f[5] = __uint_as_float(r.w.y), f[6] = __uint_as_float(r.w.z), f[7] = __uint_as_float(r.w.w);
}
// T(a + b): the sum of two 16-bit numbers rounded once.
template <typename T> __device__ __forceinline__ uint32_t add_word(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t add_word<float>(uint32_t a, uint32_t b) {
    return __float_as_uint(__fadd_rn(__uint_as_float(a), __uint_as_float(b)));
}
template <> __device__ __forceinline__ uint32_t add_word<__half>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t add_word<__nv_bfloat16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T> __device__ __forceinline__ void add_raw(Raw<T>& a, const Raw<T>& b) {
    a.v = make_uint4(add_word<T>(a.v.x, b.v.x), add_word<T>(a.v.y, b.v.y), add_word<T>(a.v.z, b.v.z), add_word<T>(a.v.w, b.v.w));
    if constexpr (sizeof(T) == 4)
        a.w = make_uint4(add_word<T>(a.w.x, b.w.x), add_word<T>(a.w.y, b.w.y), add_word<T>(a.w.z, b.w.z), add_word<T>(a.w.w, b.w.w));
}

// Vector i of the row's G threads is thread i % G's: with VEC elements 8 i .. + 7, moved 16 bytes at a time;
// without (rows off 16-byte boundaries) element e is 8 (i - i % G) + e G + i % G, so that neighbouring threads
// still touch neighbours.
template <typename T, bool VEC> struct RowPart {
    static __device__ __forceinline__ int at(int i, int e, int tid, int G) { return VEC ? 8 * i + e : 8 * (i - tid) + e * G + tid; }
    // zeros past cols
    static __device__ __forceinline__ Raw<T> load(const T* row, int cols, int i, int tid, int G) {
        Raw<T> r;
        const int k = at(i, 0, tid, G);
        if (VEC && k + 8 <= cols) {
            memcpy(&r.v, __builtin_assume_aligned(row + k, 16), 16);
            if constexpr (sizeof(T) == 4) memcpy(&r.w, __builtin_assume_aligned(row + k + 4, 16), 16);
        } else {
            alignas(16) T v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                v[e] = j < cols ? row[j] : from_f32<T>(0.f);
            }
            memcpy(&r, v, sizeof(r));
        }
        return r;
    }
    static __device__ __forceinline__ void store(T* row, int cols, int i, int tid, int G, const Raw<T>& r) {
        const int k = at(i, 0, tid, G);
        if (VEC && k + 8 <= cols) {
            *reinterpret_cast<uint4*>(row + k) = r.v;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(row + k + 4) = r.w;
        } else {
            alignas(16) T v[8];
            memcpy(v, &r, sizeof(r));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                if (j < cols) row[j] = v[e];
            }
        }
    }
    // codes, four a word (0 past cols, up to pitch)
    static __device__ __forceinline__ void store_words(int8_t* row, int pitch, int i, int tid, int G, uint2 w) {
        const int k = at(i, 0, tid, G);
        if (VEC) {
            if (k < pitch) *reinterpret_cast<uint2*>(row + k) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                if (j < pitch) row[j] = static_cast<int8_t>((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
            }
        }
    }
    // codes (lowest bytes of c)
    static __device__ __forceinline__ void store_codes(int8_t* row, int pitch, int i, int tid, int G, const uint32_t (&c)[8]) {
        const int k = at(i, 0, tid, G);
        if (VEC) {
            if (k < pitch)
                *reinterpret_cast<uint2*>(row + k) =
                    make_uint2(i8_pack4(c[0], c[1], c[2], c[3]), i8_pack4(c[4], c[5], c[6], c[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                if (j < pitch) row[j] = static_cast<int8_t>(c[e]);
            }
        }
    }
    // the same as float16
    static __device__ __forceinline__ void store_codes(__half* row, int pitch, int i, int tid, int G, const uint32_t (&c)[8]) {
        const int k = at(i, 0, tid, G);
        if (VEC) {
            const uint2 a = i8_to_f16x4(i8_pack4(c[0], c[1], c[2], c[3])), b = i8_to_f16x4(i8_pack4(c[4], c[5], c[6], c[7]));
            if (k < pitch) *reinterpret_cast<uint4*>(row + k) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                if (j < pitch) row[j] = __int2half_rn(static_cast<int8_t>(c[e]));
            }
        }
    }
};
template <typename T> __device__ __forceinline__ Raw<T> from8(const float (&f)[8]) {
    alignas(16) T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_f32<T>(f[e]);
    Raw<T> r;
    memcpy(&r, v, sizeof(r));
    return r;
}

// Not 0 where an element is not.
template <typename T> __device__ __forceinline__ uint32_t any_bits(const Raw<T>& r) {
    const uint32_t b = r.v.x | r.v.y | r.v.z | r.v.w;
    if constexpr (sizeof(T) == 4) return (b | r.w.x | r.w.y | r.w.z | r.w.w) & 0x7fffffffu;
    return b & 0x7fff7fffu;
}

// A row's place in a launch: G threads (a warp, several rows a CTA, or the CTA), its vectors, and whether they
// are kept in shared memory between the two passes over the row (else the second reads them again).  Registers
// would hold a quarter as many rows on an SM (16384 x 4096 bfloat16 quantised: 102 us).
struct RowPlan {
    int G, vecs, keep;
};

// The larger; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
struct MaxPair {  // a largest |value| and what its float32 left off
    float hi, lo;
};
__device__ __forceinline__ MaxPair max_pair(MaxPair a, MaxPair b) {
    // NaN wins (comparisons with it are false)
    const bool take = !(b.hi <= a.hi) || (b.hi == a.hi && b.lo > a.lo);
    return a.hi != a.hi ? a : take ? b : a;
}
// The largest of a row's warps' tops.
__device__ __forceinline__ void row_peak(int top, int G, int tid, float* red, int* peak) {
    if (G > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = __int_as_float(top);
        __syncthreads();
        for (int w = 0; w < G / 32; ++w) top = max(top, __float_as_int(red[w]));
    }
    if (tid == 0) *peak = top;
}

// ---- quantise ----------------------------------------------------------------------------------------
// One row by its G threads.  U: vectors whose loads are in flight together.  Codes go to out as bytes or float16.
// peak (nullable): at least the largest sum of |code| over an aligned block of 256 (see I8Rows::peak).
template <typename T, int U, bool VEC, typename C>
__device__ __forceinline__ void quantise_row(const T* row, int cols, int pitch, const RowPlan& pl, int tid, Raw<T>* kept,
                                             float* red, float* scale, C* out, int* peak) {
    using Part = RowPart<T, VEC>;
    const int G = pl.G;
    float m = 0.f;
    for (int i0 = tid; i0 < pl.vecs; i0 += U * G) {
        Raw<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * G < pl.vecs) v[u] = Part::load(row, cols, i0 + u * G, tid, G);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * G >= pl.vecs) break;
            if (pl.keep) kept[i0 + u * G] = v[u];
            float f[8];
            to8(v[u], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[e]));
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        for (int w = 0; w < G / 32; ++w) m = max_nan(m, red[w]);
    }
    const float s = i8_scale(m);
    if (tid == 0) *scale = s;
    const I8Divisor d = i8_divisor(s);
    const bool plain = d.up == 1.f && d.inv != 0.f;
    int top = VEC ? 0 : 256 * 127;  // (without VEC a warp's codes are no block)
#pragma unroll 1
    for (int i = tid; i < pl.vecs; i += G) {
        float f[8];
        to8(pl.keep ? kept[i] : Part::load(row, cols, i, tid, G), f);
        uint32_t c[8];
        if (plain) {
            float rest[8], far = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const F2 v = mul2(f2(f[e], f[e + 1]), f2(d.inv, d.inv));
                const float2 t = unpack(sub2(v, nearest2(v, c[e], c[e + 1])));
                rest[e] = t.x, rest[e + 1] = t.y;
                far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
            }
            if (far > 0.4999f) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (fabsf(rest[e]) > 0.4999f) c[e] = i8_border(f[e], d.s, static_cast<int8_t>(c[e]), rest[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = i8_code(f[e], d);
        }
        if (VEC && peak != nullptr) {  // (a warp's 32 vectors are an aligned block)
            int sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += abs(static_cast<int>(static_cast<int8_t>(c[e])));
            top = max(top, __reduce_add_sync(0xffffffffu, sum));
        }
        Part::store_codes(out, pitch, i, tid, G, c);
    }
    if (peak != nullptr) row_peak(top, G, tid, red, peak);
}

// F16: codes as float16 into x16 [rows][pitch], row r from row perm[r] of x (see launch_i8_quantize_f16).
template <typename T, int U, bool VEC, bool F16>
__global__ void __launch_bounds__(kRowThreads)
i8_quantize_kernel(const T* x, long long ld, I8View q, RowPlan pl, const int32_t* perm, const int32_t* status, __half* x16,
                   int* peak) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    __shared__ float red[kRowThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int team = threadIdx.x / pl.G, tid = threadIdx.x - team * pl.G;
    const long long r = (long long)blockIdx.x * (blockDim.x / pl.G) + team;
    if (r >= q.rows) return;  // (whole warps; G is the CTA where it is more than a warp)
    const T* row = x + r * ld;
    Raw<T>* kept = reinterpret_cast<Raw<T>*>(row_smem) + (size_t)team * pl.vecs;
    if constexpr (F16) {
        if (status != nullptr && __ldcg(status) != LORA_OK) return;  // (perm is not valid either)
        if (perm != nullptr) row = x + (long long)__ldcg(perm + r) * ld;
        quantise_row<T, U, VEC>(row, q.cols, (int)q.pitch, pl, tid, kept, red, q.scales + r, x16 + r * q.pitch,
                                peak ? peak + r : nullptr);
    } else {
        quantise_row<T, U, VEC>(row, q.cols, (int)q.pitch, pl, tid, kept, red, q.scales + r, q.codes + r * q.pitch, nullptr);
    }
}

// ---- before the product of a small batch: x's codes and the per-token shrink, one launch -------------------
// The first n CTAs each take a row of x: quantise it (or turn its stored codes into float16); the others each a
// token, 8 rows of its adapter's A and a part of K, s[part][t][j] = (alpha / r) x[t] . A[j] over the part.  Both
// read x, a few KB; bound by latency, which one launch less shortens (one token 4096 x 4096 float16: 25 us for
// the linear as three launches, 8 as two).
constexpr int kFrontThreads = 256;
struct FrontArgs {
    PoolView pool;
    const int32_t* perm;    // rows of x16
    const int32_t* idx;
    const int32_t* status;
    const void* x;
    I8View q;               // quantised into (codes, or scales alone with x16), or (stored) expanded from
    __half* x16;            // nullable: codes as bytes
    float* scales;
    int* peak;              // with x16
    float* s;
    RowPlan pl;
    int n, stored, rows, parts;  // rows: CTAs that take rows of x (n, or 0)
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kFrontThreads)
i8_front_kernel(const FrontArgs a) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    __shared__ float red[kFrontThreads / 32][8];
    pdl_wait();
    pdl_trigger();
    const int status = a.status ? __ldcg(a.status) : LORA_OK;  // (independent loads first)
    const int h = a.q.cols, R = a.pool.R, tid = threadIdx.x;
    if ((int)blockIdx.x < a.rows) {
        const int r = blockIdx.x;
        const int from = a.x16 && a.perm ? __ldcg(a.perm + r) : r;
        if (status != LORA_OK) return;
        if (a.stored) {
            const int8_t* codes = a.q.codes + (size_t)from * a.q.pitch;
            int top = 0;
            for (int k0 = 0; k0 < (int)a.q.pitch; k0 += kFrontThreads * 16) {
                const int k = k0 + tid * 16;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (k < (int)a.q.pitch) {
                    w = __ldg(reinterpret_cast<const uint4*>(codes + k));
                    const uint2 c0 = i8_to_f16x4(w.x), c1 = i8_to_f16x4(w.y), c2 = i8_to_f16x4(w.z), c3 = i8_to_f16x4(w.w);
                    uint4* out = reinterpret_cast<uint4*>(a.x16 + (size_t)r * a.q.pitch + k);
                    out[0] = make_uint4(c0.x, c0.y, c1.x, c1.y);
                    out[1] = make_uint4(c2.x, c2.y, c3.x, c3.y);
                }
                int sum = i8_abs_sum(w.x) + i8_abs_sum(w.y) + i8_abs_sum(w.z) + i8_abs_sum(w.w);
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);  // (16 lanes a block)
                top = max(top, max(sum, __shfl_xor_sync(0xffffffffu, sum, 16)));
            }
            row_peak(top, kFrontThreads, tid, &red[0][0], a.peak + r);
            if (tid == 0) a.scales[r] = __ldg(a.q.scales + from);
            return;
        }
        const T* row = static_cast<const T*>(a.x) + (size_t)from * h;
        Raw<T>* kept = reinterpret_cast<Raw<T>*>(row_smem);
        if (a.x16)
            quantise_row<T, 2, VEC>(row, h, (int)a.q.pitch, a.pl, tid, kept, &red[0][0], a.scales + r, a.x16 + (size_t)r * a.q.pitch,
                                      a.peak + r);
        else
            quantise_row<T, 2, VEC>(row, h, (int)a.q.pitch, a.pl, tid, kept, &red[0][0], a.scales + r, a.q.codes + (size_t)r * a.q.pitch,
                                      nullptr);
        return;
    }
    using Part = RowPart<T, VEC>;
    const int groups = (R + 7) / 8, b = blockIdx.x - a.rows;
    const int t = b / (groups * a.parts), g = b / a.parts % groups, p = b % a.parts;
    const int slot = __ldcg(a.idx + t);
    if (slot < 0 || status != LORA_OK) return;
    const SlotEntry e = a.pool.table[slot];
    if (g * 8 >= e.rank) return;  // (what reads s leaves out the columns past the rank)
    const T* xr = static_cast<const T*>(a.x) + (size_t)t * h;
    const T* Ab = static_cast<const T*>(a.pool.A) + ((size_t)slot * R + (size_t)g * 8) * h;
    const int vecs = (h + 7) / 8, per = ((vecs + kFrontThreads - 1) / kFrontThreads + a.parts - 1) / a.parts * kFrontThreads;
    float acc[8] = {};
    for (int i0 = p * per; i0 < min(vecs, (p + 1) * per); i0 += kFrontThreads) {
        const int i = i0 + tid;
        if (Part::at(i, 0, tid, kFrontThreads) >= h) continue;
        float xf[8];
        Raw<T> av[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) av[r] = Part::load(Ab + (size_t)min(r, R - 1 - g * 8) * h, h, i, tid, kFrontThreads);
        to8(Part::load(xr, h, i, tid, kFrontThreads), xf);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float af[8];
            to8(av[r], af);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[r] = fmaf(xf[c], af[c], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float v = acc[r];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if ((tid & 31) == 0) red[tid >> 5][r] = v;
    }
    __syncthreads();
    if (tid < 8 && g * 8 + tid < R) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kFrontThreads / 32; ++w) v += red[w][tid];
        a.s[((size_t)p * a.n + t) * R + g * 8 + tid] = e.scale * v;
    }
}

// Stored codes as float16, rows in the order of perm.  16 codes a thread; bound by memory.  (A warp a row with four
// loads in flight was slower: 4096 x 4096 13 us against 11.)
__global__ void __launch_bounds__(256)
i8_expand_kernel(I8View q, const int32_t* perm, const int32_t* status, uint4* x16, float* scales) {
    pdl_wait();
    pdl_trigger();
    if (status != nullptr && __ldcg(status) != LORA_OK) return;
    const unsigned per_row = (unsigned)(q.pitch / 16), e = blockIdx.x * 256u + threadIdx.x, r = e / per_row, c = e - r * per_row;
    if (r >= (unsigned)q.rows) return;
    const unsigned from = perm ? (unsigned)__ldcg(perm + r) : r;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(q.codes + (size_t)from * q.pitch) + c);
    const uint2 a = i8_to_f16x4(w.x), b = i8_to_f16x4(w.y), f = i8_to_f16x4(w.z), g = i8_to_f16x4(w.w);
    x16[2 * (size_t)e] = make_uint4(a.x, a.y, b.x, b.y);
    x16[2 * (size_t)e + 1] = make_uint4(f.x, f.y, g.x, g.y);
    if (c == 0 && scales != nullptr) scales[r] = __ldg(q.scales + from);
}

// ---- read back ------------------------------------------------------------------------------------------
// Bound by memory.  VEC: 16 codes a thread and 16-byte stores; else an element a thread, neighbours side by
// side.  No early release of the kernels behind: out may be the weight of a 16-bit linear, whose GEMM
// streams it without waiting for more than its release.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
i8_dequantize_kernel(I8View q, T* __restrict__ out, long long ld) {
    pdl_wait();
    const long long r = (long long)blockIdx.y * 8 + threadIdx.x / 32 + (long long)blockIdx.z * 65535 * 8;
    if (r >= q.rows) return;
    const int lane = threadIdx.x & 31;
    const float s = __ldg(q.scales + r);
    const int8_t* codes = q.codes + r * q.pitch;
    T* row = out + r * ld;
    if constexpr (VEC) {
        const int k = (blockIdx.x * 32 + lane) * 16;
        if (k >= q.cols) return;
        const int4 w = __ldcs(reinterpret_cast<const int4*>(codes + k));
        const int words[4] = {w.x, w.y, w.z, w.w};
        alignas(16) T v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = from_f32<T>(__int2float_rn((words[i / 4] << (24 - 8 * (i & 3))) >> 24) * s);
        if (k + 16 <= q.cols) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i)
                reinterpret_cast<uint4*>(row + k)[i] = reinterpret_cast<const uint4*>(v)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k + i < q.cols) row[k + i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int k = blockIdx.x * 512 + i * 32 + lane;
            if (k < q.cols) row[k] = from_f32<T>(__int2float_rn(codes[k]) * s);
        }
    }
}

// ---- residual addition, root-mean-square norm, output in 8 bits -------------------------------------------
// h = T(x + residual), r = 1 / sqrt(mean h^2 + eps), y = T(h r w), and the stored form of h r w.  The codes
// have to be those of the real h r w / s, so what a whole row shares is held in two float32 parts: the sum
// of squares (each square and each addition with its rounding error), r and r / s, to about 2^-44.  An
// element then costs one product u = h w (exact in two parts) times r / s, and near the border of two codes
// the second parts decide.  That wants h^2 and h w well inside float32's range: norm_wide takes the rows where they
// are not.
struct NormArgs {
    const void* x;
    const void* residual;  // nullable
    const void* w;
    void* h;               // nullable: where x + residual goes
    void* y;               // nullable
    I8View q;              // codes nullable
    long long ldx, ldr, ldh, ldy;
    float eps;
    int rows, cols;
    RowPlan pl;
};

struct Two {
    float hi, lo;
};

// Rows outside these bounds (of sum h^2, max |h w| and the scale) are norm_wide's: inside, r is between 2^-50 and 2^20
// and the largest |h w| between 2^-77 and 2^76, so that the second parts of all that decides a code are normal numbers.
constexpr float kMostSquares = 1e30f, kMostProduct = 0x1p76f, kLeastScale = 0x1p-64f;

// What a row shares, from its sum of squares and largest |u|.
struct NormRow {
    float r, s;  // 1 / sqrt(mean + eps), and the scale
    Two g;       // r / s
};
__device__ __forceinline__ NormRow norm_row(Two ss, MaxPair m, int cols, float eps) {
    NormRow o;
    const float n = static_cast<float>(cols), q0 = __fdiv_rn(ss.hi, n);
    const float q1 = (fmaf(-q0, n, ss.hi) + ss.lo) / n;
    float err;
    const float hi = two_sum(q0, eps, err), lo = err + q1;
    const float r0 = rsqrtf(hi), p = __fmul_rn(r0, r0);
    float e = fmaf(-hi, p, 1.f);
    e = fmaf(-hi, fmaf(r0, r0, -p), e);
    e = fmaf(-lo, p, e);
    const Two r = {r0, r0 * fmaf(0.375f * e, e, 0.5f * e)};
    o.r = r.hi + r.lo;
    // s = max|u| r / 127
    const float t = __fmul_rn(m.hi, r.hi);
    const float tl = fmaf(m.hi, r.hi, -t) + fmaf(m.hi, r.lo, m.lo * r.hi);
    const float s0 = __fdiv_rn(t, 127.f);
    o.s = s0 + (fmaf(-127.f, s0, t) + tl) / 127.f;
    o.g.hi = __fdiv_rn(r.hi, o.s);
    o.g.lo = (fmaf(-o.g.hi, o.s, r.hi) + r.lo) / o.s;
    return o;
}
// The code of u + ul (ul: what u's rounding left off) where the quotient is (u + ul) g.
__device__ __forceinline__ uint32_t norm_code(float u, float ul, Two g) {
    const float v = __fmul_rn(u, g.hi);
    // (a tiny scale is rounded coarsely: quotients may pass 127)
    int k = static_cast<int>(fminf(fmaxf(rintf(v), -127.f), 127.f));
    if (fabsf(v - static_cast<float>(k)) > 0.4999f) {
        const float rest = fmaf(u, g.hi, -v) + u * g.lo + ul * g.hi;
        const int side = v > static_cast<float>(k) ? 1 : -1;
        const float past = side * ((v - (static_cast<float>(k) + 0.5f * side)) + rest);
        if (past > 0.f || (past == 0.f && (k & 1) != 0)) k += side;
    }
    return static_cast<uint32_t>(min(max(k, -127), 127));
}
__device__ __forceinline__ uint2 pack_codes(const uint32_t (&c)[8]) {
    return make_uint2(i8_pack4(c[0], c[1], c[2], c[3]), i8_pack4(c[4], c[5], c[6], c[7]));
}
// Codes of eight elements h w, the first four in x: those next to the border of two.  (Out of line: in line its
// registers cost the common path occupancy, 144 us against 123 for 16384 x 4096.)
template <typename T> __device__ __noinline__ uint2 norm_codes(Raw<T> hr, Raw<T> wr, Two g) {
    float h[8], w[8];
    to8(hr, h);
    to8(wr, w);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float u = __fmul_rn(h[e], w[e]);
        c[e] = norm_code(u, sizeof(T) == 2 ? 0.f : fmaf(h[e], w[e], -u), g);  // (16-bit numbers' products are exact)
    }
    return pack_codes(c);
}

// A row's threads' sums and maxima together.  red: shared memory of the CTA; again: it may still be read from before.
template <bool EXACT> __device__ __forceinline__ void norm_reduce(Two& ss, MaxPair& m, int G, float (*red)[4], bool again) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        float err;
        const float oh = __shfl_xor_sync(0xffffffffu, ss.hi, d), ol = __shfl_xor_sync(0xffffffffu, ss.lo, d);
        ss.hi = two_sum(ss.hi, oh, err);
        ss.lo += ol + err;
        if constexpr (EXACT)
            m.hi = max_nan(m.hi, __shfl_xor_sync(0xffffffffu, m.hi, d));
        else
            m = max_pair(m, MaxPair{__shfl_xor_sync(0xffffffffu, m.hi, d), __shfl_xor_sync(0xffffffffu, m.lo, d)});
    }
    if (G > 32) {
        if (again) __syncthreads();  // (the CTA is one row: all or none come here)
        if ((threadIdx.x & 31) == 0)
            *reinterpret_cast<float4*>(red[threadIdx.x >> 5]) = make_float4(ss.hi, ss.lo, m.hi, m.lo);
        __syncthreads();
        ss = Two{0.f, 0.f};
        m = MaxPair{0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < G / 32; ++k) {
            const float4 o = *reinterpret_cast<const float4*>(red[k]);
            float err;
            ss.hi = two_sum(ss.hi, o.x, err);
            ss.lo += o.y + err;
            m = max_pair(m, MaxPair{o.z, o.w});
        }
    }
}

// A number as a fraction of at least 1/2 and below 1 either way, and a power of two (0 and what is not finite: themselves).
struct Frac {
    float m;
    int e;
};
__device__ __forceinline__ Frac frac(float x) {
    const uint32_t top = __float_as_uint(x) >> 23 & 255;
    const float big = top == 0 ? x * 16777216.f : x;  // (subnormal: times 2^24)
    const uint32_t b = __float_as_uint(big);
    Frac f;
    f.e = x == 0.f || top == 255 ? 0 : static_cast<int>(b >> 23 & 255) - (top == 0 ? 150 : 126);
    f.m = x == 0.f || top == 255 ? x : __uint_as_float((b & 0x807fffffu) | 0x3f000000u);
    return f;
}
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }  // -126 <= k <= 127
constexpr uint32_t kInf = 0x7f800000u;
constexpr int kNoProduct = -(1 << 20);

// The largest and least of a row's threads' numbers (red: as norm_reduce's).
__device__ __forceinline__ void row_extremes(uint32_t (&most)[2], uint32_t (&least)[2], int G, float (*red)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        most[i] = __reduce_max_sync(0xffffffffu, most[i]);
        least[i] = __reduce_min_sync(0xffffffffu, least[i]);
    }
    if (G > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
            *reinterpret_cast<uint4*>(red[threadIdx.x >> 5]) = make_uint4(most[0], most[1], least[0], least[1]);
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < G / 32; ++k) {
            const uint4 o = *reinterpret_cast<const uint4*>(red[k]);
            most[0] = max(most[0], o.x), most[1] = max(most[1], o.y);
            least[0] = min(least[0], o.z), least[1] = min(least[1], o.w);
        }
    }
}

// A row whose squares or products leave float32's range (elements from about 2^50 on, weights or products at its ends)
// or that holds an infinity or NaN.  Squares are of h 2^ea, products relative to 2^E.  Mostly one power of
// two for all of h and one for all of w bring every product between 2^-100 and 2^62; SPREAD: where none do, fractions
// and exponents apart, E the largest product's exponent.  hb, wb: bits of the largest |h| and |w| (a NaN's are the largest).
template <typename T, bool VEC, bool SPREAD>
__device__ __forceinline__ void norm_wide_row(const NormArgs& a, const Raw<T>* kept, long long r, int tid, float (*red)[4],
                                              uint32_t hb, uint32_t wb, int ea, int eb) {
    using Part = RowPart<T, VEC>;
    const int G = a.pl.G, vecs = a.pl.vecs, cols = a.cols;
    const T* src = a.h ? static_cast<const T*>(a.h) + r * a.ldh : static_cast<const T*>(a.x) + r * a.ldx;
    const T* wr = static_cast<const T*>(a.w);
    auto row = [&](int i, float (&h)[8], float (&w)[8]) {
        to8(a.pl.keep ? kept[i] : Part::load(src, cols, i, tid, G), h);
        to8(Part::load(wr, cols, i, tid, G), w);
    };
    constexpr bool EXACT = sizeof(T) == 2;  // squares and products of two 16-bit numbers are float32 numbers
    const bool bad = hb >= kInf || wb >= kInf;
    int E = -(ea + eb);
    if constexpr (SPREAD) {
        uint32_t most[2] = {0, 0}, least[2] = {0, 0};
#pragma unroll 1
        for (int i = tid; i < vecs; i += G) {
            float h[8], w[8];
            row(i, h, w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (h[e] != 0.f && w[e] != 0.f)
                    most[0] = max(most[0], static_cast<uint32_t>(frac(h[e]).e + frac(w[e]).e - kNoProduct));
        }
        row_extremes(most, least, G, red);
        E = static_cast<int>(most[0]) + kNoProduct;
    }
    const float fa = pow2(max(ea, -126)), fb = pow2(max(eb, -126));  // (without SPREAD ea and eb are at least -98)
    // h's product with w is (p + l) 2^E; g: h 2^ea
    auto product = [&](float h, float w, float& g, float& p, float& l) {
        if constexpr (SPREAD) {
            const Frac fh = frac(h), fw = frac(w);
            g = fh.m * pow2(max(fh.e + ea, -126));
            p = __fmul_rn(fh.m, fw.m);
            l = EXACT ? 0.f : fmaf(fh.m, fw.m, -p);
            const int d = fh.e + fw.e - E;
            const float x = d > -30 ? pow2(min(d, 1)) : 0.f;  // (smaller ones are codes of 0; d > 0: of what is not finite)
            p *= x;
            l *= x;
        } else {
            g = h * fa;
            const float v = w * fb;
            p = __fmul_rn(g, v);
            l = EXACT ? 0.f : fmaf(g, v, -p);
        }
    };
    Two ss = {0.f, 0.f};
    MaxPair m = {0.f, 0.f};
    if (hb < kInf && E != kNoProduct) {  // (else the row's values are 0, or those of an infinity or NaN)
#pragma unroll 1
        for (int i = tid; i < vecs; i += G) {
            float h[8], w[8];
            row(i, h, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float g, p, l, err;
                product(h[e], w[e], g, p, l);
                const float sq = __fmul_rn(g, g);
                ss.hi = two_sum(ss.hi, sq, err);
                ss.lo += EXACT ? err : err + fmaf(g, g, -sq);
                if constexpr (EXACT)
                    m.hi = max_nan(m.hi, fabsf(p));
                else
                    m = max_pair(m, MaxPair{fabsf(p), p < 0.f ? -l : l});
            }
        }
        norm_reduce<EXACT>(ss, m, G, red, true);
    }
    const int k0 = E + ea;
    const NormRow o = norm_row(ss, m, cols, a.eps * fa * fa);  // (where fa is cut off, eps counts for nothing)
    // 1 / sqrt, times 2^-ea; of a row with an infinity 0, with a NaN NaN
    const float rf = hb > kInf ? __uint_as_float(hb) : hb == kInf ? 0.f : o.r;
    float s = __uint_as_float(0x7fc00000u);
    Two g = {0.f, 0.f};
    if (!bad && !(m.hi > 0.f)) {
        s = 0.f;
    } else if (!bad) {
        const int es = frac(o.s).e + k0;
        if (o.s >= 0x1p-72f && es >= -125 && es <= 128) {
            s = ldexpf(o.s, k0);
            g = o.g;
        } else {
            // a scale with fewer bits, or 0, or too large for float32 (NaN): rounded once, from float64
            const double mean = (static_cast<double>(ss.hi) + ss.lo) / cols + ldexp(static_cast<double>(a.eps), 2 * ea);
            const double rE = ldexp(1.0 / sqrt(mean), k0), sd = (static_cast<double>(m.hi) + m.lo) * rE / 127.0;
            if (static_cast<float>(sd) <= kFltMax) s = static_cast<float>(sd);
            if (s > 0.f) {
                const double q = rE / s;
                g.hi = static_cast<float>(q);
                g.lo = static_cast<float>(q - g.hi);
            }
        }
    }
    if (a.q.codes && tid == 0) a.q.scales[r] = s;
    // (without SPREAD the 1 / sqrt is between 2^-62 and 2^10, and times a product at most 2^40)
    const float rup = rf * 0x1p62f, down = SPREAD ? 0.f : pow2(-eb - 62);
#pragma unroll 1
    for (int i = tid; i < vecs; i += G) {
        float h[8], w[8], y[8];
        row(i, h, w);
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float hg, p, l;
            product(h[e], w[e], hg, p, l);
            c[e] = g.hi > 0.f ? norm_code(p, l, g) : 0;
            if constexpr (SPREAD) {
                // (the product of fractions times rf is between 2^-62 and 2^10, or 0 or not finite: the first factor's
                // product is exact, or is an infinity that the second would have made)
                const Frac fh = frac(h[e]), fw = frac(w[e]);
                const int k = fh.e + fw.e + ea, k1 = min(max(k, -62), 127);
                y[e] = __fmul_rn(fh.m, fw.m) * rf * pow2(k1) * pow2(min(max(k - k1, -126), 127));
            } else {
                y[e] = p * rup * down;
            }
        }
        if (a.q.codes) Part::store_words(a.q.codes + r * a.q.pitch, (int)a.q.pitch, i, tid, G, pack_codes(c));
        if (a.y) Part::store(static_cast<T*>(a.y) + r * a.ldy, cols, i, tid, G, from8<T>(y));
    }
}

// norm_wide_row, with what brings the row into range.  (Out of line, for the common path's registers.  16384 x 4096 bfloat16, y and codes: 243 us where
// every row comes here, 599 where it needs SPREAD, 90 where none does.)
template <typename T, bool VEC>
__device__ __noinline__ void norm_wide(const NormArgs& a, const Raw<T>* kept, long long r, int tid, float (*red)[4]) {
    using Part = RowPart<T, VEC>;
    const int G = a.pl.G, vecs = a.pl.vecs, cols = a.cols;
    const T* src = a.h ? static_cast<const T*>(a.h) + r * a.ldh : static_cast<const T*>(a.x) + r * a.ldx;
    // the largest |h| and |w|, and one less than the least that are not 0 (their bits)
    uint32_t most[2] = {0, 0}, least[2] = {0xffffffffu, 0xffffffffu};
#pragma unroll 1
    for (int i = tid; i < vecs; i += G) {
        float v[2][8];
        to8(a.pl.keep ? kept[i] : Part::load(src, cols, i, tid, G), v[0]);
        to8(Part::load(static_cast<const T*>(a.w), cols, i, tid, G), v[1]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t b = __float_as_uint(v[e / 8][e % 8]) & 0x7fffffffu;
            most[e / 8] = max(most[e / 8], b);
            least[e / 8] = min(least[e / 8], b - 1);
        }
    }
    row_extremes(most, least, G, red);
    if (most[0] < kInf && most[1] < kInf) {
        // the largest to 2^31 at most, times 2^60 at most (eps, which is at least 2^-40, has to stay in range times 2^2ea)
        const int ea = min(31 - frac(__uint_as_float(most[0])).e, 60), eb = min(31 - frac(__uint_as_float(most[1])).e, 60);
        const int el = ea + (most[0] ? frac(__uint_as_float(least[0] + 1)).e : 0);
        const int fl = eb + (most[1] ? frac(__uint_as_float(least[1] + 1)).e : 0);
        // (a fraction is at least 1/2: products from 2^-100 on, no factor below 2^-121)
        if (el >= -120 && fl >= -120 && el + fl >= -98) {
            norm_wide_row<T, VEC, false>(a, kept, r, tid, red, most[0], most[1], ea, eb);
            return;
        }
    }
    const int eh = most[0] < kInf ? frac(__uint_as_float(most[0])).e : 0;
    norm_wide_row<T, VEC, true>(a, kept, r, tid, red, most[0], most[1], min(-eh, 60), 0);
}

template <typename T, int U, bool VEC>
__global__ void __maxnreg__(VEC || U == 1 ? 64 : 80)  // (norm_wide's needs may not cost the common path occupancy)
i8_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    __shared__ __align__(16) float red[kRowThreads / 32][4];
    pdl_wait();
    pdl_trigger();
    using Part = RowPart<T, VEC>;
    constexpr bool EXACT = sizeof(T) == 2;  // squares and products of two 16-bit numbers are float32 numbers
    const int G = a.pl.G, vecs = a.pl.vecs, team = threadIdx.x / G, tid = threadIdx.x - team * G, cols = a.cols;
    const long long r = (long long)blockIdx.x * (blockDim.x / G) + team;
    if (r >= a.rows) return;
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    const T* rr = a.residual ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    T* hr = a.h ? static_cast<T*>(a.h) + r * a.ldh : nullptr;
    const T* wr = static_cast<const T*>(a.w);
    Raw<T>* kept = reinterpret_cast<Raw<T>*>(row_smem) + (size_t)team * vecs;
    // vector i of the sum on a later pass
    auto again = [&](int i) -> Raw<T> {
        if (a.pl.keep) return kept[i];
        if (hr) return Part::load(hr, cols, i, tid, G);
        return Part::load(xr, cols, i, tid, G);  // (without residual_out there is no residual)
    };
    for (int i0 = tid; i0 < vecs; i0 += U * G) {
        Raw<T> v[U], t[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * G < vecs) v[u] = Part::load(xr, cols, i0 + u * G, tid, G);
        if (rr)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * G < vecs) t[u] = Part::load(rr, cols, i0 + u * G, tid, G);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * G;
            if (i >= vecs) break;
            if (rr) add_raw(v[u], t[u]);
            if (hr) Part::store(hr, cols, i, tid, G, v[u]);
            if (a.pl.keep) kept[i] = v[u];
        }
    }
    // (rolled up, as the loop at the end: unrolled they do not fit the instruction cache, 16384 x 4096 bfloat16
    // 147 us against 118)
    F2 sh = f2(0.f, 0.f), sl = sh;
    MaxPair m = {0.f, 0.f};
#pragma unroll 1
    for (int i = tid; i < vecs; i += G) {
        float h[8], w[8];
        to8(again(i), h);
        to8(Part::load(wr, cols, i, tid, G), w);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const F2 g = f2(h[e], h[e + 1]), sq = mul2(g, g);
            const float2 p = unpack(mul2(g, f2(w[e], w[e + 1])));
            F2 err;
            sh = two_sum2(sh, sq, err);
            if constexpr (EXACT) {
                m.hi = max_nan(m.hi, max_nan(fabsf(p.x), fabsf(p.y)));
            } else {
                const float2 q = unpack(sq);
                err = add2(err, f2(fmaf(h[e], h[e], -q.x), fmaf(h[e + 1], h[e + 1], -q.y)));
                const float lx = fmaf(h[e], w[e], -p.x), ly = fmaf(h[e + 1], w[e + 1], -p.y);
                m = max_pair(m, MaxPair{fabsf(p.x), p.x < 0.f ? -lx : lx});
                m = max_pair(m, MaxPair{fabsf(p.y), p.y < 0.f ? -ly : ly});
            }
            sl = add2(sl, err);
        }
    }
    Two ss;
    {
        const float2 hi = unpack(sh), lo = unpack(sl);
        float err;
        ss.hi = two_sum(hi.x, hi.y, err);
        ss.lo = lo.x + lo.y + err;
    }
    norm_reduce<EXACT>(ss, m, G, red, false);
    NormRow o = norm_row(ss, m, cols, a.eps);
    if (!(ss.hi <= kMostSquares && m.hi <= kMostProduct && o.s >= kLeastScale)) {
        // a row of zeros (a silent token) has nothing to take care of but 0 / 0
        uint32_t any = !(ss.hi == 0.f && m.hi == 0.f);
        if (!any)
#pragma unroll 1
            for (int i = tid; i < vecs; i += G) any |= any_bits(again(i));
        if (G > 32 ? __syncthreads_or(any) : __any_sync(0xffffffffu, any)) {
            norm_wide<T, VEC>(a, kept, r, tid, red);
            return;
        }
        o.s = o.g.hi = 0.f;
    }
    if (a.q.codes && tid == 0) a.q.scales[r] = o.s;
    // Products are taken times 2^24: 1 / sqrt is at most 2^20, so a value y that is a normal number comes from a product
    // that is one too.
    const F2 up = f2(0x1p24f, 0x1p24f), g2 = f2(o.g.hi * 0x1p-24f, o.g.hi * 0x1p-24f), r2 = f2(o.r * 0x1p-24f, o.r * 0x1p-24f);
#pragma unroll 1
    for (int i = tid; i < vecs; i += G) {
        const Raw<T> hraw = again(i), wraw = Part::load(wr, cols, i, tid, G);
        float h[8], w[8];
        to8(hraw, h);
        to8(wraw, w);
        F2 u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = mul2(mul2(f2(h[2 * e], h[2 * e + 1]), up), f2(w[2 * e], w[2 * e + 1]));
        if (a.q.codes) {
            uint32_t code[8];
            float far = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const F2 q = mul2(u[e / 2], g2);
                const float2 t = unpack(sub2(q, nearest2(q, code[e], code[e + 1])));
                far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
            }
            uint2 words = pack_codes(code);
            if (far > 0.4999f) words = norm_codes<T>(hraw, wraw, o.g);
            Part::store_words(a.q.codes + r * a.q.pitch, (int)a.q.pitch, i, tid, G, words);
        }
        if (a.y) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 p = unpack(mul2(u[e], r2));
                y[2 * e] = p.x, y[2 * e + 1] = p.y;
            }
            Part::store(static_cast<T*>(a.y) + r * a.ldy, cols, i, tid, G, from8<T>(y));
        }
    }
}

static bool aligned16(const void* p, long long ld, int rows, size_t elt) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (ld * (long long)elt) % 16 == 0);
}

// Threads a row, vectors a thread loads at once (1 or 4), threads a CTA, shared memory.  Few rows: a thread a
// vector, for the row's latency; many: four vectors a thread.
struct RowLaunch {
    RowPlan pl;
    int U, threads;
    unsigned blocks;
    size_t smem;
};
static RowLaunch row_launch(int rows, int cols, size_t elt) {
    RowLaunch l;
    const int vecs = (int)(i8_pitch(cols) / 8);
    l.U = rows <= 2 * num_sms() ? 1 : 4;
    const int need = (vecs + l.U - 1) / l.U;
    l.pl.G = std::min(kRowThreads, (need + 31) / 32 * 32);
    // whole rounds of G, so that without VEC a round's 8 G elements are all some thread's
    l.pl.vecs = (vecs + l.pl.G - 1) / l.pl.G * l.pl.G;
    l.threads = l.pl.G > 32 ? l.pl.G : 256;
    const int per = l.threads / l.pl.G;
    l.blocks = (unsigned)(((long long)rows + per - 1) / per);
    l.smem = (size_t)per * l.pl.vecs * 8 * elt;
    l.pl.keep = l.smem <= kRowSmem;
    if (!l.pl.keep) l.smem = 0;
    return l;
}
template <typename K> static int allow_smem(K fn, bool& done) {
    if (!done) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowSmem));
        done = true;
    }
    return LORA_OK;
}

template <typename T, int U, bool VEC, bool F16>
static int quantize_l(const T* x, long long ld, const I8View& q, const RowLaunch& l, const int32_t* perm,
                      const int32_t* status, __half* x16, int* peak, cudaStream_t st) {
    static bool done = false;
    const auto fn = i8_quantize_kernel<T, U, VEC, F16>;
    const int rc = allow_smem(fn, done);
    if (rc) return rc;
    void* args[] = {(void*)&x, (void*)&ld, (void*)&q, (void*)&l.pl, (void*)&perm, (void*)&status, (void*)&x16, (void*)&peak};
    LORA_CUDA_TRY(launch_pdl((const void*)fn, dim3(l.blocks), dim3(l.threads), l.smem, st, args));
    return LORA_OK;
}
template <typename T, bool F16>
static int quantize_t(const void* x, long long ld, const I8View& q, const int32_t* perm, const int32_t* status, void* x16,
                      int* peak, cudaStream_t st) {
    const bool vec = aligned16(x, ld, q.rows, sizeof(T));
    const RowLaunch l = row_launch(q.rows, q.cols, sizeof(T));
    const T* xp = static_cast<const T*>(x);
    __half* hp = static_cast<__half*>(x16);
    if (l.U == 1)
        return vec ? quantize_l<T, 1, true, F16>(xp, ld, q, l, perm, status, hp, peak, st)
                   : quantize_l<T, 1, false, F16>(xp, ld, q, l, perm, status, hp, peak, st);
    return vec ? quantize_l<T, 4, true, F16>(xp, ld, q, l, perm, status, hp, peak, st)
               : quantize_l<T, 4, false, F16>(xp, ld, q, l, perm, status, hp, peak, st);
}

int launch_i8_quantize(const void* x, int dtype, long long ld, const I8View& q, cudaStream_t st) {
    if (q.rows == 0) return LORA_OK;
    switch (dtype) {
        case LORA_F32: return quantize_t<float, false>(x, ld, q, nullptr, nullptr, nullptr, nullptr, st);
        case LORA_F16: return quantize_t<__half, false>(x, ld, q, nullptr, nullptr, nullptr, nullptr, st);
        default: return quantize_t<__nv_bfloat16, false>(x, ld, q, nullptr, nullptr, nullptr, nullptr, st);
    }
}

int launch_i8_quantize_f16(const void* x, int dtype, int rows, int cols, const int32_t* perm, const int32_t* status,
                           void* x16, float* scales, int* peak, cudaStream_t st) {
    const I8View q = i8_view(nullptr, scales, rows, cols);
    switch (dtype) {
        case LORA_F32: return quantize_t<float, true>(x, cols, q, perm, status, x16, peak, st);
        case LORA_F16: return quantize_t<__half, true>(x, cols, q, perm, status, x16, peak, st);
        default: return quantize_t<__nv_bfloat16, true>(x, cols, q, perm, status, x16, peak, st);
    }
}

// K parts of the front's shrink.
int i8_front_parts(const PoolView& pv, int n) {
    return std::max(1, std::min({(pv.h_in + 8 * kFrontThreads - 1) / (8 * kFrontThreads), 4, 256 / std::max(n, 1)}));
}

template <typename T> static int front_t(FrontArgs a, cudaStream_t st) {
    // rows of x and of A on 16-byte boundaries
    const bool vec = aligned16(a.x, a.pool.h_in, 2, sizeof(T));
    const int vecs = (int)(a.q.pitch / 8);
    a.pl.G = kFrontThreads;
    a.pl.vecs = (vecs + kFrontThreads - 1) / kFrontThreads * kFrontThreads;
    size_t smem = a.rows && !a.stored ? (size_t)a.pl.vecs * 8 * sizeof(T) : 0;
    a.pl.keep = smem <= 48 * 1024 - 1024;
    if (!a.pl.keep) smem = 0;
    const long long grid = a.rows + (long long)a.n * ((a.pool.R + 7) / 8) * a.parts;
    const void* fn = vec ? (const void*)i8_front_kernel<T, true> : (const void*)i8_front_kernel<T, false>;
    void* args[] = {(void*)&a};
    LORA_CUDA_TRY(launch_pdl(fn, dim3((unsigned)grid), dim3(kFrontThreads), smem, st, args));
    return LORA_OK;
}

int launch_i8_front(const PoolView& pv, const SegView& sv, const void* x, const I8View* xq, void* codes, bool f16,
                    float* scales, int* peak, float* s, int* s_parts, cudaStream_t st) {
    FrontArgs a;
    memset(&a, 0, sizeof(a));
    a.pool = pv;
    a.perm = sv.perm;
    a.idx = sv.idx;
    a.status = sv.status;
    a.x = x;
    a.stored = xq != nullptr;
    a.q = xq ? *xq : i8_view(codes, scales, sv.n, pv.h_in);
    a.x16 = f16 ? static_cast<__half*>(codes) : nullptr;
    a.scales = scales;
    a.peak = peak;
    a.s = s;
    a.n = sv.n;
    a.rows = xq && !f16 ? 0 : sv.n;
    a.parts = *s_parts = i8_front_parts(pv, sv.n);
    switch (pv.dtype) {
        case LORA_F32: return front_t<float>(a, st);
        case LORA_F16: return front_t<__half>(a, st);
        default: return front_t<__nv_bfloat16>(a, st);
    }
}

int launch_i8_expand_small(const I8View& x, const int32_t* perm, const int32_t* status, void* x16, float* scales,
                           int* peak, cudaStream_t st) {
    FrontArgs a;
    memset(&a, 0, sizeof(a));
    a.perm = perm;
    a.status = status;
    a.q = x;
    a.x16 = static_cast<__half*>(x16);
    a.scales = scales;
    a.peak = peak;
    a.stored = 1;
    a.rows = x.rows;  // (and no token's shrink)
    void* args[] = {(void*)&a};
    LORA_CUDA_TRY(launch_pdl((const void*)i8_front_kernel<__half, true>, dim3(x.rows), dim3(kFrontThreads), 0, st, args));
    return LORA_OK;
}

int launch_i8_expand(const I8View& x, const int32_t* perm, const int32_t* status, void* x16, float* scales, cudaStream_t st) {
    const long long chunks = (long long)x.rows * (long long)(x.pitch / 16);
    if (chunks > 0xffffff00LL) return set_error(LORA_EUNSUP, "8-bit matrix of %d x %d for a product", x.rows, x.cols);
    uint4* out = static_cast<uint4*>(x16);
    void* args[] = {(void*)&x, (void*)&perm, (void*)&status, (void*)&out, (void*)&scales};
    LORA_CUDA_TRY(launch_pdl((const void*)i8_expand_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, st, args));
    return LORA_OK;
}

template <typename T>
static int dequantize_t(const I8View& q, void* out, long long ld, cudaStream_t st) {
    T* op = static_cast<T*>(out);
    void* args[] = {(void*)&q, (void*)&op, (void*)&ld};
    const void* fn = aligned16(out, ld, q.rows, sizeof(T)) ? (const void*)i8_dequantize_kernel<T, true>
                                                           : (const void*)i8_dequantize_kernel<T, false>;
    const unsigned groups = (unsigned)(((long long)q.rows + 7) / 8);
    const dim3 grid((q.cols + 511) / 512, std::min(groups, 65535u), (groups + 65534u) / 65535u);
    LORA_CUDA_TRY(launch_pdl(fn, grid, dim3(256), 0, st, args));
    return LORA_OK;
}

int launch_i8_dequantize(const I8View& q, void* out, int dtype, long long ld, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32: return dequantize_t<float>(q, out, ld, st);
        case LORA_F16: return dequantize_t<__half>(q, out, ld, st);
        default: return dequantize_t<__nv_bfloat16>(q, out, ld, st);
    }
}

template <typename T, int U, bool VEC> static int rmsnorm_l(const NormArgs& a, const RowLaunch& l, cudaStream_t st) {
    static bool done = false;
    const auto fn = i8_rmsnorm_kernel<T, U, VEC>;
    const int rc = allow_smem(fn, done);
    if (rc) return rc;
    void* args[] = {(void*)&a};
    LORA_CUDA_TRY(launch_pdl((const void*)fn, dim3(l.blocks), dim3(l.threads), l.smem, st, args));
    return LORA_OK;
}
template <typename T> static int rmsnorm_t(NormArgs a, cudaStream_t st) {
    const bool vec = aligned16(a.x, a.ldx, a.rows, sizeof(T)) && aligned16(a.residual, a.ldr, a.rows, sizeof(T)) &&
                     aligned16(a.h, a.ldh, a.rows, sizeof(T)) && aligned16(a.y, a.ldy, a.rows, sizeof(T)) &&
                     aligned16(a.w, 0, 1, sizeof(T));
    const RowLaunch l = row_launch(a.rows, a.cols, sizeof(T));
    a.pl = l.pl;
    if (l.U == 1) return vec ? rmsnorm_l<T, 1, true>(a, l, st) : rmsnorm_l<T, 1, false>(a, l, st);
    constexpr int U = sizeof(T) == 4 ? 2 : 4;  // (16384 x 4096 float32: 184 us against 197 with four)
    return vec ? rmsnorm_l<T, U, true>(a, l, st) : rmsnorm_l<T, U, false>(a, l, st);
}

int launch_i8_rmsnorm(const lora_i8_norm& p, cudaStream_t st) {
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = p.x_dev;
    a.residual = p.residual_dev;
    a.w = p.weight_dev;
    a.h = p.residual_out_dev;
    a.y = p.y_dev;
    if (p.out) a.q = i8_view(p.out->codes_dev, p.out->scales_dev, p.out->rows, p.out->cols);
    a.ldx = p.ldx;
    a.ldr = p.ldr;
    a.ldh = p.ldro;
    a.ldy = p.ldy;
    a.eps = p.eps;
    a.rows = p.rows;
    a.cols = p.cols;
    switch (p.dtype) {
        case LORA_F32: return rmsnorm_t<float>(a, st);
        case LORA_F16: return rmsnorm_t<__half>(a, st);
        default: return rmsnorm_t<__nv_bfloat16>(a, st);
    }
}

}  // namespace lora
