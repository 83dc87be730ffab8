// Matrices stored in 8-bit integers with one float32 scale a row: quantisation, reading back, the
// root-mean-square norm that writes its output so, and the entry points of the product and of the linear
// over an 8-bit base weight.
//
// Stored form (lora.h): a row x becomes codes c and a scale s, s = max|x| / 127 rounded to float32 and c
// the whole number nearest x / s (ties to even).  Codes are those of the real quotient, not of a rounded
// one: a 16384 x 4096 batch has hundreds of elements whose float32 quotient rounds onto the border of two
// codes, and with them equal inputs would not give equal bytes on every path.
#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "i8_device.cuh"
#include "kernels.h"

namespace lora {

constexpr float kFltMax = 3.402823466e38f;

// Elements of a row that thread tid of its G holds as vector i: with VEC 8 (i G + tid) .. + 7, loaded 16
// bytes at a time; without (rows off 16-byte boundaries) element e is (8 i + e) G + tid, so that
// neighbouring threads still read neighbours.
template <typename T, bool VEC> struct RowPart {
    static __device__ __forceinline__ int at(int i, int e, int tid, int G) {
        return VEC ? 8 * (i * G + tid) + e : (8 * i + e) * G + tid;
    }
    // zeros past cols
    static __device__ __forceinline__ void load(const T* row, int cols, int i, int tid, int G, float (&v)[8]) {
        const int k = at(i, 0, tid, G);
        if (VEC && k + 8 <= cols) {
            if constexpr (sizeof(T) == 2) {
                unpack8<T>(*reinterpret_cast<const uint4*>(row + k), v);
            } else {
                const float4 a = *reinterpret_cast<const float4*>(row + k);
                const float4 b = *reinterpret_cast<const float4*>(row + k + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                v[e] = j < cols ? to_f32<T>(row[j]) : 0.f;
            }
        }
    }
    static __device__ __forceinline__ void store(T* row, int cols, int i, int tid, int G, const float (&v)[8]) {
        const int k = at(i, 0, tid, G);
        if (VEC && k + 8 <= cols) {
            alignas(16) T w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = from_f32<T>(v[e]);
#pragma unroll
            for (int e = 0; e < (int)(8 * sizeof(T) / 16); ++e)
                reinterpret_cast<uint4*>(row + k)[e] = reinterpret_cast<const uint4*>(w)[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at(i, e, tid, G);
                if (j < cols) row[j] = from_f32<T>(v[e]);
            }
        }
    }
    // codes (0 past cols, up to pitch)
    static __device__ __forceinline__ void store_codes(int8_t* row, int pitch, int i, int tid, int G, const int (&c)[8]) {
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
};

constexpr int kRowThreads = 512;  // at most, a row

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
// ---- quantise ----------------------------------------------------------------------------------------
// One read of x, one write of the codes: bound by memory.  A row is held in registers between its maximum
// and its codes, by a warp (rows of up to 1024 elements) or by a CTA; longer rows than a CTA holds are
// read twice, in pieces.
// F16: codes as float16 into x16 [rows][pitch], row r from row perm[r] of x (see launch_i8_quantize_f16).
template <typename T, int NV, bool VEC, bool F16>
__global__ void __launch_bounds__(kRowThreads)
i8_quantize_kernel(const T* x, long long ld, I8View q, int G, int pieces, const int32_t* perm, const int32_t* status,
                   __half* x16) {
    __shared__ float red[kRowThreads / 32];
    pdl_wait();
    pdl_trigger();
    using Part = RowPart<T, VEC>;
    const int team = threadIdx.x / G, tid = threadIdx.x - team * G;
    const long long r = (long long)blockIdx.x * (blockDim.x / G) + team;
    if (r >= q.rows) return;  // (whole warps; G is the CTA where it is more than a warp)
    const T* row = x + r * ld;
    if constexpr (F16) {
        if (status != nullptr && __ldcg(status) != LORA_OK) return;  // (perm is not valid either)
        if (perm != nullptr) row = x + (long long)__ldcg(perm + r) * ld;
    }
    const int span = G * NV * 8, pitch = (int)q.pitch;
    float v[NV][8];
    float m = 0.f;
    for (int off = (pieces - 1) * span; off >= 0; off -= span) {  // the first piece stays in registers
#pragma unroll
        for (int i = 0; i < NV; ++i) Part::load(row + off, q.cols - off, i, tid, G, v[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(v[i][e]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        for (int w = 0; w < G / 32; ++w) m = max_nan(m, red[w]);
    }
    const float s = i8_scale(m);
    if (tid == 0) q.scales[r] = s;
    const I8Divisor d = i8_divisor(s);
    for (int off = 0; off < pitch; off += span) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (off > 0) Part::load(row + off, q.cols - off, i, tid, G, v[i]);
            if constexpr (F16) {
                float c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = static_cast<float>(i8_code(v[i][e], d));
                RowPart<__half, VEC>::store(x16 + r * pitch + off, pitch - off, i, tid, G, c);
            } else {
                int c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = i8_code(v[i][e], d);
                Part::store_codes(q.codes + r * pitch + off, pitch - off, i, tid, G, c);
            }
        }
    }
}

// Stored codes as float16, rows in the order of perm.  16 codes a thread; bound by memory.
__global__ void __launch_bounds__(256)
i8_expand_kernel(I8View q, const int32_t* perm, const int32_t* status, uint4* x16, float* scales) {
    pdl_wait();
    pdl_trigger();
    if (status != nullptr && __ldcg(status) != LORA_OK) return;
    const int per_row = (int)(q.pitch / 16);
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    const int r = (int)(e / per_row), c = (int)(e - (long long)r * per_row);
    if (r >= q.rows) return;
    const int from = perm ? __ldcg(perm + r) : r;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(q.codes + (size_t)from * q.pitch) + c);
    const uint2 a = i8_to_f16x4(w.x), b = i8_to_f16x4(w.y), f = i8_to_f16x4(w.z), g = i8_to_f16x4(w.w);
    x16[2 * e] = make_uint4(a.x, a.y, b.x, b.y);
    x16[2 * e + 1] = make_uint4(f.x, f.y, g.x, g.y);
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
// the second parts decide.  Bound by memory: each row is read once and held in registers.
struct NormArgs {
    const void* x;
    const void* residual;  // nullable
    const void* w;
    void* h;               // nullable: where x + residual goes
    void* y;               // nullable
    I8View q;              // codes nullable
    long long ldx, ldr, ldh, ldy;
    float eps;
    int rows, cols, G, pieces;
};

struct Two {
    float hi, lo;
};

template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
i8_rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[kRowThreads / 32][4];
    pdl_wait();
    pdl_trigger();
    using Part = RowPart<T, VEC>;
    const int G = a.G, team = threadIdx.x / G, tid = threadIdx.x - team * G, cols = a.cols;
    const long long r = (long long)blockIdx.x * (blockDim.x / G) + team;
    if (r >= a.rows) return;
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    const T* rr = a.residual ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    T* hr = a.h ? static_cast<T*>(a.h) + r * a.ldh : nullptr;
    const T* wr = static_cast<const T*>(a.w);
    const int span = G * NV * 8, pitch = a.q.codes ? (int)a.q.pitch : cols;
    float h[NV][8];
    // x + residual as it is stored; a later pass reads the stored sum again where there is one
    auto load_h = [&](int off, bool again) {
        const T* src = again && hr ? hr : xr;
#pragma unroll
        for (int i = 0; i < NV; ++i) Part::load(src + off, cols - off, i, tid, G, h[i]);
        if (again && hr) return;
        if (rr) {
            float t[NV][8];
#pragma unroll
            for (int i = 0; i < NV; ++i) Part::load(rr + off, cols - off, i, tid, G, t[i]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = to_f32<T>(from_f32<T>(h[i][e] + t[i][e]));
        }
        if (hr)
#pragma unroll
            for (int i = 0; i < NV; ++i) Part::store(hr + off, cols - off, i, tid, G, h[i]);
    };
    float f = 1.f;  // the row is taken times f
    Two r2;         // r / f
    MaxPair m;      // max |u|
    for (int attempt = 0;; ++attempt) {
        Two ss{0.f, 0.f};
        m = MaxPair{0.f, 0.f};
        for (int off = (a.pieces - 1) * span; off >= 0; off -= span) {
            if (attempt == 0 || a.pieces > 1) load_h(off, attempt > 0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[8];
                Part::load(wr + off, cols - off, i, tid, G, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float g = h[i][e] * f, sq = __fmul_rn(g, g);
                    float err;
                    ss.hi = two_sum(ss.hi, sq, err);
                    if (sizeof(T) == 4) err += fmaf(g, g, -sq);  // (a 16-bit number's square is exact)
                    ss.lo += err;
                    const float u = __fmul_rn(g, w[e]), au = fabsf(u);
                    if constexpr (sizeof(T) == 4) {
                        const float l = fmaf(g, w[e], -u);
                        m = max_pair(m, MaxPair{au, u < 0.f ? -l : l});
                    } else {
                        m.hi = max_nan(m.hi, au);
                    }
                }
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            float err;
            const float oh = __shfl_xor_sync(0xffffffffu, ss.hi, d), ol = __shfl_xor_sync(0xffffffffu, ss.lo, d);
            ss.hi = two_sum(ss.hi, oh, err);
            ss.lo += ol + err;
            m = max_pair(m, MaxPair{__shfl_xor_sync(0xffffffffu, m.hi, d), __shfl_xor_sync(0xffffffffu, m.lo, d)});
        }
        if (G > 32) {
            if (attempt > 0) __syncthreads();  // (the CTA is one row: all or none come here)
            if ((threadIdx.x & 31) == 0)
                red[threadIdx.x >> 5][0] = ss.hi, red[threadIdx.x >> 5][1] = ss.lo, red[threadIdx.x >> 5][2] = m.hi,
                red[threadIdx.x >> 5][3] = m.lo;
            __syncthreads();
            ss = Two{0.f, 0.f};
            m = MaxPair{0.f, 0.f};
            for (int k = 0; k < G / 32; ++k) {
                float err;
                ss.hi = two_sum(ss.hi, red[k][0], err);
                ss.lo += red[k][1] + err;
                m = max_pair(m, MaxPair{red[k][2], red[k][3]});
            }
        }
        // the mean, + eps, its inverse root
        const float n = static_cast<float>(cols), q0 = __fdiv_rn(ss.hi, n);
        const float q1 = (fmaf(-q0, n, ss.hi) + ss.lo) / n;
        float err;
        const float hi = two_sum(q0, a.eps * f * f, err), lo = err + q1;
        const float r0 = rsqrtf(hi), p = __fmul_rn(r0, r0);
        float e = fmaf(-hi, p, 1.f);
        e = fmaf(-hi, fmaf(r0, r0, -p), e);
        e = fmaf(-lo, p, e);
        r2 = Two{r0, hi <= kFltMax ? r0 * fmaf(0.375f * e, e, 0.5f * e) : 0.f};
        // squares that overflow float32 (elements from about 2^50 on) are taken of a smaller row
        if (ss.hi <= 1e30f || attempt > 0) break;
        f = 7.888609052210118e-31f;  // 2^-100
    }
    const float rsum = r2.hi + r2.lo;
    float c = 1.f;
    Two g{0.f, 0.f};
    if (a.q.codes) {
        // s = max|u| r / 127
        const float t = __fmul_rn(m.hi, r2.hi);
        const float tl = fmaf(m.hi, r2.hi, -t) + fmaf(m.hi, r2.lo, m.lo * r2.hi);
        const float s0 = __fdiv_rn(t, 127.f);
        float s = s0 + (fmaf(-127.f, s0, t) + tl) / 127.f;
        if (!(m.hi <= kFltMax) || !(s <= kFltMax)) s = __uint_as_float(0x7fc00000u);
        if (tid == 0) a.q.scales[r] = s;
        if (s > 0.f) {
            c = s < 1e-20f ? 18446744073709551616.f : 1.f;  // 2^64: r / s stays in range
            const float sc = s * c;
            g.hi = __fdiv_rn(r2.hi, sc);
            g.lo = (fmaf(-g.hi, sc, r2.hi) + r2.lo) / sc;
        }
    }
    for (int off = 0; off < pitch; off += span) {
        if (off > 0) load_h(off, true);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[8], y[8];
            int code[8];
            Part::load(wr + off, cols - off, i, tid, G, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gh = h[i][e] * f, u = __fmul_rn(gh, w[e]);
                y[e] = u * rsum;
                const float uc = g.hi > 0.f ? u * c : 0.f, v = __fmul_rn(uc, g.hi);
                float k = rintf(v);
                if (fabsf(v - k) > 0.4999f) {
                    const float side = v > k ? 1.f : -1.f;
                    float rest = fmaf(uc, g.hi, -v) + uc * g.lo;
                    if (sizeof(T) == 4) rest += fmaf(gh, w[e], -u) * c * g.hi;
                    const float past = side * ((v - (k + 0.5f * side)) + rest);
                    if (past > 0.f || (past == 0.f && (static_cast<int>(k) & 1) != 0)) k += side;
                }
                code[e] = static_cast<int>(fminf(fmaxf(k, -127.f), 127.f));
            }
            if (a.y) Part::store(static_cast<T*>(a.y) + r * a.ldy + off, cols - off, i, tid, G, y);
            if (a.q.codes) Part::store_codes(a.q.codes + r * a.q.pitch + off, pitch - off, i, tid, G, code);
        }
    }
}

// Threads a row and vectors of 8 a thread.  Few rows: as many threads as the row has vectors, for its
// latency; many: four vectors a thread, so that enough loads are in flight.
struct RowPlan {
    int G, nv, pieces, threads;
    unsigned blocks;
};
static RowPlan row_plan(int rows, int cols) {
    RowPlan p;
    const int vecs = (int)(i8_pitch(cols) / 8);
    p.nv = rows <= 2 * num_sms() && vecs <= kRowThreads ? 1 : 4;
    const int need = (vecs + p.nv - 1) / p.nv;
    p.G = std::min(kRowThreads, (need + 31) / 32 * 32);
    p.pieces = (need + p.G - 1) / p.G;
    p.threads = p.G > 32 ? p.G : 256;
    const int per = p.threads / p.G;
    p.blocks = (unsigned)(((long long)rows + per - 1) / per);
    return p;
}

static bool aligned16(const void* p, long long ld, int rows, size_t elt) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (ld * (long long)elt) % 16 == 0);
}

template <typename T, bool F16>
static int quantize_t(const void* x, long long ld, const I8View& q, const int32_t* perm, const int32_t* status, void* x16,
                      cudaStream_t st) {
    const bool vec = aligned16(x, ld, q.rows, sizeof(T));
    const RowPlan p = row_plan(q.rows, q.cols);
    const T* xp = static_cast<const T*>(x);
    __half* hp = static_cast<__half*>(x16);
    void* args[] = {(void*)&xp, (void*)&ld, (void*)&q, (void*)&p.G, (void*)&p.pieces, (void*)&perm, (void*)&status, (void*)&hp};
    const void* fn = p.nv == 1
                         ? (vec ? (const void*)i8_quantize_kernel<T, 1, true, F16> : (const void*)i8_quantize_kernel<T, 1, false, F16>)
                         : (vec ? (const void*)i8_quantize_kernel<T, 4, true, F16> : (const void*)i8_quantize_kernel<T, 4, false, F16>);
    LORA_CUDA_TRY(launch_pdl(fn, dim3(p.blocks), dim3(p.threads), 0, st, args));
    return LORA_OK;
}

int launch_i8_quantize(const void* x, int dtype, long long ld, const I8View& q, cudaStream_t st) {
    if (q.rows == 0) return LORA_OK;
    switch (dtype) {
        case LORA_F32: return quantize_t<float, false>(x, ld, q, nullptr, nullptr, nullptr, st);
        case LORA_F16: return quantize_t<__half, false>(x, ld, q, nullptr, nullptr, nullptr, st);
        default: return quantize_t<__nv_bfloat16, false>(x, ld, q, nullptr, nullptr, nullptr, st);
    }
}

int launch_i8_quantize_f16(const void* x, int dtype, int rows, int cols, const int32_t* perm, const int32_t* status,
                           void* x16, float* scales, cudaStream_t st) {
    const I8View q = i8_view(nullptr, scales, rows, cols);
    switch (dtype) {
        case LORA_F32: return quantize_t<float, true>(x, cols, q, perm, status, x16, st);
        case LORA_F16: return quantize_t<__half, true>(x, cols, q, perm, status, x16, st);
        default: return quantize_t<__nv_bfloat16, true>(x, cols, q, perm, status, x16, st);
    }
}

int launch_i8_expand(const I8View& x, const int32_t* perm, const int32_t* status, void* x16, float* scales, cudaStream_t st) {
    const long long chunks = (long long)x.rows * (long long)(x.pitch / 16);
    uint4* out = static_cast<uint4*>(x16);
    void* args[] = {(void*)&x, (void*)&perm, (void*)&status, (void*)&out, (void*)&scales};
    if (chunks > 256LL * INT_MAX) return set_error(LORA_EUNSUP, "8-bit matrix of %d rows", x.rows);
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

template <typename T>
static int rmsnorm_t(NormArgs a, cudaStream_t st) {
    const RowPlan p = row_plan(a.rows, a.cols);
    a.G = p.G;
    a.pieces = p.pieces;
    const bool vec = aligned16(a.x, a.ldx, a.rows, sizeof(T)) && aligned16(a.residual, a.ldr, a.rows, sizeof(T)) &&
                     aligned16(a.h, a.ldh, a.rows, sizeof(T)) && aligned16(a.y, a.ldy, a.rows, sizeof(T)) &&
                     aligned16(a.w, 0, 1, sizeof(T));
    void* args[] = {(void*)&a};
    const void* fn = p.nv == 1 ? (vec ? (const void*)i8_rmsnorm_kernel<T, 1, true> : (const void*)i8_rmsnorm_kernel<T, 1, false>)
                               : (vec ? (const void*)i8_rmsnorm_kernel<T, 4, true> : (const void*)i8_rmsnorm_kernel<T, 4, false>);
    LORA_CUDA_TRY(launch_pdl(fn, dim3(p.blocks), dim3(p.threads), 0, st, args));
    return LORA_OK;
}

// 128 x 128 x cols stays below 2^31
constexpr int kI8MaxCols = 131071;

static int check_shape(int rows, int cols) {
    if (rows < 0 || cols < 1) return set_error(LORA_EINVAL, "8-bit matrix of %d x %d", rows, cols);
    if (cols > kI8MaxCols) return set_error(LORA_EUNSUP, "8-bit matrix of %d columns (at most %d)", cols, kI8MaxCols);
    return LORA_OK;
}

static int check_matrix(const lora_i8_matrix* m, const char* what) {
    if (!m) return set_error(LORA_EINVAL, "%s is NULL", what);
    const int rc = check_shape(m->rows, m->cols);
    if (rc || m->rows == 0) return rc;
    if (!m->codes_dev || !m->scales_dev) return set_error(LORA_EINVAL, "%s has no codes or scales", what);
    if ((reinterpret_cast<uintptr_t>(m->codes_dev) | reinterpret_cast<uintptr_t>(m->scales_dev)) % 256)
        return set_error(LORA_EINVAL, "%s: codes and scales must be 256-byte aligned", what);
    return LORA_OK;
}

static int check_dtype(int dtype) {
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return set_error(LORA_EINVAL, "bad dtype %d", dtype);
    return LORA_OK;
}

// A strided [rows, cols] array of dtype.
static int check_rows(const void* p, int dtype, int64_t ld, int rows, int cols, const char* what) {
    const int rc = check_dtype(dtype);
    if (rc) return rc;
    if (ld < cols) return set_error(LORA_EINVAL, "%s: row stride %lld below %d columns", what, (long long)ld, cols);
    if (rows == 0) return LORA_OK;
    if (!p) return set_error(LORA_EINVAL, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % dtype_size(dtype)) return set_error(LORA_EINVAL, "%s is misaligned", what);
    return LORA_OK;
}

static I8View view_of(const lora_i8_matrix* m) { return i8_view(m->codes_dev, m->scales_dev, m->rows, m->cols); }

// Up to this many tokens the dot products of i8_small.cu.
constexpr int kI8Small = 8;

// Above this many tokens the pair kernel.
constexpr int kI8Tile = 256;

// What a product keeps in its workspace: x in float16 codes and its scales, and above kI8Tile rows the weight
// in float16 codes.
struct I8ProductWs {
    size_t scales_off, w_off, total;
};
static I8ProductWs product_ws(int n, int h_out, int h_in) {
    I8ProductWs L = {0, 0, 0};
    if (n <= kI8Small) return L;
    L.scales_off = align256((size_t)n * i8_pitch(h_in) * 2);
    L.w_off = L.scales_off + align256((size_t)n * 4);
    L.total = L.w_off + (n > kI8Tile ? align256((size_t)h_out * i8_pitch(h_in) * 2) : 0);
    return L;
}

// Workspace of lora_i8_linear_fwd: the shrink output in its K parts, x's codes (in bytes for a few tokens,
// else in float16) and scales, the weight in float16 codes.
struct I8WsLayout {
    size_t codes_off, scales_off, w_off, total;
};
static int ws_layout(lora_pool_t pool, int n, I8WsLayout* L) {
    if (n < 0) return set_error(LORA_EINVAL, "n_tokens < 0");
    const PoolView pv = pool_view(pool);
    if (pv.h_in > kI8MaxCols) return set_error(LORA_EUNSUP, "8-bit linear of %d features (at most %d)", pv.h_in, kI8MaxCols);
    // rows of shrink output over all K parts: at most what any batch of up to n tokens has (16-bit: at most
    // 256 / n parts up to 256 tokens; float32: 24 parts, and four CTAs an SM of 64 tokens)
    const long long m = std::max(n, 1);
    const long long rows = std::max(m, pv.dtype == LORA_F32 ? std::min(24 * m, 4LL * num_sms() * 64) : std::min(4 * m, 256LL));
    L->codes_off = align256((size_t)rows * pv.R * 4);
    const I8ProductWs P = product_ws(n, pv.h_out, pv.h_in);
    L->scales_off = L->codes_off + (n <= kI8Small ? align256((size_t)n * i8_pitch(pv.h_in)) : P.scales_off);
    L->w_off = L->scales_off + align256((size_t)n * 4);
    L->total = L->w_off + P.total - P.w_off;
    return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" {

int lora_i8_bytes(int rows, int cols, size_t* codes_bytes, size_t* scales_bytes) {
    if (!codes_bytes || !scales_bytes) return set_error(LORA_EINVAL, "codes_bytes/scales_bytes is NULL");
    const int rc = check_shape(rows, cols);
    if (rc) return rc;
    *codes_bytes = (size_t)rows * i8_pitch(cols);
    *scales_bytes = (size_t)rows * 4;
    return LORA_OK;
}

int lora_i8_quantize(const void* x_dev, int dtype, int64_t ld, const lora_i8_matrix* out, void* stream) {
    int rc = check_matrix(out, "out");
    if (rc) return rc;
    rc = check_rows(x_dev, dtype, ld, out->rows, out->cols, "x");
    if (rc) return rc;
    return launch_i8_quantize(x_dev, dtype, ld, view_of(out), static_cast<cudaStream_t>(stream));
}

int lora_i8_dequantize(const lora_i8_matrix* q, void* out_dev, int dtype, int64_t ld, void* stream) {
    int rc = check_matrix(q, "q");
    if (rc) return rc;
    rc = check_rows(out_dev, dtype, ld, q->rows, q->cols, "out");
    if (rc || q->rows == 0) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case LORA_F32: return dequantize_t<float>(view_of(q), out_dev, ld, st);
        case LORA_F16: return dequantize_t<__half>(view_of(q), out_dev, ld, st);
        default: return dequantize_t<__nv_bfloat16>(view_of(q), out_dev, ld, st);
    }
}

int lora_i8_rmsnorm(const lora_i8_norm* p, void* stream) {
    if (!p) return set_error(LORA_EINVAL, "the arguments are NULL");
    int rc = check_dtype(p->dtype);
    if (!rc) rc = check_shape(p->rows, p->cols);
    if (rc) return rc;
    if (!(p->eps >= 1e-12f && p->eps <= 1.f)) return set_error(LORA_EINVAL, "eps %g outside [1e-12, 1]", (double)p->eps);
    if (!p->y_dev && !p->out) return set_error(LORA_EINVAL, "neither y nor out is wanted");
    if (p->residual_dev && !p->residual_out_dev) return set_error(LORA_EINVAL, "residual without residual_out");
    rc = check_rows(p->x_dev, p->dtype, p->ldx, p->rows, p->cols, "x");
    if (!rc) rc = check_rows(p->weight_dev, p->dtype, p->cols, p->rows ? 1 : 0, p->cols, "weight");
    if (!rc && p->residual_dev) rc = check_rows(p->residual_dev, p->dtype, p->ldr, p->rows, p->cols, "residual");
    if (!rc && p->residual_out_dev)
        rc = check_rows(p->residual_out_dev, p->dtype, p->ldro, p->rows, p->cols, "residual_out");
    if (!rc && p->y_dev) rc = check_rows(p->y_dev, p->dtype, p->ldy, p->rows, p->cols, "y");
    if (!rc && p->out) rc = check_matrix(p->out, "out");
    if (rc) return rc;
    if (p->out && (p->out->rows != p->rows || p->out->cols != p->cols))
        return set_error(LORA_EINVAL, "out is %d x %d, x %d x %d", p->out->rows, p->out->cols, p->rows, p->cols);
    if (p->rows == 0) return LORA_OK;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = p->x_dev;
    a.residual = p->residual_dev;
    a.w = p->weight_dev;
    a.h = p->residual_out_dev;
    a.y = p->y_dev;
    if (p->out) a.q = view_of(p->out);
    a.ldx = p->ldx;
    a.ldr = p->ldr;
    a.ldh = p->ldro;
    a.ldy = p->ldy;
    a.eps = p->eps;
    a.rows = p->rows;
    a.cols = p->cols;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p->dtype) {
        case LORA_F32: return rmsnorm_t<float>(a, st);
        case LORA_F16: return rmsnorm_t<__half>(a, st);
        default: return rmsnorm_t<__nv_bfloat16>(a, st);
    }
}

int lora_i8_matmul_workspace_bytes(int x_rows, int w_rows, int cols, size_t* bytes) {
    if (!bytes) return set_error(LORA_EINVAL, "bytes is NULL");
    int rc = check_shape(x_rows, cols);
    if (!rc) rc = check_shape(w_rows, cols);
    if (rc) return rc;
    *bytes = product_ws(x_rows, w_rows, cols).total;
    return LORA_OK;
}

int lora_i8_matmul(const lora_i8_matrix* x, const lora_i8_matrix* w, void* y_dev, int dtype, int64_t ldy, void* ws_dev,
                   size_t ws_bytes, void* stream) {
    int rc = check_matrix(x, "x");
    if (!rc) rc = check_matrix(w, "w");
    if (rc) return rc;
    if (x->cols != w->cols) return set_error(LORA_EINVAL, "x has %d columns, w %d", x->cols, w->cols);
    rc = check_rows(y_dev, dtype, ldy, w->rows ? x->rows : 0, w->rows, "y");
    if (rc || x->rows == 0 || w->rows == 0) return rc;
    const I8ProductWs L = product_ws(x->rows, w->rows, x->cols);
    if (L.total && !ws_dev) return set_error(LORA_EINVAL, "ws is NULL");
    if (reinterpret_cast<uintptr_t>(ws_dev) % 256) return set_error(LORA_EINVAL, "ws must be 256-byte aligned");
    if (ws_bytes < L.total)
        return set_error(LORA_ENOSPACE, "8-bit product workspace needs %zu bytes, got %zu", L.total, ws_bytes);
    const I8View xv = view_of(x), wv = view_of(w);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x->rows <= kI8Small) return launch_i8_small(xv, wv, y_dev, dtype, ldy, nullptr, /*early_w=*/false, nullptr, st);
    char* ws = static_cast<char*>(ws_dev);
    float* sx = reinterpret_cast<float*>(ws + L.scales_off);
    rc = launch_i8_expand(xv, nullptr, nullptr, ws, sx, st);
    if (rc) return rc;
    const I8Rows rows = {ws, sx, nullptr, x->rows, x->cols};
    if (x->rows <= kI8Tile)
        return launch_i8_tile(rows, wv, y_dev, dtype, ldy, nullptr, /*early=*/1, /*release=*/false, nullptr, st);
    rc = launch_i8_expand(wv, nullptr, nullptr, ws + L.w_off, nullptr, st);
    if (rc) return rc;
    const I8Rows wrows = {ws + L.w_off, wv.scales, nullptr, w->rows, w->cols};
    return launch_i8_pair(rows, wrows, y_dev, dtype, ldy, nullptr, /*release=*/false, nullptr, st);
}

int lora_i8_linear_workspace_bytes(lora_pool_t pool, int n_tokens, size_t* bytes) {
    if (!pool || !bytes) return set_error(LORA_EINVAL, "pool/bytes is NULL");
    I8WsLayout L;
    const int rc = ws_layout(pool, n_tokens, &L);
    if (rc) return rc;
    *bytes = L.total;
    return LORA_OK;
}

int lora_i8_linear_fwd(lora_pool_t pool, const lora_i8_matrix* w, const void* x_dev, const lora_i8_matrix* xq,
                       void* y_dev, const lora_segments* seg, void* ws_dev, size_t ws_bytes, void* stream) {
    if (!pool || !seg) return set_error(LORA_EINVAL, "pool/seg is NULL");
    const PoolView pv = pool_view(pool);
    const int n = seg->n_tokens;
    if (seg->n_slots != pv.S)
        return set_error(LORA_EINVAL, "segments were built for %d slots, pool has %d", seg->n_slots, pv.S);
    int rc = check_matrix(w, "w");
    if (rc) return rc;
    if (w->rows != pv.h_out || w->cols != pv.h_in)
        return set_error(LORA_EINVAL, "w is %d x %d, the pool's linear %d x %d", w->rows, w->cols, pv.h_out, pv.h_in);
    if (xq) {
        rc = check_matrix(xq, "xq");
        if (rc) return rc;
        if (xq->rows != n || xq->cols != pv.h_in)
            return set_error(LORA_EINVAL, "xq is %d x %d, x %d x %d", xq->rows, xq->cols, n, pv.h_in);
    }
    if (n == 0) return LORA_OK;
    if (!x_dev || !y_dev || !ws_dev) return set_error(LORA_EINVAL, "x/y/ws is NULL");
    const size_t align = pv.dtype == LORA_F32 ? 4 : 16;
    if ((reinterpret_cast<uintptr_t>(x_dev) | reinterpret_cast<uintptr_t>(y_dev)) % align)
        return set_error(LORA_EINVAL, "x/y must be %zu-byte aligned", align);
    if (reinterpret_cast<uintptr_t>(ws_dev) % 256) return set_error(LORA_EINVAL, "ws must be 256-byte aligned");
    I8WsLayout L;
    rc = ws_layout(pool, n, &L);
    if (rc) return rc;
    if (ws_bytes < L.total)
        return set_error(LORA_ENOSPACE, "8-bit linear workspace needs %zu bytes, got %zu", L.total, ws_bytes);
    char* ws = static_cast<char*>(ws_dev);
    float* s_buf = reinterpret_cast<float*>(ws);
    float* sx = reinterpret_cast<float*>(ws + L.scales_off);
    const SegView sv = seg_view(seg);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool few = n <= kI8Small;
    const I8View q = xq ? view_of(xq) : i8_view(ws + L.codes_off, sx, n, pv.h_in);
    if (!few)  // rows in the order of the segments
        rc = xq ? launch_i8_expand(q, sv.perm, sv.status, ws + L.codes_off, sx, st)
                : launch_i8_quantize_f16(x_dev, pv.dtype, n, pv.h_in, sv.perm, sv.status, ws + L.codes_off, sx, st);
    else if (!xq)
        rc = launch_i8_quantize(x_dev, pv.dtype, pv.h_in, q, st);
    int s_parts = 1;
    if (!rc) {
        if (pv.dtype == LORA_F32) {
            s_parts = f32_shrink_parts(pv, n);
            rc = launch_f32_shrink(pv, sv, x_dev, s_buf, st);
        } else if (n > 256 && shrink_tc_supported(pv)) {
            rc = launch_shrink_tc(pv, sv, x_dev, s_buf, st);
        } else {
            rc = launch_shrink(pv, sv, x_dev, s_buf, st, /*tiled=*/n > 256, &s_parts);
        }
    }
    if (rc) return rc;
    const I8Lora lora = {&pv, sv.idx, s_buf, s_parts};
    if (few) return launch_i8_small(q, view_of(w), y_dev, pv.dtype, pv.h_out, sv.status, /*early_w=*/true, &lora, st);
    const I8Rows rows = {ws + L.codes_off, sx, sv.perm, n, pv.h_in};
    if (n > kI8Tile) {
        const I8View wv = view_of(w);
        rc = launch_i8_expand(wv, nullptr, nullptr, ws + L.w_off, nullptr, st);
        if (rc) return rc;
        const I8Rows wrows = {ws + L.w_off, wv.scales, nullptr, wv.rows, wv.cols};
        rc = launch_i8_pair(rows, wrows, y_dev, pv.dtype, pv.h_out, sv.status, /*release=*/true, &lora, st);
        if (rc || pv.dtype != LORA_F32) return rc;
        return launch_f32_expand(pv, sv, s_buf, s_parts, y_dev, st);
    }
    return launch_i8_tile(rows, view_of(w), y_dev, pv.dtype, pv.h_out, sv.status, /*early=*/2, /*release=*/true, &lora, st);
}

}  // extern "C"
