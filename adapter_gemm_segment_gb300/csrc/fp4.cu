// Microscaled 4-bit matrices (MXFP4): quantisation, reading back, and the entry points of the
// linear over a 4-bit base weight.
//
// Stored form (lora.h): rows of 4-bit codes (e2m1: sign, two exponent bits, one mantissa bit) and,
// per block of 32 elements, one power-of-two scale byte, the scale bytes in tiles of 128 rows x 4
// blocks.  With E the biased float32 exponent of the block's largest |x|, the scale byte is
// max(E - 2, 0): the largest element then lies in [4, 8) times the scale, of which [6, 8) saturates
// at 6.  The factor 2^(127 - byte) and the product with it are exact in float32, so the rounding to
// e2m1 is the only one.
//
// Both kernels move every byte once and are bound by memory: 16384 x 4096 bf16, 134 MB of x and 36 MB
// stored, quantised and read back one after the other in 51.9 us together, 6.5 TB/s, against 50.1 at the
// measured copy rate; below about 4 MB by the launch (one row of 4096: 4 us each).  A warp takes 256
// columns of the four rows r, r + 32, r + 64, r + 96 of a 128-row tile: a lane holds 8 consecutive
// elements of each row (16-byte loads of 16-bit data, a warp's lanes side by side), four lanes share a
// block (two shuffles give its maximum), and the 4 x 4 scale bytes of those rows' four blocks are 16
// consecutive bytes of a scale tile, written by one lane.
#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "fp4_device.cuh"
#include "kernels.h"

namespace lora {

constexpr int kFp4Threads = 256;  // 8 warps: 8 of the 32 row quadruples of a row tile
constexpr int kFp4Cols = 256;     // columns per warp

// 8 elements starting at column c of a row (zeros past cols), in loads of W bytes: the widest of 16, 4
// and the element's size that every row is aligned to.  (2392 x 4074 float16 at a row stride of 4174, in
// elements: 4 bytes at a time 6.3 us, singly, at 4173, 7.8 us.)
template <typename T, int W>
__device__ __forceinline__ Raw8<T> load8(const T* __restrict__ row, int c, int cols) {
    Raw8<T> r;
    if (W > (int)sizeof(T) && c + 8 <= cols) {
        if constexpr (W == 4) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(row + c);
            const uint4 v = make_uint4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
            memcpy(&r, &v, 16);
        } else if constexpr (sizeof(T) == 2) {
            r.v = __ldcs(reinterpret_cast<const uint4*>(row + c));
        } else {
            r.a = __ldcs(reinterpret_cast<const float4*>(row + c));
            r.b = __ldcs(reinterpret_cast<const float4*>(row + c + 4));
        }
        return r;
    }
    alignas(16) T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? row[c + e] : from_f32<T>(0.f);
    memcpy(&r, v, sizeof(r));
    return r;
}
// That width for rows of a strided array.
static int row_width(const void* p, long long ld, size_t elt) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (long long)elt);
    return a % 16 == 0 ? 16 : a % 4 == 0 ? 4 : 2;
}

template <typename T, int W>
__global__ void __launch_bounds__(kFp4Threads)
fp4_quantize_kernel(const T* __restrict__ x, long long ld, Fp4View q) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r32 = blockIdx.y * 8 + warp;  // row within each 32-row quarter
    const int r0 = blockIdx.z * 128 + r32;
    const int c = blockIdx.x * kFp4Cols + lane * 8;
    Raw8<T> v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j;
        if (r < q.rows)
            v[j] = load8<T, W>(x + (long long)r * ld, c, q.cols);
        else
            memset(&v[j], 0, sizeof(v[j]));
    }
    uint32_t codes[4], sw[4];
    quantise_rows<T, 4>(v, codes, sw, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j;
        // c / 32 < blocks: the last block's codes past cols are written (as zeros) too
        if (r < q.rows && c / 32 < q.blocks)
            *reinterpret_cast<uint32_t*>(q.codes + (size_t)r * q.pitch + c / 2) = codes[j];
    }
    if ((lane & 15) == 0) {
        const size_t tile = (size_t)blockIdx.z * q.ktiles + blockIdx.x * 2 + (lane >> 4);
        *reinterpret_cast<uint4*>(q.scales + tile * 512 + r32 * 16) = make_uint4(sw[0], sw[1], sw[2], sw[3]);
    }
}

// Two e2m1 codes of a byte to float32 values times s.
__device__ __forceinline__ float2 decode_e2m1x2(uint32_t byte, float s) {
    uint32_t h2;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.u8.u32 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h2)
        : "r"(byte));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    return make_float2(v.x * s, v.y * s);
}

// 2^(byte - 127); 2^-127 is a subnormal float32, byte 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7fc00000u)
                                                                  : __uint_as_float(byte << 23);
}

template <typename T, int W>
__global__ void __launch_bounds__(kFp4Threads)
fp4_dequantize_kernel(Fp4View q, T* __restrict__ out, long long ld) {
    // No early release of the kernels behind: out may be the weight of a 16-bit linear, whose GEMM streams
    // it without waiting for more than its release.
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r32 = blockIdx.y * 8 + warp;
    const int r0 = blockIdx.z * 128 + r32;
    const int c = blockIdx.x * kFp4Cols + lane * 8;
    const bool live = c < q.cols;
    const size_t tile = (size_t)blockIdx.z * q.ktiles + blockIdx.x * 2 + (lane >> 4);
    const uint4 sv = __ldg(reinterpret_cast<const uint4*>(q.scales + tile * 512 + r32 * 16));
    const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
    uint32_t codes[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j;
        codes[j] = live && r < q.rows ? __ldg(reinterpret_cast<const uint32_t*>(q.codes + (size_t)r * q.pitch + c / 2)) : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j;
        if (r >= q.rows) break;
        const float s = scale_value((sw[j] >> (8 * ((lane >> 2) & 3))) & 255u);
        alignas(16) T v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = decode_e2m1x2((codes[j] >> (8 * e)) & 255u, s);
            v[2 * e] = from_f32<T>(f.x);
            v[2 * e + 1] = from_f32<T>(f.y);
        }
        T* row = out + (long long)r * ld;
        if constexpr (W == 16) {
            if (c + 8 <= q.cols) {
#pragma unroll
                for (int e = 0; e < (int)(8 * sizeof(T) / 16); ++e)
                    reinterpret_cast<uint4*>(row + c)[e] = reinterpret_cast<const uint4*>(v)[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < q.cols) row[c + e] = v[e];
            }
        } else {
            // Rows off 16-byte boundaries: the warp's 256 values change lanes through shared memory, so
            // that neighbouring lanes write neighbours (2392 x 4073 float16: 30 us without, 5.9 with)
            __shared__ __align__(16) T staged[kFp4Threads / 32][kFp4Cols];
            T* st = staged[warp];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < (int)(8 * sizeof(T) / 16); ++e)
                reinterpret_cast<uint4*>(st + lane * 8)[e] = reinterpret_cast<const uint4*>(v)[e];
            __syncwarp();
            const int c0 = blockIdx.x * kFp4Cols;
            constexpr int per = W > (int)sizeof(T) ? W / (int)sizeof(T) : 1;  // elements per store
#pragma unroll
            for (int e = lane * per; e < kFp4Cols; e += 32 * per) {
                if (per == 2 && c0 + e + 2 <= q.cols) {
                    *reinterpret_cast<uint32_t*>(row + c0 + e) = *reinterpret_cast<const uint32_t*>(st + e);
                } else {
#pragma unroll
                    for (int i = 0; i < per; ++i)
                        if (c0 + e + i < q.cols) row[c0 + e + i] = st[e + i];
                }
            }
        }
    }
}

__device__ __forceinline__ void unpack_raw(const Raw8<__half>& v, float (&f)[8]) { unpack8<__half>(v.v, f); }
__device__ __forceinline__ void unpack_raw(const Raw8<__nv_bfloat16>& v, float (&f)[8]) { unpack8<__nv_bfloat16>(v.v, f); }
__device__ __forceinline__ void unpack_raw(const Raw8<float>& v, float (&f)[8]) {
    f[0] = v.a.x, f[1] = v.a.y, f[2] = v.a.z, f[3] = v.a.w;
    f[4] = v.b.x, f[5] = v.b.y, f[6] = v.b.z, f[7] = v.b.w;
}

// ---- before the product of a small batch: x quantised and the per-token shrink, one launch -------
// One CTA per (token, 8 adapter rows, K part), 128 threads with 8 consecutive features each in sweeps
// of 1024, as the framework's per-token shrink; the CTAs of the first 8 rows also quantise the features
// they hold.  Bound by latency: a chain of slot, A rows and a reduction.  W: bytes of a load, as above
// (16-bit pools have rows on 16-byte boundaries).
template <typename T, int W>
__global__ void __launch_bounds__(128)
fp4_front_kernel(PoolView pool, SegView seg, const T* __restrict__ x, Fp4View q, float* __restrict__ s_out) {
    __shared__ float red[4][8];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, g = blockIdx.y, ks = blockIdx.z;
    const int h = pool.h_in, R = pool.R, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = q.ktiles * 128;  // the last block of scale tiles is filled up with zeros
    const int sweeps = ((width + 1023) / 1024 + gridDim.z - 1) / gridDim.z;
    const int k_beg = ks * sweeps * 1024, k_end = min(width, k_beg + sweeps * 1024);
    // independent loads first
    const int status = __ldcg(seg.status);
    const int slot = __ldcg(seg.idx + t);
    const bool lora = slot >= 0 && status == LORA_OK && g * 8 < R;
    const SlotEntry e = lora ? pool.table[slot] : SlotEntry{0, 0, 0.f, 0};
    const T* xr = x + (size_t)t * h;
    const T* Ab = static_cast<const T*>(pool.A) + ((size_t)max(slot, 0) * R + (size_t)g * 8) * h;
    const bool rows = lora && g * 8 < e.rank;  // rows past the adapter's rank are zeros
    const bool store = g == 0 && q.codes != nullptr && status == LORA_OK;
    float acc[8] = {};
    for (int k0 = k_beg; k0 < k_end; k0 += 1024) {
        const int k = k0 + threadIdx.x * 8;
        Raw8<T> v[2], av[8];
        memset(v, 0, sizeof(v));
        if (k < h) {
            if constexpr (sizeof(T) == 2)
                v[0].v = __ldcg(reinterpret_cast<const uint4*>(xr + k));
            else
                v[0] = load8<T, W>(xr, k, h);
            if (rows)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if constexpr (sizeof(T) == 2)
                        av[r].v = __ldg(reinterpret_cast<const uint4*>(Ab + (size_t)r * h + k));
                    else
                        av[r] = load8<T, W>(Ab + (size_t)min(r, R - 1 - g * 8) * h, k, h);  // (r_max not a multiple of 8)
                }
        }
        if (store) {
            uint32_t codes[2], words[2];
            quantise_rows<T, 2>(v, codes, words, lane);
            if (k / 32 < q.blocks) *reinterpret_cast<uint32_t*>(q.codes + (size_t)t * q.pitch + k / 2) = codes[0];
            if ((lane & 15) == 0 && k < width)
                *reinterpret_cast<uint32_t*>(q.scales + ((size_t)(t / 128) * q.ktiles + k / 128) * 512 + (t % 32) * 16 +
                                             (t % 128) / 32 * 4) = words[0];
        }
        if (rows && k < h) {
            float xf[8];
            unpack_raw(v[0], xf);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float af[8];
                unpack_raw(av[r], af);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[r] = fmaf(xf[i], af[i], acc[r]);
            }
        }
    }
    if (!lora) return;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float v = acc[r];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) red[warp][r] = v;
    }
    __syncthreads();
    if (threadIdx.x < 8 && g * 8 + threadIdx.x < R) {
        const int r = threadIdx.x;
        s_out[((size_t)ks * seg.n + t) * R + g * 8 + r] = e.scale * (red[0][r] + red[1][r] + red[2][r] + red[3][r]);
    }
}

template <typename T, int W>
static int launch_front_t(const PoolView& pv, const SegView& sv, const void* x, const Fp4View& q, float* s_out,
                          int s_parts, cudaStream_t st) {
    const T* xp = static_cast<const T*>(x);
    void* args[] = {(void*)&pv, (void*)&sv, (void*)&xp, (void*)&q, (void*)&s_out};
    LORA_CUDA_TRY(launch_pdl((const void*)fp4_front_kernel<T, W>, dim3(sv.n, (pv.R + 7) / 8, s_parts), dim3(128), 0, st, args));
    return LORA_OK;
}

// ---- after the product where the LoRA term is separate: y = product + s B^T, rounded once ---------
// One CTA per work item (up to 4 sorted tokens of one adapter) and 256 * fpt features, as the framework's
// segmented expand, but the product comes in float32 and y is written here alone; the CTAs behind the
// items' take the tokens without an adapter, four at a time.  Bound by latency: item, then s, B and the
// product's rows, which are in L2.
constexpr int kFp4ItemTok = 4;  // tokens of a work item
template <typename T>
__global__ void __launch_bounds__(256)
fp4_expand_kernel(PoolView pool, SegView seg, const float* __restrict__ s_in, int s_parts,
                  const float* __restrict__ y32, T* __restrict__ y, int fpt, int items, int rank_aware) {
    extern __shared__ float ss[];  // [4][R]: the item's shrink rows (K parts summed)
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, R = pool.R, h_out = pool.h_out;
    const int status = __ldcg(seg.status);  // (independent loads first)
    int slot = -1, nt, tok[kFp4ItemTok];
    if (b < items) {
        const int n_items = __ldcg(seg.nseg + 1);
        const int4 head = __ldcg(reinterpret_cast<const int4*>(seg.items + (size_t)b * 8));      // slot, count, tokens 0, 1
        const int2 tail = __ldcg(reinterpret_cast<const int2*>(seg.items + (size_t)b * 8 + 4));  // tokens 2, 3
        slot = head.x, nt = b < n_items ? head.y : 0;
        tok[0] = head.z, tok[1] = head.w, tok[2] = tail.x, tok[3] = tail.y;
    } else {  // the segment of no adapter is the first
        const int j0 = (b - items) * kFp4ItemTok;
        const int nseg = __ldcg(seg.nseg), first = __ldcg(seg.seg_slot), end = __ldcg(seg.seg_start + 1);
#pragma unroll
        for (int u = 0; u < kFp4ItemTok; ++u) tok[u] = __ldcg(seg.perm + min(j0 + u, seg.n - 1));
        nt = nseg > 0 && first < 0 ? min(kFp4ItemTok, end - j0) : 0;
    }
    if (status != LORA_OK || nt <= 0) return;
    const int o = blockIdx.y * 256 * fpt + threadIdx.x;
    const bool live[2] = {o < h_out, fpt == 2 && o + 256 < h_out};
    float acc[2][kFp4ItemTok];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int u = 0; u < kFp4ItemTok; ++u)
            acc[f][u] = live[f] && u < nt ? __ldcg(y32 + (size_t)tok[u] * h_out + o + 256 * f) : 0.f;
    if (slot >= 0) {
        for (int e = threadIdx.x; e < kFp4ItemTok * R; e += blockDim.x) {
            const int u = e / R, j = e - u * R, t = u == 0 ? tok[0] : u == 1 ? tok[1] : u == 2 ? tok[2] : tok[3];
            float v = 0.f;
            if (u < nt)
                for (int k = 0; k < s_parts; ++k) v += __ldcg(s_in + ((size_t)k * seg.n + t) * R + j);
            ss[e] = v;
        }
        __syncthreads();
        if (live[0]) {
            const T* Br = static_cast<const T*>(pool.B) + ((size_t)slot * h_out + o) * R;
            // columns past the adapter's true rank are zeros
            const int jmax = rank_aware ? min(R, (max(pool.table[slot].rank, 1) + 7) & ~7) : R;
            float term[2][kFp4ItemTok] = {};  // summed by itself: y32 may be far larger
            for (int j = 0; j < jmax; j += 8) {
                float b0[8], b1[8];
                unpack8<T>(__ldg(reinterpret_cast<const uint4*>(Br + j)), b0);
                unpack8<T>(live[1] ? __ldg(reinterpret_cast<const uint4*>(Br + (size_t)256 * R + j)) : make_uint4(0, 0, 0, 0), b1);
#pragma unroll
                for (int u = 0; u < kFp4ItemTok; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float sv = ss[u * R + j + e];
                        term[0][u] = fmaf(b0[e], sv, term[0][u]);
                        term[1][u] = fmaf(b1[e], sv, term[1][u]);
                    }
            }
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int u = 0; u < kFp4ItemTok; ++u) acc[f][u] += term[f][u];
        }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int u = 0; u < kFp4ItemTok; ++u)
            if (live[f] && u < nt) y[(size_t)tok[u] * h_out + o + 256 * f] = from_f32<T>(acc[f][u]);
}

template <typename T>
static int launch_fp4_expand_t(const PoolView& pv, const SegView& sv, const float* s_in, int s_parts, const float* y32,
                               void* y, cudaStream_t st) {
    // at most one item per LoRA token, and per segment one partial item beyond n / 4
    const int quads = (sv.n + kFp4ItemTok - 1) / kFp4ItemTok;
    int items = std::min(sv.n, std::min(sv.n, pv.S) + quads);
    // two features a thread where the grid keeps two CTAs an SM that way
    int fpt = (long long)items * ((pv.h_out + 511) / 512) >= 2LL * num_sms() ? 2 : 1;
    int rank_aware = has_padded_slots(pv);
    T* yp = static_cast<T*>(y);
    void* args[] = {(void*)&pv, (void*)&sv, (void*)&s_in, (void*)&s_parts, (void*)&y32, (void*)&yp, (void*)&fpt, (void*)&items, (void*)&rank_aware};
    const dim3 grid(items + quads, (pv.h_out + 256 * fpt - 1) / (256 * fpt));
    LORA_CUDA_TRY(launch_pdl((const void*)fp4_expand_kernel<T>, grid, dim3(256), sizeof(float) * kFp4ItemTok * pv.R, st, args));
    return LORA_OK;
}

// float32 pools: whether the per-token shrink (which reads an adapter's rows for each of its tokens) takes
// the batch, with the quantisation in the same launch, rather than the tiled one; and its K parts.  Both
// are weighed in us: the tiled one by its tiles' steps of 32 features (as many adapters as can be), and the
// launch that it adds, the per-token one by its sweeps of 1024 features.  Measured, us a linear, tiled / per
// token: 1 token 4096 x 4096 r_max 16 16.5 / 11.6; 64 tokens, 100 slots, r_max 8 31.5 / 16.6; 200 tokens,
// 6 slots, 11008 x 4096 r_max 64 110 / 84; 1000 tokens, 10 slots, 4096 x 1000 r_max 32 50.6 / 60.3; 15226
// tokens, 10 slots, 336 x 488 r_max 64 94 / 341; 4096 tokens, 100 slots, 4096 x 512 r_max 8 101 / 84.
static bool f32_front(const PoolView& pv, int n) {
    const int rows = pv.R <= 16 ? 16 : pv.R <= 32 ? 32 : 64;
    const double tiles = n / 64. + std::min(n, pv.S), groups = (pv.R + rows - 1) / rows, steps = (pv.h_in + 31) / 32;
    const double tiled = 4 + tiles * groups * steps * (rows == 16 ? 0.004 : rows == 32 ? 0.008 : 0.014);
    return (double)n * ((pv.R + 7) / 8) * ((pv.h_in + 1023) / 1024) * 0.0024 <= tiled;
}
static int f32_front_parts(const PoolView& pv, int n) {
    return std::max(1, std::min({(pv.h_in + 1023) / 1024, 4, 256 / std::max(n, 1)}));
}

int launch_fp4_front(const PoolView& pv, const SegView& sv, const void* x, const Fp4View* q, float* s_out, int* s_parts,
                     cudaStream_t st) {
    const Fp4View view = q ? *q : fp4_view(nullptr, nullptr, sv.n, pv.h_in);
    if (pv.dtype == LORA_F32) {
        *s_parts = f32_front_parts(pv, sv.n);
        return row_width(x, pv.h_in, 4) == 16 ? launch_front_t<float, 16>(pv, sv, x, view, s_out, *s_parts, st)
                                              : launch_front_t<float, 4>(pv, sv, x, view, s_out, *s_parts, st);
    }
    *s_parts = shrink_parts(pv, sv.n, false);
    if (pv.dtype == LORA_F16) return launch_front_t<__half, 16>(pv, sv, x, view, s_out, *s_parts, st);
    return launch_front_t<__nv_bfloat16, 16>(pv, sv, x, view, s_out, *s_parts, st);
}

static dim3 fp4_grid(const Fp4View& q) {
    return dim3(q.ktiles / 2, 4, (q.rows + 127) / 128);
}

template <typename T>
static int quantize_t(const void* x, long long ld, const Fp4View& q, cudaStream_t st) {
    const int w = row_width(x, ld, sizeof(T));
    const T* xp = static_cast<const T*>(x);
    void* args[] = {(void*)&xp, (void*)&ld, (void*)&q};
    const void* fn = w == 16  ? (const void*)fp4_quantize_kernel<T, 16>
                     : w == 4 ? (const void*)fp4_quantize_kernel<T, 4>
                              : (const void*)fp4_quantize_kernel<T, 2>;
    LORA_CUDA_TRY(launch_pdl(fn, fp4_grid(q), dim3(kFp4Threads), 0, st, args));
    return LORA_OK;
}

int launch_fp4_quantize(const void* x, int dtype, long long ld, const Fp4View& q, cudaStream_t st) {
    if (q.rows == 0) return LORA_OK;
    switch (dtype) {
        case LORA_F32: return quantize_t<float>(x, ld, q, st);
        case LORA_F16: return quantize_t<__half>(x, ld, q, st);
        default: return quantize_t<__nv_bfloat16>(x, ld, q, st);
    }
}

template <typename T>
static int dequantize_t(const Fp4View& q, void* out, long long ld, cudaStream_t st) {
    const int w = row_width(out, ld, sizeof(T));
    T* op = static_cast<T*>(out);
    void* args[] = {(void*)&q, (void*)&op, (void*)&ld};
    const void* fn = w == 16  ? (const void*)fp4_dequantize_kernel<T, 16>
                     : w == 4 ? (const void*)fp4_dequantize_kernel<T, 4>
                              : (const void*)fp4_dequantize_kernel<T, 2>;
    LORA_CUDA_TRY(launch_pdl(fn, fp4_grid(q), dim3(kFp4Threads), 0, st, args));
    return LORA_OK;
}

// early: as launch_fp4_decode's.
static int launch_fp4_product(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status,
                              int early, cudaStream_t st) {
    // The pair kernel also for batches whose split sums would not fit beside the receive buffer (more than
    // 224 tokens), unless K is long, and for wide outputs, where the decode kernel does not split K.
    // Measured, us a call, decode / pair: 256 tokens 4096 x 4096 14.6 / 11.6, 1024 x 1024 11.3 / 7.5,
    // 11008 x 4096 17.9 / 20.4, 4096 x 11008 14.4 / 12.1; 160 tokens 4096 x 4096 10.0 / 11.5; 96 tokens
    // 4096 x 4096 8.0 / 11.5, 11008 x 11008 27.8 / 21.2, 4096 x 32000 27.6 / 20.2.  Wide outputs of few tiles lose
    // by it up to 128 tokens (96 tokens 4096 x 11008 10.4 / 11.9, 1024 x 11008 5.1 / 8.0).
    const bool wide = (w.rows + 127) / 128 * 2 > num_sms();
    const bool pair = x.rows > 256 || (x.rows > 224 && x.cols <= 8192) || (x.rows > 64 && wide);
    return pair ? launch_fp4_pair(x, w, y, dtype, ldy, status, /*early_w=*/early >= 1, nullptr, st)
                : launch_fp4_decode(x, w, y, dtype, ldy, status, early, nullptr, st);
}

// grid.z counts 128-row tiles
constexpr int kFp4MaxRows = 65535 * 128;

static int check_shape(int rows, int cols) {
    if (rows < 0 || cols < 1) return set_error(LORA_EINVAL, "4-bit matrix of %d x %d", rows, cols);
    if (rows > kFp4MaxRows || cols > (1 << 30))
        return set_error(LORA_EUNSUP, "4-bit matrix of %d x %d is too large", rows, cols);
    return LORA_OK;
}

static int check_matrix(const lora_fp4_matrix* m, const char* what) {
    if (!m) return set_error(LORA_EINVAL, "%s is NULL", what);
    const int rc = check_shape(m->rows, m->cols);
    if (rc) return rc;
    if (m->rows == 0) return LORA_OK;
    if (!m->codes_dev || !m->scales_dev) return set_error(LORA_EINVAL, "%s has no codes or scales", what);
    if ((reinterpret_cast<uintptr_t>(m->codes_dev) | reinterpret_cast<uintptr_t>(m->scales_dev)) % 256)
        return set_error(LORA_EINVAL, "%s: codes and scales must be 256-byte aligned", what);
    return LORA_OK;
}

// A strided [rows, cols] array of dtype (what the 4-bit form is made from or read into).
static int check_rows(const void* p, int dtype, int64_t ld, int rows, int cols, const char* what) {
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return set_error(LORA_EINVAL, "bad dtype %d", dtype);
    if (ld < cols) return set_error(LORA_EINVAL, "%s: row stride %lld below %d columns", what, (long long)ld, cols);
    if (rows == 0) return LORA_OK;
    if (!p) return set_error(LORA_EINVAL, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % dtype_size(dtype)) return set_error(LORA_EINVAL, "%s is misaligned", what);
    return LORA_OK;
}

static Fp4View view_of(const lora_fp4_matrix* m) { return fp4_view(m->codes_dev, m->scales_dev, m->rows, m->cols); }

// Batches of more than 256 tokens whose tokens are spread over many adapters (fewer than 16 a slot) at
// ranks of up to 32: the product without the LoRA term, and a segmented expand after it.  The fused
// product then builds LoRA blocks for almost every adapter in every tile.  Measured, us a linear
// separate / fused, 4096 x 4096, 100 slots, r_max 16, every token its own adapter: 300 tokens 32.8 / 66.4,
// 600 39 / 84, 1200 60 / 92, 2400 93 / 87; a run of 512 tokens an adapter: 600 tokens 34 / 26, 1200 53 / 34.
// At r_max 64 the expand takes 69 / 32 where 600 tokens come in runs and 86 / 243 where they are spread, which the host cannot tell apart, and the fused product stays.  Slots count
// as adapters whether mounted or not, and more than 100 were not measured.
//
// From 32 to 256 tokens the same choice weighs, in us, the blocks that each of the decode kernel's CTAs
// would build if as many adapters as can be are there, against the expand and its launch.  Measured,
// fused / separate, Zipf-distributed adapters, 4096 -> 4096 and 4096 -> 11008 features: 64 tokens, 100 slots
// r_max 8 13.8 / 15.3 and 25.8 / 26.5, r_max 32 25.0 / 19.6 and 62 / 33; 128 tokens, 30 slots r_max 16
// 20.3 / 20.0 and 37.9 / 30.8; 250 tokens, 6 slots r_max 64 30.4 / 40.9 and 47 / 68, 100 slots r_max 64
// 88 / 55 and 249 / 97.  (16 tokens: fused throughout.)
//
// The product then goes to the workspace in float32 (4 n h_out bytes), so that y is rounded once: at most
// kFp4SumElements of it.
constexpr long long kFp4SumElements = 32 << 20;
static bool fp4_separate(const PoolView& pv, int n) {
    if (pv.dtype == LORA_F32 || (long long)n * pv.h_out > kFp4SumElements) return false;
    const int adapters = std::min(n, pv.S);
    if (n > 256) return pv.R <= 32 && n < 16LL * adapters;
    if (n < 32) return false;
    const double blocks = (double)adapters * pv.R / 32 / fp4_decode_splits(pv.h_out, pv.h_in);
    return blocks * (0.35 + 0.0025 * n) > 4 + (double)n * pv.R * pv.h_out / 6e6;
}

// The largest batch of more than 256 and at most n tokens for which that holds (0: none).
static int fp4_separate_most(const PoolView& pv, int n) {
    const int m = (int)std::min<long long>({(long long)n, 16LL * pv.S - 1, kFp4SumElements / pv.h_out});
    return m > 256 && fp4_separate(pv, m) ? m : 0;
}

static int f32_parts(const PoolView& pv, int n) { return f32_front(pv, n) ? f32_front_parts(pv, n) : f32_shrink_parts(pv, n); }

// Workspace of lora_fp4_linear_fwd: the shrink output (in K parts, and for large batches their sum), the
// product where the expand is separate, then the stored form of x.
struct Fp4WsLayout {
    size_t sum_off, y32_off, codes_off, scales_off, total;
};
static int fp4_ws_layout(lora_pool_t pool, int n, Fp4WsLayout* L) {
    size_t s_bytes;
    const int rc = lora_linear_workspace_bytes(pool, n, &s_bytes);
    if (rc) return rc;
    const int h_in = pool->desc.h_in;
    size_t sum_bytes = 0, y32_bytes = 0;
    const PoolView pv = pool_view(pool);
    if (fp4_separate(pv, n)) {
        y32_bytes = (size_t)n * pv.h_out * 4;
    } else if (n > 256 && pv.dtype != LORA_F32) {
        const int parts = fp4_prepare_parts(n, fp4_view(nullptr, nullptr, n, h_in).ktiles);
        sum_bytes = (size_t)n * pool->desc.r_max * 4;
        s_bytes = parts > 1 ? (size_t)parts * sum_bytes : 0;
    }
    if (pool->desc.dtype == LORA_F32)
        s_bytes = (size_t)f32_parts(pv, n) * std::max(n, 1) * pool->desc.r_max * 4;
    L->sum_off = align256(s_bytes);
    L->y32_off = L->sum_off + align256(sum_bytes);
    L->codes_off = L->y32_off + align256(y32_bytes);
    L->scales_off = L->codes_off + align256(fp4_codes_bytes(n, h_in));
    L->total = L->scales_off + align256(fp4_scales_bytes(n, h_in));
    return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" {

int lora_fp4_bytes(int rows, int cols, size_t* codes_bytes, size_t* scales_bytes) {
    if (!codes_bytes || !scales_bytes) return set_error(LORA_EINVAL, "codes_bytes/scales_bytes is NULL");
    const int rc = check_shape(rows, cols);
    if (rc) return rc;
    *codes_bytes = fp4_codes_bytes(rows, cols);
    *scales_bytes = fp4_scales_bytes(rows, cols);
    return LORA_OK;
}

int lora_fp4_quantize(const void* x_dev, int dtype, int64_t ld, const lora_fp4_matrix* out, void* stream) {
    int rc = check_matrix(out, "out");
    if (rc) return rc;
    rc = check_rows(x_dev, dtype, ld, out->rows, out->cols, "x");
    if (rc) return rc;
    return launch_fp4_quantize(x_dev, dtype, ld, view_of(out), static_cast<cudaStream_t>(stream));
}

int lora_fp4_dequantize(const lora_fp4_matrix* q, void* out_dev, int dtype, int64_t ld, void* stream) {
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

int lora_fp4_matmul(const lora_fp4_matrix* x, const lora_fp4_matrix* w, void* y_dev, int dtype, int64_t ldy,
                    void* stream) {
    int rc = check_matrix(x, "x");
    if (!rc) rc = check_matrix(w, "w");
    if (rc) return rc;
    if (x->cols != w->cols) return set_error(LORA_EINVAL, "x has %d columns, w %d", x->cols, w->cols);
    rc = check_rows(y_dev, dtype, ldy, w->rows ? x->rows : 0, w->rows, "y");
    if (rc || x->rows == 0 || w->rows == 0) return rc;
    return launch_fp4_product(view_of(x), view_of(w), y_dev, dtype, ldy, nullptr, /*early=*/0,
                              static_cast<cudaStream_t>(stream));
}

int lora_fp4_linear_workspace_bytes(lora_pool_t pool, int n_tokens, size_t* bytes) {
    if (!pool || !bytes) return set_error(LORA_EINVAL, "pool/bytes is NULL");
    Fp4WsLayout L;
    int rc = fp4_ws_layout(pool, n_tokens, &L);
    if (rc) return rc;
    *bytes = L.total;
    // Smaller batches may need more: they split K into more parts.  From 256 tokens on the need grows within
    // each 64 (the paths before and after a change of path too: the one for more tokens needs no less), and
    // there is one part from 64 tokens for each of 4 CTAs an SM on.  The separate expand's largest batch is
    // looked up by itself.
    const int last = std::min(n_tokens, 64 * 4 * num_sms() + 128);
    for (int m = 1; m < last; m += m < 256 ? 1 : 64) {
        rc = fp4_ws_layout(pool, m, &L);
        if (rc) return rc;
        *bytes = std::max(*bytes, L.total);
    }
    const int separate = fp4_separate_most(pool_view(pool), n_tokens);
    if (separate) {
        rc = fp4_ws_layout(pool, separate, &L);
        if (rc) return rc;
        *bytes = std::max(*bytes, L.total);
    }
    return LORA_OK;
}

int lora_fp4_linear_fwd(lora_pool_t pool, const lora_fp4_matrix* w, const void* x_dev, const lora_fp4_matrix* xq,
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
    // the fused decode kernel's boxes of B have 32-bit coordinates (slot * h_out + feature)
    if (pv.dtype != LORA_F32 && n <= 256 && !fp4_separate(pv, n) && (long long)pv.S * pv.h_out > INT_MAX)
        return set_error(LORA_EUNSUP, "4-bit linear of %d tokens over %d slots x %d features", n, pv.S, pv.h_out);
    Fp4WsLayout L;
    rc = fp4_ws_layout(pool, n, &L);
    if (rc) return rc;
    if (ws_bytes < L.total)
        return set_error(LORA_ENOSPACE, "4-bit linear workspace needs %zu bytes, got %zu", L.total, ws_bytes);
    char* ws = static_cast<char*>(ws_dev);
    float* s_buf = reinterpret_cast<float*>(ws);
    const Fp4View q = xq ? view_of(xq) : fp4_view(ws + L.codes_off, ws + L.scales_off, n, pv.h_in);
    const SegView sv = seg_view(seg);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);

    if (fp4_separate(pv, n)) {
        int s_parts = 1;
        if (!xq) rc = launch_fp4_quantize(x_dev, pv.dtype, pv.h_in, q, st);
        if (!rc) rc = launch_shrink(pv, sv, x_dev, s_buf, st, /*tiled=*/false, &s_parts);
        float* y32 = reinterpret_cast<float*>(ws + L.y32_off);
        if (!rc) rc = launch_fp4_product(q, view_of(w), y32, LORA_F32, pv.h_out, sv.status, /*early=*/2, st);
        if (rc) return rc;
        return pv.dtype == LORA_F16 ? launch_fp4_expand_t<__half>(pv, sv, s_buf, s_parts, y32, y_dev, st)
                                    : launch_fp4_expand_t<__nv_bfloat16>(pv, sv, s_buf, s_parts, y32, y_dev, st);
    }
    if (n > 256 && pv.dtype != LORA_F32) {
        float* sum = reinterpret_cast<float*>(ws + L.sum_off);
        const Fp4View own = fp4_view(ws + L.codes_off, ws + L.scales_off, n, pv.h_in);
        rc = launch_fp4_prepare(pv, sv, x_dev, xq ? &q : nullptr, own, s_buf, sum, st);
        if (rc) return rc;
        const Fp4Lora lora = {sv.perm, sv.idx, sum, pv.B, pv.R};
        return launch_fp4_pair(own, view_of(w), y_dev, pv.dtype, pv.h_out, sv.status, /*early_w=*/true, &lora, st);
    }
    int s_parts = 1;
    if (pv.dtype != LORA_F32) {
        // One kernel quantises x and computes the per-token shrink; the product behind it streams its
        // weight meanwhile.  Where the shrink reads each adapter once per 4 tokens instead (many rows of
        // A), x is quantised first and the product's main loop overlaps the shrink.
        int early = 1;
        if (shrink_segmented(pv, n)) {
            if (!xq) rc = launch_fp4_quantize(x_dev, pv.dtype, pv.h_in, q, st);
            if (!rc) rc = launch_shrink(pv, sv, x_dev, s_buf, st, /*tiled=*/false, &s_parts);
            early = 2;
        } else {
            rc = launch_fp4_front(pv, sv, x_dev, xq ? nullptr : &q, s_buf, &s_parts, st);
            if (xq) early = 2;
        }
        if (rc) return rc;
        const Fp4DecodeLora lora = {&pv, sv.idx, s_buf, s_parts};
        return launch_fp4_decode(q, view_of(w), y_dev, pv.dtype, pv.h_out, sv.status, early, &lora, st);
    }
    // float32 pools: the LoRA term in float32, around the product
    int early = 2;
    if (f32_front(pv, n)) {
        rc = launch_fp4_front(pv, sv, x_dev, xq ? nullptr : &q, s_buf, &s_parts, st);
        if (!xq) early = 1;  // the kernel just launched stores x
    } else {
        s_parts = f32_shrink_parts(pv, n);
        if (!xq) rc = launch_fp4_quantize(x_dev, pv.dtype, pv.h_in, q, st);
        if (!rc) rc = launch_f32_shrink(pv, sv, x_dev, s_buf, st);
    }
    if (rc) return rc;
    rc = launch_fp4_product(q, view_of(w), y_dev, pv.dtype, pv.h_out, sv.status, early, st);
    if (rc) return rc;
    return launch_f32_expand(pv, sv, s_buf, s_parts, y_dev, st);
}

}  // extern "C"
