// float32 pools over a 4-bit base: the LoRA term in float32 on CUDA cores, around the 4-bit product.  (The
// tensor cores have no float32 product; one from operands split into 16-bit parts was not tried.)
//
// Both kernels are register-tiled products over tiles of up to 64 tokens of one segment (tokens that
// share an adapter), so an adapter's rows are read once per 64 of its tokens:
//   shrink  s[t, j] = (alpha / r) sum_k x[t, k] A[j, k]     64 tokens x 16, 32 or 64 rows, part of K
//   expand  y[t, o] += sum_j s[t, j] B[o, j]                64 tokens x 64 features
// 256 threads; a thread keeps 4 tokens x 4 columns.  Operands pass through shared memory 32 deep, k-major,
// so that a step of k is two 16-byte reads for 16 multiply-adds; the next 32 are on their way meanwhile.
// Bound by the multiply-adds at r_max 64, by the reads of x and y below.  (1000 tokens, 4096 x 1000, r_max 32:
// 51 us a linear, against 31 with a 16-bit pool on the tensor cores.)  Where segments hold few tokens, the
// expand gives a thread one feature of up to 8 tokens instead, and the shrink goes token by token,
// together with the quantisation (fp4_front_kernel).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace lora {

constexpr int kFTok = 64;   // tokens per tile
constexpr int kFK = 32;     // depth of a step
constexpr int kFPad = 4;    // keeps rows of the k-major tiles 16-byte aligned and off one another's banks

// The tile blockIdx.x of up to TOK sorted tokens of one adapter segment: its slot (-1: none), first
// sorted position and count.
struct SegTile {
    int slot, j0, cnt;
};
template <int TOK = kFTok>
__device__ __forceinline__ SegTile find_tile(const SegView& seg, SegTile* sh) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, nseg = __ldcg(seg.nseg);
        int run = 0;
        SegTile t{-1, 0, 0};
        for (int base = 0; base < nseg; base += 32) {
            const int i = base + lane;
            int slot = -1, beg = 0, end = 0, tiles = 0;
            if (i < nseg) {
                slot = __ldcg(seg.seg_slot + i);
                beg = __ldcg(seg.seg_start + i);
                end = __ldcg(seg.seg_start + i + 1);
                if (slot >= 0) tiles = (end - beg + TOK - 1) / TOK;
            }
            int v = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += u;
            }
            const int first = run + v - tiles, want = (int)blockIdx.x;
            if (want >= first && want < first + tiles) {
                const int j0 = beg + (want - first) * TOK;
                *sh = SegTile{slot, j0, min(TOK, end - j0)};
            }
            run += __shfl_sync(0xffffffffu, v, 31);
            if (want < run) break;
        }
        if ((int)blockIdx.x >= run && lane == 0) *sh = t;
    }
    __syncthreads();
    return *sh;
}

// Four consecutive floats of a row from column c (zeros past cols).
__device__ __forceinline__ float4 load4(const float* row, int c, int cols, bool vec) {
    if (vec && c + 4 <= cols) return __ldcg(reinterpret_cast<const float4*>(row + c));
    float4 v;
    v.x = c < cols ? __ldcg(row + c) : 0.f;
    v.y = c + 1 < cols ? __ldcg(row + c + 1) : 0.f;
    v.z = c + 2 < cols ? __ldcg(row + c + 2) : 0.f;
    v.w = c + 3 < cols ? __ldcg(row + c + 3) : 0.f;
    return v;
}

// RT adapter rows per CTA.  A thread keeps 4 tokens x 4 rows; with fewer than 64 rows the threads form
// 64 / RT groups that take every so-manieth k and are added up at the end.
template <int RT>
__global__ void __launch_bounds__(256)
f32_shrink_kernel(PoolView pool, SegView seg, const float* __restrict__ x, float* __restrict__ s_out, int vec, int steps) {
    constexpr int G = 64 / RT, TX = RT / 4;
    __shared__ float xs[kFK][kFTok + kFPad];
    __shared__ float as[kFK][RT + kFPad];
    __shared__ float red[G > 1 ? G - 1 : 1][kFTok * RT];
    __shared__ SegTile sh;
    __shared__ int tok[kFTok];
    pdl_wait();
    pdl_trigger();
    if (__ldcg(seg.status) != LORA_OK) return;
    const SegTile tile = find_tile(seg, &sh);
    if (tile.slot < 0) return;
    const int tid = threadIdx.x, grp = tid / (16 * TX), in = tid % (16 * TX), ty = in / TX, tx = in % TX;
    if (tid < kFTok) tok[tid] = tid < tile.cnt ? __ldcg(seg.perm + tile.j0 + tid) : -1;
    __syncthreads();
    const int h = pool.h_in, R = pool.R, r0 = blockIdx.y * RT;
    const int k_beg = blockIdx.z * steps * kFK, k_end = min(h, k_beg + steps * kFK);
    const float* A = static_cast<const float*>(pool.A) + ((size_t)tile.slot * R + r0) * h;
    // loads: thread -> row tid / 8 (and the rows 32 further), columns 4 (tid % 8) of a step
    const int lr = tid >> 3, lc = (tid & 7) * 4;
    constexpr int AR = (RT + 31) / 32;
    float4 xv[2], av[AR];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tok[lr + 32 * i];
            xv[i] = t >= 0 ? load4(x + (size_t)t * h, k0 + lc, k_end, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < AR; ++i) {
            const int r = lr + 32 * i;
            av[i] = r < RT && r0 + r < R ? load4(A + (size_t)r * h, k0 + lc, k_end, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    float acc[4][4] = {};
    load(k_beg);
    for (int k0 = k_beg; k0 < k_end; k0 += kFK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            xs[lc][lr + 32 * i] = xv[i].x, xs[lc + 1][lr + 32 * i] = xv[i].y;
            xs[lc + 2][lr + 32 * i] = xv[i].z, xs[lc + 3][lr + 32 * i] = xv[i].w;
        }
#pragma unroll
        for (int i = 0; i < AR; ++i) {
            const int r = lr + 32 * i;
            if (r < RT) as[lc][r] = av[i].x, as[lc + 1][r] = av[i].y, as[lc + 2][r] = av[i].z, as[lc + 3][r] = av[i].w;
        }
        __syncthreads();
        if (k0 + kFK < k_end) load(k0 + kFK);
#pragma unroll 8
        for (int kk = 0; kk < kFK / G; ++kk) {
            const float4 xq = *reinterpret_cast<const float4*>(&xs[kk * G + grp][ty * 4]);
            const float4 aq = *reinterpret_cast<const float4*>(&as[kk * G + grp][tx * 4]);
            const float x4[4] = {xq.x, xq.y, xq.z, xq.w}, a4[4] = {aq.x, aq.y, aq.z, aq.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x4[i], a4[j], acc[i][j]);
        }
    }
    if (G > 1) {
        if (grp > 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) red[grp - 1][e * 16 * TX + in] = acc[e / 4][e % 4];
        __syncthreads();
        if (grp > 0) return;
#pragma unroll
        for (int g = 1; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e / 4][e % 4] += red[g - 1][e * 16 * TX + in];
    }
    const float scale = pool.table[tile.slot].scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = tok[ty * 4 + i];
        if (t < 0) continue;
        float* out = s_out + ((size_t)blockIdx.z * seg.n + t) * R + r0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + tx * 4 + j < R) out[tx * 4 + j] = scale * acc[i][j];
    }
}

// A CTA keeps its tokens' s in shared memory and goes over every gridDim.y-th tile of 64 features: finding
// its tokens takes five dependent loads, as long as the product of one feature tile.  (6122 tokens, 2992
// features, r_max 24, a CTA per feature tile: 93 us, this way 54.)  B of the next step and y of the next
// feature tile are on their way while a step is multiplied.
__global__ void __launch_bounds__(256)
f32_expand_kernel(PoolView pool, SegView seg, const float* __restrict__ s_in, int s_parts, float* __restrict__ y, int vec,
                  int vec_y) {
    extern __shared__ float4 ss_raw[];
    float(*ss)[kFTok + kFPad] = reinterpret_cast<float(*)[kFTok + kFPad]>(ss_raw);  // [r_max rounded up to kFK]
    __shared__ float bs[kFK][64 + kFPad];
    __shared__ SegTile sh;
    __shared__ int tok[kFTok];
    pdl_wait();
    pdl_trigger();
    if (__ldcg(seg.status) != LORA_OK) return;
    const SegTile tile = find_tile(seg, &sh);
    if (tile.slot < 0) return;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    if (tid < kFTok) tok[tid] = tid < tile.cnt ? __ldcg(seg.perm + tile.j0 + tid) : -1;
    __syncthreads();
    const int h_out = pool.h_out, R = pool.R, step_o = gridDim.y * 64;
    const float* B = static_cast<const float*>(pool.B) + (size_t)tile.slot * h_out * R;
    const int lr = tid >> 3, lc = (tid & 7) * 4;
    float4 bv[2], yv[4];
    auto load_b = [&](int o0, int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = o0 + lr + 32 * i;
            bv[i] = o < h_out ? load4(B + (size_t)o * R, k0 + lc, R, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto load_y = [&](int o0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tok[ty * 4 + i];
            yv[i] = t >= 0 ? load4(y + (size_t)t * h_out, o0 + tx * 4, h_out, vec_y) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    int o0 = blockIdx.y * 64;
    load_b(o0, 0);
    load_y(o0);
    for (int k0 = 0; k0 < R; k0 += kFK) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lr + 32 * i, t = tok[r];
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t >= 0)
                for (int p0 = 0; p0 < s_parts; p0 += 4) {  // four parts' loads in flight
                    float4 u[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        u[p] = load4(s_in + ((size_t)min(p0 + p, s_parts - 1) * seg.n + t) * R, k0 + lc, R, vec);
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (p0 + p < s_parts) v.x += u[p].x, v.y += u[p].y, v.z += u[p].z, v.w += u[p].w;
                }
            ss[k0 + lc][r] = v.x, ss[k0 + lc + 1][r] = v.y, ss[k0 + lc + 2][r] = v.z, ss[k0 + lc + 3][r] = v.w;
        }
    }
    for (; o0 < h_out; o0 += step_o) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < R; k0 += kFK) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lr + 32 * i;
                bs[lc][r] = bv[i].x, bs[lc + 1][r] = bv[i].y, bs[lc + 2][r] = bv[i].z, bs[lc + 3][r] = bv[i].w;
            }
            __syncthreads();
            if (k0 + kFK < R)
                load_b(o0, k0 + kFK);
            else if (o0 + step_o < h_out)
                load_b(o0 + step_o, 0);
            const int depth = min(kFK, R - k0);
            for (int kk = 0; kk < depth; ++kk) {
                const float4 sq = *reinterpret_cast<const float4*>(&ss[k0 + kk][ty * 4]);
                const float4 bq = *reinterpret_cast<const float4*>(&bs[kk][tx * 4]);
                const float s4[4] = {sq.x, sq.y, sq.z, sq.w}, b4[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s4[i], b4[j], acc[i][j]);
            }
        }
        const int o = o0 + tx * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tok[ty * 4 + i];
            if (t < 0) continue;
            float* yr = y + (size_t)t * h_out + o;
            const float v[4] = {yv[i].x + acc[i][0], yv[i].y + acc[i][1], yv[i].z + acc[i][2], yv[i].w + acc[i][3]};
            if (vec_y && o + 4 <= h_out) {
                *reinterpret_cast<float4*>(yr) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (o + j < h_out) yr[j] = v[j];
            }
        }
        if (o0 + step_o < h_out) load_y(o0 + step_o);
    }
}

constexpr int kFSmallTok = 8;
__global__ void __launch_bounds__(128)
f32_expand_small_kernel(PoolView pool, SegView seg, const float* __restrict__ s_in, int s_parts, float* __restrict__ y,
                        int vec) {
    __shared__ __align__(16) float ss[kFSmallTok][kMaxRank];
    __shared__ SegTile sh;
    pdl_wait();
    pdl_trigger();
    if (__ldcg(seg.status) != LORA_OK) return;
    const SegTile tile = find_tile<kFSmallTok>(seg, &sh);
    if (tile.slot < 0) return;
    const int h_out = pool.h_out, R = pool.R, o = blockIdx.y * 128 + threadIdx.x;
    int tok[kFSmallTok];
    float yv[kFSmallTok], acc[kFSmallTok];
#pragma unroll
    for (int i = 0; i < kFSmallTok; ++i) tok[i] = i < tile.cnt ? __ldcg(seg.perm + tile.j0 + i) : -1;
#pragma unroll
    for (int i = 0; i < kFSmallTok; ++i) {
        yv[i] = tok[i] >= 0 && o < h_out ? __ldcg(y + (size_t)tok[i] * h_out + o) : 0.f;
        acc[i] = 0.f;
    }
    for (int e = threadIdx.x; e < tile.cnt * R; e += 128) {
        const int i = e / R, j = e - i * R, t = __ldcg(seg.perm + tile.j0 + i);
        float v = 0.f;
        for (int p0 = 0; p0 < s_parts; p0 += 8) {
            float u[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) u[p] = __ldcg(s_in + ((size_t)min(p0 + p, s_parts - 1) * seg.n + t) * R + j);
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p0 + p < s_parts) v += u[p];
        }
        ss[i][j] = v;
    }
    __syncthreads();
    if (o >= h_out) return;
    const float* Br = static_cast<const float*>(pool.B) + ((size_t)tile.slot * h_out + o) * R;
    for (int j = 0; j < R; j += 4) {
        const float4 b = load4(Br, j, R, vec);
#pragma unroll
        for (int i = 0; i < kFSmallTok; ++i) {
            if (i >= tile.cnt) break;
            acc[i] = fmaf(b.x, ss[i][j], acc[i]);
            if (j + 1 < R) acc[i] = fmaf(b.y, ss[i][j + 1], acc[i]);
            if (j + 2 < R) acc[i] = fmaf(b.z, ss[i][j + 2], acc[i]);
            if (j + 3 < R) acc[i] = fmaf(b.w, ss[i][j + 3], acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kFSmallTok; ++i)
        if (tok[i] >= 0) y[(size_t)tok[i] * h_out + o] = yv[i] + acc[i];
}

static int f32_tiles(const PoolView& pv, int n) { return (n + kFTok - 1) / kFTok + std::min(n, pv.S); }

// K parts of the shrink (the expand adds them up): four CTAs an SM where K allows parts of at least 3
// steps.  Measured, us a linear with two CTAs an SM and 8 steps / this way: 98 tokens, 312 x 96, r_max 24
// 24.7 / 19.2; 3218 tokens, 10056 x 368, r_max 16 183 / 118; 16384 tokens, 4096 x 4096, r_max 16 520 / 411.
int f32_shrink_parts(const PoolView& pv, int n) {
    const int rows = pv.R <= 16 ? 16 : pv.R <= 32 ? 32 : 64;
    const int ctas = std::max(1, (n + kFTok - 1) / kFTok * ((pv.R + rows - 1) / rows));
    const int steps = (pv.h_in + kFK - 1) / kFK;
    int parts = std::max(1, std::min({4 * num_sms() / ctas, 24, steps / 3}));
    const int per = (steps + parts - 1) / parts;
    return (steps + per - 1) / per;
}

int launch_f32_shrink(const PoolView& pv, const SegView& sv, const void* x, float* s_out, cudaStream_t st) {
    const float* xp = static_cast<const float*>(x);
    // 16-byte loads where rows of x and A start on 16-byte boundaries
    int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && pv.h_in % 4 == 0;
    const int parts = f32_shrink_parts(pv, sv.n), all = (pv.h_in + kFK - 1) / kFK;
    int steps = (all + parts - 1) / parts;
    void* args[] = {(void*)&pv, (void*)&sv, (void*)&xp, (void*)&s_out, (void*)&vec, (void*)&steps};
    const int rows = pv.R <= 16 ? 16 : pv.R <= 32 ? 32 : 64;
    const void* fn = rows == 16   ? (const void*)f32_shrink_kernel<16>
                     : rows == 32 ? (const void*)f32_shrink_kernel<32>
                                  : (const void*)f32_shrink_kernel<64>;
    const dim3 grid(f32_tiles(pv, sv.n), (pv.R + rows - 1) / rows, parts);
    LORA_CUDA_TRY(launch_pdl(fn, grid, dim3(256), 0, st, args));
    return LORA_OK;
}

int launch_f32_expand(const PoolView& pv, const SegView& sv, const float* s_in, int s_parts, void* y, cudaStream_t st) {
    float* yp = static_cast<float*>(y);
    int vec = pv.R % 4 == 0;
    void* args[] = {(void*)&pv, (void*)&sv, (void*)&s_in, (void*)&s_parts, (void*)&yp, (void*)&vec};
    // up to 8 tokens a slot (64 tokens over 100 slots, r_max 8, 4096 features: 76 -> 35 us a linear); with
    // more the tiled kernel reads B less often (200 tokens over 6 slots, r_max 64: 158 -> 132 us)
    if (sv.n <= 8 * std::min(sv.n, pv.S)) {
        const dim3 small((sv.n + kFSmallTok - 1) / kFSmallTok + std::min(sv.n, pv.S), (pv.h_out + 127) / 128);
        if (small.y > 65535) return set_error(LORA_EUNSUP, "float32 expand of %d features", pv.h_out);
        LORA_CUDA_TRY(launch_pdl((const void*)f32_expand_small_kernel, small, dim3(128), 0, st, args));
        return LORA_OK;
    }
    // feature tiles are spread over as many CTAs as make about four an SM
    const int tiles = (sv.n + kFTok - 1) / kFTok, features = (pv.h_out + 63) / 64;
    const dim3 grid(f32_tiles(pv, sv.n), std::min(features, (4 * num_sms() + tiles - 1) / tiles));
    const size_t smem = (size_t)(pv.R + kFK - 1) / kFK * kFK * (kFTok + kFPad) * 4;
    static bool attr = false;
    if (!attr) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(f32_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMaxRank * (kFTok + kFPad) * 4));
        attr = true;
    }
    int vec_y = reinterpret_cast<uintptr_t>(y) % 16 == 0 && pv.h_out % 4 == 0;
    void* targs[] = {(void*)&pv, (void*)&sv, (void*)&s_in, (void*)&s_parts, (void*)&yp, (void*)&vec, (void*)&vec_y};
    LORA_CUDA_TRY(launch_pdl((const void*)f32_expand_kernel, grid, dim3(256), smem, st, targs));
    return LORA_OK;
}

}  // namespace lora
