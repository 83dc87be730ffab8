// Products of a few tokens over an 8-bit weight, with the LoRA term.
//
// y[t, o] = sx[t] sw[o] sum_k cx[t, k] cw[o, k] (+ s[t, :] . B_slot(t)[o, :]): the sum in 32-bit integers by
// four-way dot products, so it is exact in any order.  The weight streams through once per group of NT
// tokens; a warp takes RW of its rows, 16 bytes a lane, and its lanes' sums meet in one reduction.  Bound by memory
// and latency: 4096 x 4096 float16 5.3 us with one token (its bytes 2.5), 6.9 with 8; to 11008 features 17.2 with 8.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "i8_device.cuh"
#include "kernels.h"

namespace lora {

constexpr int kSmallThreads = 256;

struct SmallArgs {
    I8View x, w;
    void* y;
    long long ldy;
    const int32_t* status;  // nullable
    int early_w;
    // the LoRA term (FUSE)
    const SlotEntry* table;
    const void* B;
    const int32_t* idx;
    const float* s_in;
    int R, s_parts;
};

// FUSE: with the LoRA term.  Bound by latency: every warp has its first pieces of the weight in flight before it
// waits for the kernel ahead (early_w), and the LoRA term's B rows while the shrink output is added up.
template <typename T, int NT, int RW, bool FUSE>
__global__ void __launch_bounds__(kSmallThreads)
i8_small_kernel(const SmallArgs a) {
    constexpr int kSmallAhead = NT <= 2 ? 4 : 2;  // pieces of 512 codes whose loads are in flight together
    extern __shared__ float s_sm[];  // FUSE: [NT][R] shrink output, zeros past the adapter's rank
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int o0 = (blockIdx.x * (kSmallThreads / 32) + warp) * RW, t0 = blockIdx.y * NT;
    const int n = a.x.rows, h_out = a.w.rows, pitch = (int)a.w.pitch;
    int4 wv[kSmallAhead][RW];
    auto load_w = [&](int k, int4 (&v)[RW]) {
#pragma unroll
        for (int i = 0; i < RW; ++i)
            if (k < pitch && o0 < h_out)
                v[i] = __ldcs(reinterpret_cast<const int4*>(a.w.codes + (size_t)min(o0 + i, h_out - 1) * pitch + k));
            else
                v[i] = make_int4(0, 0, 0, 0);
    };
    if (!a.early_w) pdl_wait();
#pragma unroll
    for (int h = 0; h < kSmallAhead; ++h) load_w(lane * 16 + h * 512, wv[h]);
    if (a.early_w) {
        pdl_trigger();
        pdl_wait();
    }
    const int status = a.status ? __ldcg(a.status) : LORA_OK;
    // this lane's output, and its adapter's rows
    const int o = o0 + lane % RW, t = t0 + lane / RW;
    const bool mine = lane < RW * NT && o < h_out && t < n;
    const float sw = mine ? __ldg(a.w.scales + o) : 0.f, sx = mine ? __ldcg(a.x.scales + t) : 0.f;
    int slot = -1, rank = 0;
    const T* b = nullptr;
    float bf[8];
    if constexpr (FUSE) {
        if (mine) slot = __ldcg(a.idx + t);
        if (status != LORA_OK) return;
        if (slot >= 0) {
            rank = a.table[slot].rank;
            b = static_cast<const T*>(a.B) + ((size_t)slot * h_out + o) * a.R;
            load_b8<T>(b, 0, a.R, bf);
        }
        const size_t part = (size_t)n * a.R;
        for (int e = threadIdx.x; e < NT * a.R; e += kSmallThreads) {
            const int u = t0 + e / a.R, j = e % a.R, us = u < n ? __ldcg(a.idx + u) : -1;
            float v = 0.f;
            if (us >= 0 && j < a.table[us].rank)
                for (int p = 0; p < a.s_parts; ++p) v += __ldcg(a.s_in + p * part + (size_t)u * a.R + j);
            s_sm[e] = v;
        }
    } else {
        if (status != LORA_OK) return;
    }
    int acc[RW][NT] = {};
    for (int k0 = lane * 16; k0 < pitch; k0 += 512 * kSmallAhead) {
#pragma unroll
        for (int h = 0; h < kSmallAhead; ++h) {
            const int k = k0 + h * 512;
            if (k >= pitch) break;
            int4 xv[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                xv[j] = __ldcg(reinterpret_cast<const int4*>(a.x.codes + (size_t)min(t0 + j, n - 1) * pitch + k));
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[i][j] = __dp4a(wv[h][i].x, xv[j].x, acc[i][j]);
                    acc[i][j] = __dp4a(wv[h][i].y, xv[j].y, acc[i][j]);
                    acc[i][j] = __dp4a(wv[h][i].z, xv[j].z, acc[i][j]);
                    acc[i][j] = __dp4a(wv[h][i].w, xv[j].w, acc[i][j]);
                }
            load_w(k + 512 * kSmallAhead, wv[h]);
        }
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int v = __reduce_add_sync(0xffffffffu, acc[i][j]);
            if (lane == j * RW + i) sum = v;
        }
    float v = i8_scaled(sum, sx, sw);
    if constexpr (FUSE) {
        __syncthreads();
        if (slot >= 0) {
            const float* s = s_sm + (lane / RW) * a.R;
            float l = 0.f;
            for (int j = 0; j < rank; j += 8) {
                if (j > 0) load_b8<T>(b, j, a.R, bf);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j + e < rank) l = fmaf(bf[e], s[j + e], l);
            }
            v += l;
        }
    }
    if (mine) static_cast<T*>(a.y)[(long long)t * a.ldy + o] = from_f32<T>(v);
}

template <typename T, bool FUSE>
static int launch_small_t(const SmallArgs& a, cudaStream_t st) {
    const int n = a.x.rows, rw = n <= 2 ? 2 : 4, nt = n == 1 ? 1 : n == 2 ? 2 : n <= 4 ? 4 : 8;
    const void* fn = nt == 1   ? (const void*)i8_small_kernel<T, 1, 2, FUSE>
                     : nt == 2 ? (const void*)i8_small_kernel<T, 2, 2, FUSE>
                     : nt == 4 ? (const void*)i8_small_kernel<T, 4, 4, FUSE>
                               : (const void*)i8_small_kernel<T, 8, 4, FUSE>;
    const int rows = kSmallThreads / 32 * rw;
    const dim3 grid((a.w.rows + rows - 1) / rows, (n + nt - 1) / nt);
    void* args[] = {(void*)&a};
    LORA_CUDA_TRY(launch_pdl(fn, grid, dim3(kSmallThreads), FUSE ? (size_t)nt * a.R * 4 : 0, st, args));
    return LORA_OK;
}

int launch_i8_small(const I8View& x, const I8View& w, void* y, int dtype, long long ldy, int32_t* status, bool early_w,
                    const I8Lora* lora, cudaStream_t st) {
    SmallArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.w = w;
    a.y = y;
    a.ldy = ldy;
    a.status = status;
    a.early_w = early_w;
    if (lora) {
        a.B = lora->pool->B;
        a.idx = lora->idx;
        a.s_in = lora->s_in;
        a.R = lora->pool->R;
        a.table = lora->pool->table;
        a.s_parts = lora->s_parts;
    }
    switch (dtype) {
        case LORA_F32: return lora ? launch_small_t<float, true>(a, st) : launch_small_t<float, false>(a, st);
        case LORA_F16: return lora ? launch_small_t<__half, true>(a, st) : launch_small_t<__half, false>(a, st);
        default: return lora ? launch_small_t<__nv_bfloat16, true>(a, st) : launch_small_t<__nv_bfloat16, false>(a, st);
    }
}

}  // namespace lora
