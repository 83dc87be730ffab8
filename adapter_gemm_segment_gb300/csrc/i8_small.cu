// Products of a few tokens over an 8-bit weight, with the LoRA term.
//
// y[t, o] = sx[t] sw[o] sum_k cx[t, k] cw[o, k] (+ s[t, :] . B_slot(t)[o, :]): the sum in 32-bit integers by
// four-way dot products, so it is exact in any order.  The weight streams through once per group of NT
// tokens; a warp takes RW of its rows, 16 bytes a lane, and its lanes' sums meet in one reduction.
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
    // the LoRA term (B nullable)
    const void* B;
    const int32_t* idx;
    const float* s_in;
    int R, S, s_parts;
};

template <typename T> __device__ __forceinline__ float lora_dot(const SmallArgs& a, int t, int o) {
    const int slot = __ldcg(a.idx + t);
    if (slot < 0) return 0.f;
    const T* b = static_cast<const T*>(a.B) + ((size_t)slot * a.w.rows + o) * a.R;
    const size_t part = (size_t)a.x.rows * a.R;
    const float* s = a.s_in + (size_t)t * a.R;
    float acc = 0.f;
    for (int j = 0; j < a.R; ++j) {
        float v = 0.f;
        for (int p = 0; p < a.s_parts; ++p) v += __ldcg(s + p * part + j);
        acc = fmaf(to_f32<T>(b[j]), v, acc);
    }
    return acc;
}

template <typename T, int NT, int RW>
__global__ void __launch_bounds__(kSmallThreads)
i8_small_kernel(const SmallArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int o0 = (blockIdx.x * (kSmallThreads / 32) + warp) * RW, t0 = blockIdx.y * NT;
    const int n = a.x.rows, h_out = a.w.rows;
    pdl_wait();
    if (a.early_w) pdl_trigger();
    if (a.status && __ldcg(a.status) != LORA_OK) return;
    if (o0 >= h_out) return;
    int acc[RW][NT] = {};
    const int pitch = (int)a.w.pitch;
    for (int k = lane * 16; k < pitch; k += 512) {
        int4 wv[RW], xv[NT];
#pragma unroll
        for (int i = 0; i < RW; ++i)
            wv[i] = __ldcs(reinterpret_cast<const int4*>(a.w.codes + (size_t)min(o0 + i, h_out - 1) * pitch + k));
#pragma unroll
        for (int j = 0; j < NT; ++j)
            xv[j] = __ldcg(reinterpret_cast<const int4*>(a.x.codes + (size_t)min(t0 + j, n - 1) * pitch + k));
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[i][j] = __dp4a(wv[i].x, xv[j].x, acc[i][j]);
                acc[i][j] = __dp4a(wv[i].y, xv[j].y, acc[i][j]);
                acc[i][j] = __dp4a(wv[i].z, xv[j].z, acc[i][j]);
                acc[i][j] = __dp4a(wv[i].w, xv[j].w, acc[i][j]);
            }
    }
    int mine = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int v = __reduce_add_sync(0xffffffffu, acc[i][j]);
            if (lane == j * RW + i) mine = v;
        }
    const int o = o0 + lane % RW, t = t0 + lane / RW;
    if (lane >= RW * NT || o >= h_out || t >= n) return;
    float v = i8_scaled(mine, __ldcg(a.x.scales + t), __ldg(a.w.scales + o));
    if (a.B) v += lora_dot<T>(a, t, o);
    static_cast<T*>(a.y)[(long long)t * a.ldy + o] = from_f32<T>(v);
}

template <typename T>
static int launch_small_t(const SmallArgs& a, cudaStream_t st) {
    const int n = a.x.rows, rw = n <= 2 ? 2 : 4, nt = n == 1 ? 1 : n == 2 ? 2 : n <= 4 ? 4 : 8;
    const void* fn = nt == 1   ? (const void*)i8_small_kernel<T, 1, 2>
                     : nt == 2 ? (const void*)i8_small_kernel<T, 2, 2>
                     : nt == 4 ? (const void*)i8_small_kernel<T, 4, 4>
                               : (const void*)i8_small_kernel<T, 8, 4>;
    const int rows = kSmallThreads / 32 * rw;
    const dim3 grid((a.w.rows + rows - 1) / rows, (n + nt - 1) / nt);
    if (grid.y > 65535) return set_error(LORA_EUNSUP, "8-bit product of %d rows", n);
    void* args[] = {(void*)&a};
    LORA_CUDA_TRY(launch_pdl(fn, grid, dim3(kSmallThreads), 0, st, args));
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
        a.S = lora->pool->S;
        a.s_parts = lora->s_parts;
    }
    switch (dtype) {
        case LORA_F32: return launch_small_t<float>(a, st);
        case LORA_F16: return launch_small_t<__half>(a, st);
        default: return launch_small_t<__nv_bfloat16>(a, st);
    }
}

}  // namespace lora
