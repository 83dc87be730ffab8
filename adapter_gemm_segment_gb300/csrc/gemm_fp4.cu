// Product of two microscaled 4-bit matrices on the tensor cores (tcgen05 kind::mxf4, the block
// scales applied by the instruction, float32 accumulation in tensor memory).
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace lora {
namespace tc {

using namespace ptx;

constexpr int kF4M = 128;        // rows of the M operand per tile (MMA M)
constexpr int kF4N = 256;        // rows of the N operand per tile
constexpr int kF4K = 256;        // elements of K per stage: one 128-byte swizzle row of codes, 2 scale tiles
constexpr int kF4Threads = 192;  // producer warp, MMA warp, 4 epilogue warps
constexpr int kF4Stages = 4;
constexpr uint32_t kF4ABytes = kF4M * 128, kF4BBytes = kF4N * 128;
constexpr uint32_t kF4SaBytes = 1024, kF4SbBytes = 2048;
constexpr uint32_t kF4StageBytes = kF4ABytes + kF4BBytes + kF4SaBytes + kF4SbBytes;
static_assert(kF4StageBytes % 1024 == 0, "swizzle atoms stay aligned");

struct Fp4GemmArgs {
    const uint8_t* sx;  // scale tiles of x and w
    const uint8_t* sw;
    void* y;
    int32_t* status;
    long long ldy;
    int n, h_out, nkb, ktiles;
    int early_w;
};

template <typename T>
__global__ void __launch_bounds__(kF4Threads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Fp4GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kF4Stages * kF4StageBytes);
    uint64_t* empty = full + kF4Stages;
    uint64_t* acc_full = empty + kF4Stages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = blockIdx.y * kF4M, n0 = blockIdx.x * kF4N;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kF4Stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        flags[0] = 0;
        fence_barrier_init();
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            // the second 128-row scale tile of w exists only if its rows do
            const int wtiles = n0 + 128 < a.h_out ? 2 : 1;
            const uint32_t bytes = kF4ABytes + kF4BBytes + kF4SaBytes + 1024u * wtiles;
            int it = 0;
            for (; it < a.nkb; ++it) {
                const int s = it % kF4Stages;
                if (it >= kF4Stages && !mbar_wait(&empty[s], ((it / kF4Stages) & 1) ^ 1, flags)) break;
                uint8_t* st = smem + s * kF4StageBytes;
                mbar_arrive_expect_tx(&full[s], bytes);
                tma_load_2d_cta(st, &tmX, &full[s], it * 128, m0);
                tma_load_2d_cta(st + kF4ABytes, &tmW, &full[s], it * 128, n0);
                uint8_t* sc = st + kF4ABytes + kF4BBytes;
                bulk_g2s(sc, a.sx + ((size_t)blockIdx.y * a.ktiles + 2 * it) * 512, 1024, &full[s]);
                for (int h = 0; h < wtiles; ++h)
                    bulk_g2s(sc + kF4SaBytes + h * 1024, a.sw + ((size_t)(blockIdx.x * 2 + h) * a.ktiles + 2 * it) * 512,
                             1024, &full[s]);
            }
            if (flags[0]) {
                for (int i = max(0, it - kF4Stages); i < it; ++i) {
                    const unsigned long long t0 = globaltimer();
                    while (!mbar_try_wait(&full[i % kF4Stages], (i / kF4Stages) & 1) && globaltimer() - t0 < kWaitLimitNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < a.nkb; ++i) {
                const int s = i % kF4Stages;
                if (!mbar_wait(&full[s], (i / kF4Stages) & 1, flags)) break;
                tc_fence_after();
                const uint32_t xa = smem_u32(smem + s * kF4StageBytes), wa = xa + kF4ABytes, sc = wa + kF4BBytes;
                // scale columns of this stage: x's two tiles (4 columns each), then w's (8 each)
                const uint32_t sfa = tmem + kF4N + s * 24, sfb = sfa + 8;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tmem_cp_scales(sfa + 4 * j, sdesc_scales(sc + 512 * j));
                    tmem_cp_scales(sfb + 8 * j, sdesc_scales(sc + kF4SaBytes + 512 * j));
                    tmem_cp_scales(sfb + 8 * j + 4, sdesc_scales(sc + kF4SaBytes + 1024 + 512 * j));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_mxf4(tmem, sdesc_sw128(xa + k * 32), sdesc_sw128(wa + k * 32),
                              idesc_mxf4(kF4M, kF4N, (k & 1) * 2), sfa + 4 * (k >> 1), sfb + 8 * (k >> 1),
                              (i > 0 || k > 0) ? 1u : 0u);
                umma_commit(&empty[s]);
            }
            umma_commit(acc_full);
        }
    } else {
        const int q = warp & 3;
        const int t = m0 + q * 32 + lane;
        const int status = a.status ? __ldcg(a.status) : LORA_OK;
        const bool got = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, flags));
        if (got && status == LORA_OK) {
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
            T* y = static_cast<T*>(a.y);
            for (int c0 = 0; c0 < kF4N; c0 += 16) {
                uint32_t r[16];
                __syncwarp();
                tmem_ld16(taddr + c0, r);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (t < a.n && n0 + c0 + c < a.h_out)
                        y[(long long)t * a.ldy + n0 + c0 + c] = from_f32<T>(__uint_as_float(r[c]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename T>
static int launch_fp4_gemm_t(const Fp4View& x, const Fp4View& w, void* y, long long ldy, int32_t* status,
                             bool early_w, cudaStream_t st) {
    Fp4GemmArgs a;
    a.sx = x.scales;
    a.sw = w.scales;
    a.y = y;
    a.status = status;
    a.ldy = ldy;
    a.n = x.rows;
    a.h_out = w.rows;
    a.nkb = x.ktiles / 2;
    a.ktiles = x.ktiles;
    a.early_w = early_w;
    CUtensorMap mX, mW;
    int rc = make_map_fp4(&mX, x.codes, x.pitch, x.rows, kF4M);
    if (rc) return rc;
    rc = make_map_fp4(&mW, w.codes, w.pitch, w.rows, kF4N);
    if (rc) return rc;
    const size_t smem = (size_t)kF4Stages * kF4StageBytes + 1024 + 256;
    static bool attr = false;
    if (!attr) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(fp4_gemm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        attr = true;
    }
    void* args[] = {(void*)&mX, (void*)&mW, (void*)&a};
    const dim3 grid((w.rows + kF4N - 1) / kF4N, (x.rows + kF4M - 1) / kF4M);
    LORA_CUDA_TRY(launch_pdl((const void*)fp4_gemm_kernel<T>, grid, dim3(kF4Threads), smem, st, args));
    return LORA_OK;
}

}  // namespace tc

int launch_fp4_gemm(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status,
                    bool early_w, cudaStream_t st) {
    if (x.rows > 256) return launch_fp4_pair(x, w, y, dtype, ldy, status, early_w, nullptr, st);
    switch (dtype) {
        case LORA_F32: return tc::launch_fp4_gemm_t<float>(x, w, y, ldy, status, early_w, st);
        case LORA_F16: return tc::launch_fp4_gemm_t<__half>(x, w, y, ldy, status, early_w, st);
        default: return tc::launch_fp4_gemm_t<__nv_bfloat16>(x, w, y, ldy, status, early_w, st);
    }
}

}  // namespace lora
