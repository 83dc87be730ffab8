// Products of many tokens over an 8-bit weight: persistent tiles on CTA pairs (tcgen05 cta_group::2).
//
// As in i8_tile.cu codes are float16 operands and every 1024 codes the accumulator is read into 32-bit
// integers, so sums are exact.  A pair of CTAs shares a tile of 256 features x N <= 256 tokens, each staging
// half of both.  Here both operands come as float16: with hundreds of tokens the weight's 3 bytes a code of
// extra traffic, once a call, cost less than converting it on the SM for every tile of tokens (through
// tensor memory, as i8_tile.cu does: 8191 x 11008 x 4096 took 580 us, its MMAs alone 364; the thread that
// issues them then waits for two more barriers and commits to two more every 64 codes).
//
// Tensor memory: two accumulators of N columns, so that the MMAs go on while one is read.
//
// Warps: 0 loads, 1 issues MMAs (even CTA), 2-9 drain the accumulator: lane <-> feature, every second 16
// tokens.  They add the LoRA term in float32 (tokens come in the order of the segments: neighbours share
// their adapter's rows of B) and write y through shared memory while the MMAs are at the next tile.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "i8_device.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace lora {
namespace tc {

using namespace ptx;

constexpr int kJM = 128;           // features per CTA
constexpr int kJMaxN = 256;        // tokens per pair tile, at most
constexpr int kJThreads = 320;
constexpr int kJChunk = 16;        // steps of 64 codes between two readings of the accumulator
constexpr uint32_t kJWBytes = kJM * 128;
constexpr int kJMaxStages = 8;
constexpr int kJUnits = kJMaxN / 32;  // 16-token units of a drain warp, at most
constexpr int kJStage = 16 * 33;      // floats a drain warp stages: 16 tokens x 32 features, rows padded
constexpr size_t kJTail = 8 * kJStage * 4 + kJMaxN * 12 + 512 + 1024;
constexpr size_t kJSmemMax = 227 * 1024;

struct I8PairArgs {
    void* y;
    int32_t* status;       // nullable
    const int32_t* perm;   // row of y of each row of x (nullable)
    const float* sx;
    const float* sw;
    long long ldy;
    int n, N, h_out, m_tiles, n_tiles, nkb, stages, release, vec;
    // the LoRA term (FUSE)
    const SlotEntry* table;
    const void* B;
    const int32_t* idx;    // by token
    const float* s;        // [n][R], by token
    int R;
};

template <typename T, bool FUSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kJThreads, 1)
i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8PairArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const int stages = a.stages, N = a.N;
    const uint32_t x_bytes = static_cast<uint32_t>(N) * 64;      // N / 2 rows of 64 float16
    const uint32_t stage_bytes = kJWBytes + x_bytes;
    float* staged = reinterpret_cast<float*>(smem + stages * stage_bytes);  // [8 warps][16][33]
    int* row_sm = reinterpret_cast<int*>(staged + 8 * kJStage);  // [N] row of y of a token of the tile (-1: none)
    int* slot_sm = row_sm + kJMaxN;                              // [N] its adapter
    float* sx_sm = reinterpret_cast<float*>(slot_sm + kJMaxN);   // [N] its scale
    uint64_t* full = reinterpret_cast<uint64_t*>(sx_sm + kJMaxN);  // even CTA: both CTAs' halves landed
    uint64_t* empty = full + kJMaxStages;      // (multicast)
    uint64_t* acc_full = empty + kJMaxStages;  // [2] (multicast)
    uint64_t* acc_empty = acc_full + 2;        // [2] even CTA (8 warps of both CTAs)
    uint64_t* drained = acc_empty + 2;         // even CTA: every MMA has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);  // abort
    static_assert((2 * kJMaxStages + 5) * 8 + 8 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int total = a.m_tiles * a.n_tiles;
    const int nkb = a.nkb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);
        }
        mbar_init(drained, 1);
        flags[0] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either arrives on the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (a.release) pdl_trigger();

    // tile -> features 256 (tile % m_tiles).., tokens N (tile / m_tiles)..: the pairs at work at one time share
    // the tokens of few tiles and the whole weight
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            auto load_w = [&](int s, int kb, int m0) {
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
                tma_load_2d_pair(smem + s * stage_bytes, &tmW, full0 + static_cast<uint32_t>(s) * 8u, kb * 64,
                                 m0 + static_cast<int>(rank) * kJM);
            };
            auto load_x = [&](int s, int kb, int n0) {
                tma_load_2d_pair(smem + s * stage_bytes + kJWBytes, &tmX, full0 + static_cast<uint32_t>(s) * 8u, kb * 64,
                                 n0 + static_cast<int>(rank) * (N / 2));
            };
            pdl_wait();
            int it = 0, s = 0;
            uint32_t ph = 0;
            for (int tile = pair; tile < total && !flags[0]; tile += npairs) {
                const int m0 = tile % a.m_tiles * 2 * kJM, n0 = tile / a.m_tiles * N;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    if (it >= stages && !mbar_wait(&empty[s], ph ^ 1, flags)) break;
                    load_w(s, kb, m0);
                    load_x(s, kb, n0);
                    if (++s == stages) s = 0, ph ^= 1;
                }
            }
            if (flags[0]) {  // aborted: give the copies in flight (both CTAs') time to land
                if (a.status) report_timeout_status(a.status);
                const unsigned long long t0 = globaltimer();
                while (globaltimer() - t0 < kWaitLimitNs / 8) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_f16(2 * kJM, N, false);
            bool ok = true;
            int s = 0, chunk = 0;
            uint32_t ph = 0;
            for (int tile = pair; tile < total && ok; tile += npairs) {
                for (int kb = 0; kb < nkb && ok; ++chunk) {
                    const int buf = chunk & 1, end = min(nkb, kb + kJChunk);
                    const uint32_t acc = tmem + buf * N;
                    if (chunk >= 2 && !mbar_wait(&acc_empty[buf], ((chunk >> 1) & 1) ^ 1, flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t more = 0;
                    for (; kb < end; ++kb) {
                        if (!mbar_wait(&full[s], ph, flags)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t wd = sdesc_sw128(smem_u32(smem + s * stage_bytes)), xd = wd + (kJWBytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            umma_pair_f16(acc, wd + 2 * k, xd + 2 * k, idesc, more);
                            more = 1;
                        }
                        umma_pair_commit(&empty[s], 0x3);
                        if (++s == stages) s = 0, ph ^= 1;
                    }
                    if (ok) umma_pair_commit(&acc_full[buf], 0x3);
                }
            }
            if (!ok && a.status) report_timeout_status(a.status);
            // every MMA issued above has completed before the pair may tear down
            umma_pair_commit(drained, 0x1);
            const unsigned long long t0 = globaltimer();
            while (!mbar_try_wait(drained, 0) && globaltimer() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        // ---- drain ----
        const int q = warp & 3, hv = (warp - 2) >> 2, lt = threadIdx.x - 64;
        const int units = N / 16;
        const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
        float* st = staged + (warp - 2) * kJStage;
        pdl_wait();
        const bool store = !a.status || __ldcg(a.status) == LORA_OK;
        T* y = static_cast<T*>(a.y);
        int chunk = 0;
        bool ok = true;
        for (int tile = pair; tile < total; tile += npairs) {
            const int o0 = tile % a.m_tiles * 2 * kJM + static_cast<int>(rank) * kJM + q * 32, n0 = tile / a.m_tiles * N;
            const int o = o0 + lane;
            named_bar_sync(2, 256);  // the tile before is through with the tokens' rows
            if (lt < N) {
                const int r = n0 + lt;
                const bool live = r < a.n && store;
                const int t = !live ? -1 : a.perm ? __ldcg(a.perm + r) : r;
                row_sm[lt] = t;
                sx_sm[lt] = live ? __ldcg(a.sx + r) : 0.f;
                if constexpr (FUSE) slot_sm[lt] = live ? __ldcg(a.idx + t) : -1;
            }
            const float sw = o < a.h_out ? __ldg(a.sw + o) : 0.f;
            named_bar_sync(2, 256);
            int sum[kJUnits][16];
#pragma unroll
            for (int i = 0; i < kJUnits; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[i][e] = 0;
            for (int kb = 0; kb < nkb; kb += kJChunk, ++chunk) {
                const int buf = chunk & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (chunk >> 1) & 1, flags));
                if (!ok) break;
                tc_fence_after();
                const uint32_t taddr = tmem + buf * N + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
                for (int i = 0; i < kJUnits; ++i) {
                    const int u = 2 * i + hv;
                    if (u < units) {
                        uint32_t r[16];
                        __syncwarp();
                        tmem_ld16(taddr + u * 16, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[i][e] += __float2int_rn(__uint_as_float(r[e]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + static_cast<uint32_t>(buf) * 8u);
            }
            // all eight warps leave together
            if (!named_bar_and(3, 256, ok)) break;
            if (!store) continue;
#pragma unroll 1
            for (int i = 0; i < kJUnits; ++i) {
                const int u = 2 * i + hv;
                if (u >= units) break;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kJUnits; ++j)
                    if (j == i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) st[e * 33 + lane] = i8_scaled(sum[j][e], sx_sm[u * 16 + e], sw);
                if constexpr (FUSE) {
                    const T* Bo = static_cast<const T*>(a.B) + (size_t)min(o, a.h_out - 1) * a.R;
                    const size_t slot_elems = (size_t)a.h_out * a.R;
#pragma unroll 1
                    for (int e0 = 0; e0 < 16; e0 += 4) {
                        int slot[4];
                        const float* sp[4];
                        bool same = true, any = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = u * 16 + e0 + k;
                            slot[k] = slot_sm[t];
                            sp[k] = a.s + (size_t)max(row_sm[t], 0) * a.R;
                            same = same && slot[k] == slot[0];
                            any = any || slot[k] >= 0;
                        }
                        if (!any) continue;
                        float acc[4] = {};
                        if (same) {
                            const T* b = Bo + slot[0] * slot_elems;
                            const int jl = a.table[slot[0]].rank;  // columns past the rank are zeros
                            for (int j = 0; j < jl; j += 8) {
                                float bf[8];
                                load_b8<T>(b, j, a.R, bf);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    float sv[8];
                                    load_s8(sp[k], j, a.R, jl, sv);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) acc[k] = fmaf(bf[e], sv[e], acc[k]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (slot[k] < 0) continue;
                                const T* b = Bo + slot[k] * slot_elems;
                                const int jl = a.table[slot[k]].rank;
                                for (int j = 0; j < jl; j += 8) {
                                    float bf[8], sv[8];
                                    load_b8<T>(b, j, a.R, bf);
                                    load_s8(sp[k], j, a.R, jl, sv);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) acc[k] = fmaf(bf[e], sv[e], acc[k]);
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) st[(e0 + k) * 33 + lane] += acc[k];
                    }
                }
                __syncwarp();
                if (a.vec) {
                    // 16 bytes a lane, neighbouring lanes a token's 32 features
                    constexpr int per = 16 / sizeof(T), lanes = 32 / per;
                    const int c = (lane % lanes) * per, col = o0 + c;
#pragma unroll
                    for (int e0 = 0; e0 < 16; e0 += 32 / lanes) {
                        const int e = e0 + lane / lanes, row = row_sm[u * 16 + e];
                        alignas(16) T w[per];
#pragma unroll
                        for (int k = 0; k < per; ++k) w[k] = from_f32<T>(st[e * 33 + c + k]);
                        if (row < 0) continue;
                        T* yp = y + (long long)row * a.ldy + col;
                        if (col + per <= a.h_out) {
                            *reinterpret_cast<uint4*>(yp) = *reinterpret_cast<const uint4*>(w);
                        } else {
#pragma unroll
                            for (int k = 0; k < per; ++k)
                                if (col + k < a.h_out) yp[k] = w[k];
                        }
                    }
                } else if (o < a.h_out) {
                    for (int e = 0; e < 16; ++e) {
                        const int row = row_sm[u * 16 + e];
                        if (row >= 0) y[(long long)row * a.ldy + o] = from_f32<T>(st[e * 33 + lane]);
                    }
                }
            }
        }
        if (!ok && a.status && lane == 0) report_timeout_status(a.status);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves (or frees tensor memory) while its pair may still use it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Pairs the GPU holds at once (an SM left over in a group of SMs cannot host a pair).
static int max_pairs() {
    static int pairs = 0;  // every variant takes all of an SM's shared memory: the same for each
    if (!pairs) {
        cudaLaunchConfig_t q;
        memset(&q, 0, sizeof(q));
        q.gridDim = dim3(2 * (num_sms() / 2));
        q.blockDim = dim3(kJThreads);
        q.dynamicSmemBytes = kJSmemMax;
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 2;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, (const void*)i8_pair_kernel<float, false>, &q) != cudaSuccess || c < 1) {
            (void)cudaGetLastError();
            c = num_sms() / 2;
        }
        pairs = std::min(c, num_sms() / 2);
    }
    return pairs;
}

template <typename T, bool FUSE>
static int launch_pair_t(const I8Rows& x, const I8Rows& w, void* y, long long ldy, int32_t* status, bool release,
                         const I8Lora* lora, cudaStream_t st) {
    static bool attr = false;
    if (!attr) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(i8_pair_kernel<T, FUSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kJSmemMax));
        LORA_CUDA_TRY(cudaFuncSetAttribute(i8_pair_kernel<float, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kJSmemMax));
        attr = true;
    }
    I8PairArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.status = status;
    a.perm = x.perm;
    a.sx = x.scales;
    a.sw = w.scales;
    a.ldy = ldy;
    a.n = x.rows;
    a.h_out = w.rows;
    a.m_tiles = (w.rows + 2 * kJM - 1) / (2 * kJM);
    const size_t pitch = i8_pitch(x.cols);
    a.nkb = (int)((pitch + 63) / 64);
    a.release = release;
    a.vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (long long)sizeof(T)) % 16 == 0;
    // tokens a tile: as few as fill the pairs' last round best
    const int pairs = max_pairs();
    long long best = LLONG_MAX;
    for (int N = kJMaxN; N >= 96; N -= 32) {
        const long long tiles = (long long)a.m_tiles * ((x.rows + N - 1) / N), cost = (tiles + pairs - 1) / pairs * (N + 8);
        if (cost < best) best = cost, a.N = N;
    }
    a.n_tiles = (x.rows + a.N - 1) / a.N;
    const long long tiles = (long long)a.m_tiles * a.n_tiles;
    if (tiles * a.nkb > INT_MAX / 2) return set_error(LORA_EUNSUP, "8-bit product of %d x %d outputs is too large", x.rows, w.rows);
    if (lora) {
        const PoolView& pv = *lora->pool;
        a.table = pv.table;
        a.B = pv.B;
        a.idx = lora->idx;
        a.s = lora->s_in;
        a.R = pv.R;
    }
    const size_t stage_bytes = kJWBytes + (size_t)a.N * 64;
    a.stages = (int)std::min<size_t>((kJSmemMax - kJTail) / stage_bytes, kJMaxStages);
    CUtensorMap mW, mX;
    int rc = make_map(&mW, w.x16, 0, pitch, w.rows, kJM);
    if (!rc) rc = make_map(&mX, x.x16, 0, pitch, x.rows, a.N / 2);
    if (rc) return rc;
    void* args[] = {(void*)&mW, (void*)&mX, (void*)&a};
    LORA_CUDA_TRY(launch_pdl((const void*)i8_pair_kernel<T, FUSE>, dim3(2 * (unsigned)std::min<long long>(tiles, pairs)),
                             dim3(kJThreads), a.stages * stage_bytes + kJTail, st, args));
    return LORA_OK;
}

}  // namespace tc

int launch_i8_pair(const I8Rows& x, const I8Rows& w, void* y, int dtype, long long ldy, int32_t* status,
                   bool release, const I8Lora* lora, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32:
            return lora ? tc::launch_pair_t<float, true>(x, w, y, ldy, status, release, lora, st)
                        : tc::launch_pair_t<float, false>(x, w, y, ldy, status, release, nullptr, st);
        case LORA_F16:
            return lora ? tc::launch_pair_t<__half, true>(x, w, y, ldy, status, release, lora, st)
                        : tc::launch_pair_t<__half, false>(x, w, y, ldy, status, release, nullptr, st);
        default:
            return lora ? tc::launch_pair_t<__nv_bfloat16, true>(x, w, y, ldy, status, release, lora, st)
                        : tc::launch_pair_t<__nv_bfloat16, false>(x, w, y, ldy, status, release, nullptr, st);
    }
}

}  // namespace lora
