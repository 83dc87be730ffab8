// Products over an 8-bit weight on the tensor cores, whole-number sums kept exact.
//
// sm_103a's tensor cores take no 8-bit integers, but a code is a float16 number and a product of two codes
// is exact in float32, so is a sum of 1024 of them (1024 * 128 * 128 = 2^24).  Codes go through
// tcgen05.mma kind::f16; every 1024 of K the accumulator is read into 32-bit integers in registers and
// started again.
//
// The weight is the MMA's M side (128 features a tile) and up to 128 tokens its N side.  The weight stays
// in bytes until it is on the SM: TMA brings 128 x 128 codes, eight warps turn them into float16 and store
// them to tensor memory as the MMA's A operand (tcgen05.st), so float16 weights never pass through shared
// memory.  K is split over the CTAs of a thread-block cluster until the grid fills the GPU; the split sums
// (integers: any order gives the same) meet in shared memory, each CTA finishing its share of the tokens.
//
// The LoRA term is added there in float32: y[t, o] = sx sw sum + s[t, :] . B[o, :].  The warps that drain
// the accumulator are idle during the main loop, and compute it then for the tokens their CTA will finish.
// Tokens come in the order of the segments, so neighbouring tokens share their adapter's rows of B.
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

constexpr int kIM = 128;          // features per tile
constexpr int kIN = 128;          // tokens per tile, at most
constexpr int kIK = 128;          // codes of a step along K
constexpr int kIChunk = 8;        // steps between two readings of the accumulator: 1024 codes
constexpr int kIThreads = 576;    // warp 0 loads, 1 MMAs, 2-9 convert, 10-17 LoRA term and accumulator
constexpr int kIASlots = 4;       // at most: steps of the weight in tensor memory, 64 columns each
constexpr int kIACol = 2 * kIN;   // behind two accumulators
constexpr int kISRanks = 32;      // columns of the shrink output staged at once
constexpr uint32_t kIWBytes = kIM * kIK;
constexpr int kIBars = 512;

struct I8TileArgs {
    void* y;
    int32_t* status;       // nullable
    const int32_t* perm;   // row of y of each row of x (nullable)
    const float* sx;
    const float* sw;
    long long ldy;
    int n, n_pad, h_out, kb_total, kb_per_split, splits, stages, aslots, early, release, vec, ring_bytes, push, per;
    // the LoRA term (FUSE)
    const SlotEntry* table;
    const void* B;
    const int32_t* idx;    // by token
    const float* s_in;     // [s_parts][n][R], by token
    int R, s_parts;
};

template <typename T, bool FUSE>
__global__ void __launch_bounds__(kIThreads, 1)
i8_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8TileArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const int stages = a.stages, aslots = a.aslots, n_pad = a.n_pad;
    const uint32_t x_bytes = static_cast<uint32_t>(n_pad) * 256;  // two boxes of 64 float16 columns
    const uint32_t stage_bytes = kIWBytes + x_bytes;
    float* L = reinterpret_cast<float*>(smem + a.ring_bytes);            // FUSE: [per][128] LoRA terms
    float* S = L + (FUSE ? a.per * kIM : 0);                             // FUSE: [per][kISRanks] shrink output
    int* tok_slot = reinterpret_cast<int*>(S + (FUSE ? a.per * kISRanks : 0));  // FUSE: [per]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_align(reinterpret_cast<uint8_t*>(tok_slot + (FUSE ? a.per : 0)), 8));
    uint64_t* empty = full + stages;
    uint64_t* conv = empty + stages;          // [kIASlots] the step's weight is in tensor memory (8 warps)
    uint64_t* acc_full = conv + kIASlots;     // [2]
    uint64_t* acc_empty = acc_full + 2;       // [2] (8 warps)
    uint64_t* rbar = acc_empty + 2;           // the other CTAs' sums of this CTA's tokens have arrived
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rbar + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);  // abort
    int* P = reinterpret_cast<int*>(smem);    // after the main loop: [n_pad][128] sums of this CTA's part of K

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m_tile = blockIdx.x, split = blockIdx.y, row0 = blockIdx.z * kIN;
    const int n = min(a.n - row0, kIN);
    const int kb0 = split * a.kb_per_split;
    const int nkb = min(a.kb_total, kb0 + a.kb_per_split) - kb0;
    const int nchunks = (nkb + kIChunk - 1) / kIChunk;
    // the tokens this CTA finishes
    const int t0 = min(n, split * a.per), cnt = min(n, t0 + a.per) - t0;

    auto issue_w = [&](int i) {
        const int s = i % stages;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        tma_load_2d_cta(smem + (size_t)s * stage_bytes, &tmW, &full[s], (kb0 + i) * kIK, m_tile * kIM);
    };
    auto issue_x = [&](int i) {
        const int s = i % stages;
        uint8_t* dst = smem + (size_t)s * stage_bytes + kIWBytes;
        tma_load_2d_cta(dst, &tmX, &full[s], (kb0 + i) * kIK, row0);
        tma_load_2d_cta(dst + n_pad * 128, &tmX, &full[s], (kb0 + i) * kIK + 64, row0);
    };
    const int pre = min(stages, nkb);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kIASlots; ++s) mbar_init(&conv[s], 8);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        mbar_init(rbar, 1);
        flags[0] = 0;
        fence_barrier_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        // what is complete when this grid starts is loaded at once
        if (a.early >= 1)
            for (int i = 0; i < pre; ++i) {
                issue_w(i);
                if (a.early >= 2) issue_x(i);
            }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (a.release) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            if (a.early < 2) pdl_wait();
            if (a.early >= 1) {
                if (a.early < 2)
                    for (int i = 0; i < pre; ++i) issue_x(i);
                issued = pre;
            }
            for (int i = issued; i < nkb; ++i) {
                const int s = i % stages;
                if (i >= stages && !mbar_wait(&empty[s], ((i / stages) & 1) ^ 1, flags)) break;
                issue_w(i);
                issue_x(i);
                ++issued;
            }
            if (flags[0]) {
                if (a.status) report_timeout_status(a.status);
                for (int i = max(0, issued - stages); i < issued; ++i) {
                    const unsigned long long t = globaltimer();
                    while (!mbar_try_wait(&full[i % stages], (i / stages) & 1) && globaltimer() - t < kWaitLimitNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            const uint32_t idesc = idesc_f16(kIM, n_pad, false);
            int i = 0;
            for (int c = 0; c < nchunks && ok; ++c) {
                const int buf = c & 1, end = min(nkb, (c + 1) * kIChunk);
                const uint32_t acc = tmem + buf * n_pad;
                if (c >= 2 && !mbar_wait(&acc_empty[buf], ((c >> 1) & 1) ^ 1, flags)) {
                    ok = false;
                    break;
                }
                for (bool first = true; i < end; ++i) {
                    const int s = i % stages, slot = i % aslots;
                    if (!mbar_wait(&full[s], (i / stages) & 1, flags) || !mbar_wait(&conv[slot], (i / aslots) & 1, flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t xa = smem_u32(smem + (size_t)s * stage_bytes + kIWBytes);
                    const uint32_t wa = tmem + kIACol + slot * 64;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        umma_f16_ta(acc, wa + k * 8, sdesc_sw128(xa + (k >> 2) * n_pad * 128 + (k & 3) * 32), idesc,
                                    first ? 0u : 1u);
                        first = false;
                    }
                    umma_commit(&empty[s]);
                }
                if (ok) umma_commit(&acc_full[buf]);
            }
            if (!ok) {
                if (a.status) report_timeout_status(a.status);
                // every MMA issued above completes before the CTA may leave
                umma_commit(rbar);
                const unsigned long long t = globaltimer();
                while (!mbar_try_wait(rbar, 0) && globaltimer() - t < kWaitLimitNs) {
                }
            }
        }
    } else if (warp < 10) {
        // ---- codes to float16 in tensor memory: 32 features and 64 codes of a step a warp ----
        const int q = warp & 3, h = (warp - 2) >> 2;
        const int row = q * 32 + lane;
        const uint32_t taddr = tmem + kIACol + h * 32 + (static_cast<uint32_t>(q * 32) << 16);
        for (int i = 0; i < nkb; ++i) {
            const int s = i % stages, slot = i % aslots;
            bool ok = mbar_wait(&full[s], (i / stages) & 1, flags);
            // the slot's last readers
            if (ok && i >= aslots) ok = mbar_wait(&empty[(i - aslots) % stages], ((i - aslots) / stages) & 1, flags);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint8_t* wr = smem + (size_t)s * stage_bytes + row * 128;
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(wr + (((h * 4 + c) ^ (row & 7)) << 4));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint2 f = i8_to_f16x4(w[e]);
                    r[c * 8 + e * 2] = f.x;
                    r[c * 8 + e * 2 + 1] = f.y;
                }
            }
            tc_fence_after();
            tmem_st32(taddr + slot * 64, r);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&conv[slot]);
        }
    } else {
        const int lt = threadIdx.x - 320;  // 0..255
        if constexpr (FUSE) {
            // ---- the LoRA terms of this CTA's tokens: a feature a thread, every second token ----
            const int f = lt & 127, half = lt >> 7, o = m_tile * kIM + f, R = a.R;
            if (a.early < 2) pdl_wait();  // (perm and the segments are older than the kernel ahead otherwise)
            const bool st_ok = !a.status || __ldcg(a.status) == LORA_OK;
            for (int u = lt; u < cnt; u += 256) tok_slot[u] = st_ok ? __ldcg(a.idx + __ldcg(a.perm + row0 + t0 + u)) : -1;
            pdl_wait();  // the shrink output
            const size_t part = (size_t)a.n * R;
            for (int j0 = 0; j0 < R; j0 += kISRanks) {
                named_bar_sync(2, 256);
                for (int e = lt; e < cnt * kISRanks; e += 256) {
                    const int u = e / kISRanks, j = j0 + e % kISRanks;
                    float v = 0.f;
                    if (tok_slot[u] >= 0 && j < a.table[tok_slot[u]].rank) {
                        const float* sp = a.s_in + (size_t)__ldcg(a.perm + row0 + t0 + u) * R + j;
                        for (int p = 0; p < a.s_parts; ++p) v += __ldcg(sp + p * part);
                    }
                    S[e] = v;
                }
                named_bar_sync(2, 256);
                const int jn = min(kISRanks, R - j0);
                for (int u0 = half; u0 < cnt; u0 += 8) {  // four tokens at once
                    float acc[4];
                    int slot[4];
                    bool same = true;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int u = u0 + 2 * k;
                        slot[k] = u < cnt ? tok_slot[u] : -1;
                        acc[k] = j0 > 0 && u < cnt ? L[u * kIM + f] : 0.f;
                        same = same && slot[k] == slot[0];
                    }
                    if (o < a.h_out) {
                        const T* Bo = static_cast<const T*>(a.B) + (size_t)o * R + j0;
                        if (same) {
                            if (slot[0] >= 0) {
                                const T* b = Bo + (size_t)slot[0] * a.h_out * R;
                                const int jl = min(jn, a.table[slot[0]].rank - j0);  // columns past the rank are zeros
                                for (int j = 0; j < jl; j += 8) {
                                    float bf[8];
                                    load_b8<T>(b, j, R - j0, bf);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float* sp = S + min(u0 + 2 * k, cnt - 1) * kISRanks + j;
#pragma unroll
                                        for (int e = 0; e < 8; ++e) acc[k] = fmaf(bf[e], sp[e], acc[k]);
                                    }
                                }
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (slot[k] < 0) continue;
                                const T* b = Bo + (size_t)slot[k] * a.h_out * R;
                                const int jl = min(jn, a.table[slot[k]].rank - j0);
                                const float* sp = S + (u0 + 2 * k) * kISRanks;
                                for (int j = 0; j < jl; j += 8) {
                                    float bf[8];
                                    load_b8<T>(b, j, R - j0, bf);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) acc[k] = fmaf(bf[e], sp[j + e], acc[k]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (u0 + 2 * k < cnt) L[(u0 + 2 * k) * kIM + f] = acc[k];
                }
            }
        }
        // ---- accumulator: 32 features a warp, every second 16 tokens; its chunks added up in integers ----
        const int q = warp & 3, hv = (warp - 10) >> 2;
        const int units = n_pad / 16;
        int sum[4][16] = {};
        bool ok = true;
        for (int c = 0; c < nchunks && ok; ++c) {
            const int buf = c & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (c >> 1) & 1, flags));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + buf * n_pad + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
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
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        if (ok) {
            // (the last accumulator is complete: every MMA has read its operands, the ring is idle)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = 2 * i + hv;
                if (u < units)
#pragma unroll
                    for (int e = 0; e < 16; ++e) P[(u * 16 + e) * kIM + q * 32 + lane] = sum[i][e];
            }
            fence_proxy_async_smem();  // read by the bulk copies
        } else if (lane == 0) {
            flags[0] = 1;
        }
    }
    bool store = false;
    if (warp >= 2) {
        pdl_wait();
        store = !a.status || __ldcg(a.status) == LORA_OK;
    }
    tc_fence_before();
    __syncthreads();
    // ---- each CTA adds up its share of the tokens and stores them.  The sums reach their owner by one bulk copy
    // from each other CTA (a token's row is 512 bytes, an owner's rows are contiguous) where a receive buffer
    // fits, else they are read remotely. ----
    bool good = flags[0] == 0;
    int* rcv = P + (size_t)n_pad * kIM;  // [splits - 1][per][128]
    bool recv = true;
    if (a.splits > 1) {
        if (a.push && threadIdx.x == 64 && cnt > 0 && good)
            mbar_arrive_expect_tx(rbar, static_cast<uint32_t>((a.splits - 1) * cnt * kIM * 4));
        cluster_sync();
        good = cluster_unaborted(flags, a.splits);
        if (a.push) {
            const int dst = (int)threadIdx.x - 64;
            if (good && dst >= 0 && dst < a.splits && dst != split) {
                const int d0 = min(n, dst * a.per), dcnt = min(n, d0 + a.per) - d0;
                if (dcnt > 0)
                    bulk_s2cluster(mapa_shared(smem_u32(rcv + (size_t)(split < dst ? split : split - 1) * a.per * kIM),
                                               static_cast<uint32_t>(dst)),
                                   P + (size_t)d0 * kIM, static_cast<uint32_t>(dcnt * kIM * 4),
                                   mapa_shared(smem_u32(rbar), static_cast<uint32_t>(dst)));
            }
            __syncwarp();
            if (good && cnt > 0) recv = __all_sync(0xffffffffu, mbar_wait(rbar, 0, flags));
            cluster_arrive();  // (the last wait below: every copy out of this CTA has then landed)
        }
    }
    if (warp >= 2 && good && store && recv) {
        T* y = static_cast<T*>(a.y);
        auto yrow = [&](int u) -> T* {
            const int r = row0 + t0 + u;
            return y + (long long)(a.perm ? __ldcg(a.perm + r) : r) * a.ldy;
        };
        const int ot = threadIdx.x - 64;  // 0..511
        if (a.vec) {
            // 8 features a thread, 16 neighbouring threads a token's 128
            const int o8 = (ot & 15) * 8, o = m_tile * kIM + o8;
            float sw[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) sw[e] = o + e < a.h_out ? __ldg(a.sw + o + e) : 0.f;
            for (int u = ot >> 4; u < cnt; u += 32) {
                int v[8];
                const int4* own = reinterpret_cast<const int4*>(P + (t0 + u) * kIM + o8);
                *reinterpret_cast<int4*>(v) = own[0];
                *reinterpret_cast<int4*>(v + 4) = own[1];
                for (int c = 0; c < a.splits; ++c) {
                    if (c == split) continue;
                    if (a.push) {
                        const int4* p =
                            reinterpret_cast<const int4*>(rcv + ((size_t)(c < split ? c : c - 1) * a.per + u) * kIM + o8);
                        const int4 lo = p[0], hi = p[1];
                        v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
                        v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
                    } else {
                        const uint32_t at = mapa_shared(smem_u32(own), static_cast<uint32_t>(c));
                        const float4 lo = ld_dsmem_f32x4(at), hi = ld_dsmem_f32x4(at + 16);
                        v[0] += __float_as_int(lo.x), v[1] += __float_as_int(lo.y), v[2] += __float_as_int(lo.z);
                        v[3] += __float_as_int(lo.w), v[4] += __float_as_int(hi.x), v[5] += __float_as_int(hi.y);
                        v[6] += __float_as_int(hi.z), v[7] += __float_as_int(hi.w);
                    }
                }
                const float sx = __ldcg(a.sx + row0 + t0 + u);
                alignas(16) T w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float r = i8_scaled(v[e], sx, sw[e]);
                    if constexpr (FUSE) r += L[u * kIM + o8 + e];
                    w[e] = from_f32<T>(r);
                }
                T* yp = yrow(u) + o;
                if (o + 8 <= a.h_out) {
#pragma unroll
                    for (int e = 0; e < (int)(8 * sizeof(T) / 16); ++e)
                        reinterpret_cast<uint4*>(yp)[e] = reinterpret_cast<const uint4*>(w)[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (o + e < a.h_out) yp[e] = w[e];
                }
            }
        } else {
            // rows off 16-byte boundaries: a feature a thread, neighbours side by side
            const int f = ot & 127, o = m_tile * kIM + f;
            const float sw = o < a.h_out ? __ldg(a.sw + o) : 0.f;
            for (int u = ot >> 7; u < cnt; u += 4) {
                const int* own = P + (t0 + u) * kIM + f;
                int v = *own;
                for (int c = 0; c < a.splits; ++c) {
                    if (c == split) continue;
                    v += a.push ? rcv[((size_t)(c < split ? c : c - 1) * a.per + u) * kIM + f]
                                : __float_as_int(ld_dsmem_f32(mapa_shared(smem_u32(own), static_cast<uint32_t>(c))));
                }
                float r = i8_scaled(v, __ldcg(a.sx + row0 + t0 + u), sw);
                if constexpr (FUSE) r += L[u * kIM + f];
                if (o < a.h_out) yrow(u)[o] = from_f32<T>(r);
            }
        }
    }
    if (!recv && a.status) report_timeout_status(a.status);
    // no CTA leaves while its sums may still be read or copied
    if (a.splits > 1) {
        if (!a.push) cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename T, bool FUSE>
static int launch_tile_t(const I8Rows& x, const I8View& w, void* y, long long ldy, int32_t* status, int early, bool release,
                         const I8Lora* lora, cudaStream_t st) {
    I8TileArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.status = status;
    a.perm = x.perm;
    a.sx = x.scales;
    a.sw = w.scales;
    a.ldy = ldy;
    a.n = x.rows;
    a.n_pad = (std::min(x.rows, kIN) + 15) / 16 * 16;
    a.h_out = w.rows;
    a.kb_total = (int)((w.pitch + kIK - 1) / kIK);
    a.early = early;
    a.release = release;
    // y is written 16 bytes at a time when every row starts on a 16-byte boundary
    a.vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (long long)sizeof(T)) % 16 == 0;
    const int m_tiles = (w.rows + kIM - 1) / kIM, groups = (x.rows + kIN - 1) / kIN;
    if (groups > 65535) return set_error(LORA_EUNSUP, "8-bit product of %d rows", x.rows);
    // CTAs (a cluster) that share K: as many as let every tile have an SM a CTA
    const long long tiles = (long long)m_tiles * groups;
    const int splits = (int)std::min<long long>({std::max<long long>(1, num_sms() / tiles), 8, a.kb_total});
    a.kb_per_split = (a.kb_total + splits - 1) / splits;
    a.splits = (a.kb_total + a.kb_per_split - 1) / a.kb_per_split;
    a.per = (std::min(x.rows, kIN) + a.splits - 1) / a.splits;
    if (lora) {
        const PoolView& pv = *lora->pool;
        a.table = pv.table;
        a.B = pv.B;
        a.idx = lora->idx;
        a.s_in = lora->s_in;
        a.R = pv.R;
        a.s_parts = lora->s_parts;
    }
    const size_t tail = (FUSE ? (size_t)a.per * (kIM + kISRanks + 1) * 4 : 0) + kIBars + 1024 + 16;
    const size_t room = 227 * 1024 - tail;
    const size_t stage_bytes = kIWBytes + (size_t)a.n_pad * 256;
    a.stages = (int)std::min<size_t>({room / stage_bytes, 8, (size_t)a.kb_per_split});
    a.aslots = std::min(kIASlots, a.stages);  // (no more: a slot's last reader is found by its stage's barrier)
    // the stages are idle when the sums are parked in their place
    const size_t park = (size_t)a.n_pad * kIM * 4, rcv = (size_t)(a.splits - 1) * a.per * kIM * 4;
    a.push = a.splits > 1 && park + rcv <= room / 1024 * 1024;
    a.ring_bytes = (int)((std::max(a.stages * stage_bytes, park + (a.push ? rcv : 0)) + 1023) / 1024 * 1024);
    const size_t smem = a.ring_bytes + tail;
    if (a.stages < 1 || smem > 227 * 1024) return set_error(LORA_EUNSUP, "internal: 8-bit tile plan");
    CUtensorMap mW, mX;
    int rc = make_map_fp4(&mW, w.codes, w.pitch, w.rows, kIM);  // (bytes in boxes of 128)
    if (!rc) rc = make_map(&mX, x.x16, 0, w.pitch, x.rows, a.n_pad);
    if (rc) return rc;
    static bool attr_set = false;
    if (!attr_set) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(i8_tile_kernel<T, FUSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
        attr_set = true;
    }
    void* args[] = {(void*)&mW, (void*)&mX, (void*)&a};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(m_tiles, a.splits, groups);
    cfg.blockDim = dim3(kIThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = a.splits;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    LORA_CUDA_TRY(cudaLaunchKernelExC(&cfg, (const void*)i8_tile_kernel<T, FUSE>, args));
    count_launch();
    return LORA_OK;
}

}  // namespace tc

int launch_i8_tile(const I8Rows& x, const I8View& w, void* y, int dtype, long long ldy, int32_t* status, int early,
                   bool release, const I8Lora* lora, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32:
            return lora ? tc::launch_tile_t<float, true>(x, w, y, ldy, status, early, release, lora, st)
                        : tc::launch_tile_t<float, false>(x, w, y, ldy, status, early, release, nullptr, st);
        case LORA_F16:
            return lora ? tc::launch_tile_t<__half, true>(x, w, y, ldy, status, early, release, lora, st)
                        : tc::launch_tile_t<__half, false>(x, w, y, ldy, status, early, release, nullptr, st);
        default:
            return lora ? tc::launch_tile_t<__nv_bfloat16, true>(x, w, y, ldy, status, early, release, lora, st)
                        : tc::launch_tile_t<__nv_bfloat16, false>(x, w, y, ldy, status, early, release, nullptr, st);
    }
}

}  // namespace lora
