// Batches of up to 256 tokens over a 4-bit base weight.
//
// The weight is the MMA's M side (128 features a tile) and the tokens its N side, so the weight
// streams through once; K is split over the CTAs of a thread-block cluster until the grid fills the
// GPU.  At 4 bits a 4096 x 4096 weight is 8.9 MB, 1.3 us of HBM time: the call is bound by latency
// (launch, the first loads, the reduction), so every CTA has its share of the weight in flight
// before it waits for anything, and the split sums meet in shared memory.  (One token 4096 x 4096: 5.6 us;
// the 64 tokens of a decode batch with their adapters, with the kernel before it, 13.4.)  The block scales reach
// tensor memory through registers, by the warps that drain the accumulator later: copied there by
// tcgen05.cp from the MMA thread, a step of 256 along K took 580 ns whatever the batch.
//
// The LoRA term is more K blocks of the same accumulator, divided over the cluster's CTAs: for the
// batch's distinct adapters d, columns d * r_max + j hold B_d[o, j] on the feature side (TMA boxes
// of 128 rows x 8 columns, which land as the tensor cores take them) and s[t, j] on the token side
// (zero unless token t uses d), in two 16-bit parts that multiply the same B: one would add its own
// rounding to y's.  An adapter's B rows are thus read once per feature tile, however many tokens use
// it.  Infinities and NaNs in B are replaced by zeros in the block -- 0 * inf would reach every
// token -- and added afterwards to the tokens of that adapter alone, as is what of s a float16 cannot
// hold.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "fp4_device.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace lora {
namespace tc {

using namespace ptx;

constexpr int kDM = 128;         // features per tile
constexpr int kDThreads = 320;   // warp 0 loads, 1 MMAs, 2-5 scales, 2-9 LoRA blocks, 2-5 accumulator
constexpr uint32_t kDWBytes = kDM * 128;
constexpr int kDChunks = 4;      // 8-column chunks per LoRA block
constexpr int kDScratch = 64 * 4 + 64 * 4 + 3 * 256 * 4 + 1024;
constexpr int kDBars = 512;

struct Fp4DecodeArgs {
    const uint8_t* sx;
    const uint8_t* sw;
    void* y;
    int32_t* status;      // nullable
    long long ldy;
    int n, n_pad, h_out, kb_total, kb_per_split, splits, stages, tmem_cols, kt, early_w, early_x, vec, ring_bytes, push;
    // the LoRA term (fuse)
    int R, s_parts, bf16;
    const float* s_in;    // [s_parts][n][R]
    const int32_t* idx;
    const void* B;
};

// The token side of LoRA chunks p0 .. p0 + 3: for token t and chunk p, columns 8 c .. of its shrink
// output if chunk p is c of t's own adapter (index dl[t] among the batch's), else zeros; the four
// chunks' high parts, then their low ones.  U (token, chunk) items and K parts of the sum are loaded
// at once, whether they are wanted or not: a row's loads then wait for memory once.  Chunks with
// values that the parts leave out are marked in badmap.
template <typename T, int U, int K>
__device__ __forceinline__ void build_tokens(const Fp4DecodeArgs& a, uint8_t* S, uint32_t schunk, const int* dl, int p0,
                                             int chunks, int lt, uint32_t* badmap, volatile int* any_bad) {
    const size_t part = (size_t)a.n * a.R;
    for (int e0 = lt; e0 < a.n_pad * kDChunks; e0 += 256 * U) {
        float4 lo[U], hi[U];
        bool mine[U];
        const float* src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + 256 * u, t = min(e / kDChunks, a.n - 1);
            const int c = p0 + e % kDChunks - dl[t] * chunks;
            mine[u] = e / kDChunks < a.n && dl[t] >= 0 && c >= 0 && c < chunks;
            src[u] = a.s_in + (size_t)t * a.R + max(0, min(c, chunks - 1)) * 8;
            lo[u] = hi[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int k0 = 0; k0 < a.s_parts; k0 += K) {
            float4 c[U][K], d[U][K];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float4* p = reinterpret_cast<const float4*>(src[u] + min(k0 + k, a.s_parts - 1) * part);
                    c[u][k] = __ldcg(p);
                    d[u][k] = __ldcg(p + 1);
                }
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k0 + k < a.s_parts)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        lo[u].x += c[u][k].x, lo[u].y += c[u][k].y, lo[u].z += c[u][k].z, lo[u].w += c[u][k].w;
                        hi[u].x += d[u][k].x, hi[u].y += d[u][k].y, hi[u].z += d[u][k].z, hi[u].w += d[u][k].w;
                    }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + 256 * u;
            if (e >= a.n_pad * kDChunks) break;
            const float v[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
            uint4 h16 = make_uint4(0, 0, 0, 0), l16 = h16;
            const int p = p0 + e % kDChunks;
            if (mine[u] && split8<T>(v, h16, l16)) {
                atomicOr(&badmap[p >> 5], 1u << (p & 31));
                *any_bad = 1;
            }
            uint8_t* at = S + (e % kDChunks) * schunk + e / kDChunks * 16;
            *reinterpret_cast<uint4*>(at) = h16;
            *reinterpret_cast<uint4*>(at + kDChunks * schunk) = l16;
        }
    }
}

// FUSE: with the LoRA term.  Without it the kernel is a third as long.
template <typename T, bool FUSE>
__global__ void __launch_bounds__(kDThreads, 1)
fp4_decode_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmB, const Fp4DecodeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const int stages = a.stages, n = a.n, n_pad = a.n_pad;
    const bool xt2 = n_pad > 128;  // a second scale tile of x
    const uint32_t x_bytes = static_cast<uint32_t>(n_pad) * 128;
    const uint32_t stage_bytes = kDWBytes + x_bytes;
    const uint32_t schunk = static_cast<uint32_t>(n_pad) * 16;                 // token side of a chunk
    const uint32_t lora_bytes = FUSE ? kDChunks * (2048 + 2 * schunk) : 0;
    uint8_t* lora_sm = smem + (size_t)stages * stage_bytes;                    // [2] {features, tokens' high parts, low parts}
    uint32_t* seen = reinterpret_cast<uint32_t*>(smem + a.ring_bytes);         // [64]
    int* before = reinterpret_cast<int*>(seen + 64);                           // [64]
    int* dlist = before + 64;                                                  // [256]
    int* slot_sm = dlist + 256;                                                // [256] slot of each token
    int* dl_sm = slot_sm + 256;                                                // [256] its index among the batch's
    uint32_t* badmap = reinterpret_cast<uint32_t*>(dl_sm + 256);               // [256]
    uint64_t* full = reinterpret_cast<uint64_t*>(badmap + 256);
    uint64_t* empty = full + stages;
    uint64_t* acc_full = empty + stages;
    uint64_t* lora_tma = acc_full + 1;    // [2] feature side landed
    uint64_t* lora_full = lora_tma + 2;   // [2] block complete (8 warps)
    uint64_t* lora_empty = lora_full + 2; // [2]
    uint64_t* linfo = lora_empty + 2;     // number of LoRA blocks known
    uint64_t* lora_done = linfo + 1;      // slots, bad chunks: complete (8 warps)
    uint64_t* rbar = lora_done + 1;       // the other CTAs' sums of this CTA's tokens have arrived
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rbar + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);  // abort, LoRA blocks, any bad chunk
    float* P = reinterpret_cast<float*>(smem);  // after the main loop: [n_pad][128] (partial) sums

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m_tile = blockIdx.x, split = blockIdx.y;
    const int kb0 = split * a.kb_per_split;
    const int nkb = min(a.kb_total, kb0 + a.kb_per_split) - kb0;
    T* y = static_cast<T*>(a.y);

    auto issue_w = [&](int i) {
        const int s = i % stages;
        uint8_t* st = smem + (size_t)s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        tma_load_2d_cta(st, &tmW, &full[s], (kb0 + i) * 128, m_tile * kDM);
    };
    auto issue_x = [&](int i) {
        const int s = i % stages;
        tma_load_2d_cta(smem + (size_t)s * stage_bytes + kDWBytes, &tmX, &full[s], (kb0 + i) * 128, 0);
    };
    const int pre = min(stages, nkb);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 5);  // the loads and the four scale warps
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&lora_tma[b], 1);
            mbar_init(&lora_full[b], 8);
            mbar_init(&lora_empty[b], 1);
        }
        mbar_init(linfo, 1);
        mbar_init(lora_done, 8);
        mbar_init(rbar, 1);
        flags[0] = flags[1] = flags[2] = 0;
        fence_barrier_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        // what is complete when this grid starts, behind a kernel that waited for its writers, is
        // loaded at once: the weight, or also x where it was stored before that kernel
        if (a.early_w)
            for (int i = 0; i < pre; ++i) {
                issue_w(i);
                if (a.early_x) issue_x(i);
            }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, a.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a product by itself releases nothing early: its y may be a weight that a 16-bit linear streams unwaited
    if (a.early_w) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            if (a.early_w) {
                if (!a.early_x) {
                    pdl_wait();
                    for (int i = 0; i < pre; ++i) issue_x(i);
                }
                issued = pre;
            } else {
                pdl_wait();
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
                    const unsigned long long t0 = globaltimer();
                    while (!mbar_try_wait(&full[i % stages], (i / stages) & 1) && globaltimer() - t0 < kWaitLimitNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            const uint32_t id0 = idesc_mxf4(kDM, n_pad, 0), id2 = idesc_mxf4(kDM, n_pad, 2);
            for (int i = 0; i < nkb; ++i) {
                const int s = i % stages;
                if (!mbar_wait(&full[s], (i / stages) & 1, flags)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t wa = smem_u32(smem + (size_t)s * stage_bytes), xa = wa + kDWBytes;
                // each stage has its own scale columns: w's two tiles (4 each), x's two (8 each)
                const uint32_t sfw = tmem + static_cast<uint32_t>(n_pad + s * 24), sfx = sfw + 8;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_mxf4(tmem, sdesc_sw128(wa + k * 32), sdesc_sw128(xa + k * 32), (k & 1) ? id2 : id0,
                              sfw + 4 * (k >> 1), sfx + 8 * (k >> 1), (i > 0 || k > 0) ? 1u : 0u);
                umma_commit(&empty[s]);
            }
            if (FUSE && ok) {
                ok = mbar_wait(linfo, 0, flags);
                const int blocks = ok ? flags[1] : 0;
                const uint32_t idesc_lora = idesc_f16(kDM, n_pad, a.bf16 != 0);
                for (int b = 0; b < blocks; ++b) {
                    const int lbuf = b & 1;
                    if (!mbar_wait(&lora_full[lbuf], (b >> 1) & 1, flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ba = smem_u32(lora_sm + lbuf * lora_bytes), sa = ba + kDChunks * 2048;
#pragma unroll
                    for (int k = 0; k < kDChunks; ++k)  // the high parts' two steps, then the low parts'
                        umma_f16(tmem, sdesc_chunks(ba + (k & 1) * 2 * 2048, 2048), sdesc_chunks(sa + 2 * k * schunk, schunk),
                                 idesc_lora, 1u);
                    umma_commit(&lora_empty[lbuf]);
                }
            }
            if (!ok && a.status) report_timeout_status(a.status);
            umma_commit(acc_full);  // also on abort: fires once the issued MMAs have finished
        }
    }

    if (warp >= 2 && warp < 6) {
        // ---- scales: each warp fills its 32 lanes (the four hold the same), four steps' loads ahead ----
        if (!a.early_w) pdl_wait();
        const uint32_t taddr = tmem + static_cast<uint32_t>(n_pad) + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint4* pw = reinterpret_cast<const uint4*>(a.sw + ((size_t)m_tile * a.kt + 2 * kb0) * 512) + lane;
        const uint4* px = reinterpret_cast<const uint4*>(a.sx + (size_t)(2 * kb0) * 512) + lane;
        const uint4* px2 = px + (size_t)a.kt * 32;
        constexpr int kAhead = 4;
        uint4 v[kAhead][6];
        auto load_w = [&](int i, uint4 (&u)[6]) {
            if (i >= nkb) return;
            u[0] = __ldg(pw + i * 64);
            u[1] = __ldg(pw + i * 64 + 32);
        };
        auto load_x = [&](int i, uint4 (&u)[6]) {
            if (i >= nkb) return;
            u[2] = __ldcg(px + i * 64);
            u[3] = __ldcg(px + i * 64 + 32);
            if (xt2) {
                u[4] = __ldcg(px2 + i * 64);
                u[5] = __ldcg(px2 + i * 64 + 32);
            }
        };
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
#pragma unroll
            for (int e = 0; e < 6; ++e) v[h][e] = make_uint4(0, 0, 0, 0);
            load_w(h, v[h]);
        }
        if (a.early_w && !a.early_x) pdl_wait();
#pragma unroll
        for (int h = 0; h < kAhead; ++h) load_x(h, v[h]);
        // the first stages' columns have no earlier readers: one wait for all their stores
        auto put = [&](int s, const uint4 (&u)[6]) {
            const uint32_t t = taddr + static_cast<uint32_t>(s * 24);
            tmem_st8(t, u[0], u[1]);
            tmem_st8(t + 8, u[2], u[4]);
            tmem_st8(t + 16, u[3], u[5]);
        };
        const int first = min(kAhead, min(stages, nkb));
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
            if (h < first) put(h, v[h]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            for (int h = 0; h < first; ++h) mbar_arrive(&full[h]);
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
            if (h < first) {
                load_w(kAhead + h, v[h]);
                load_x(kAhead + h, v[h]);
            }
        for (int i0 = 0; i0 < nkb; i0 += kAhead) {
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                const int i = i0 + h, s = i % stages;
                if (i < first || i >= nkb) continue;
                // the columns' last readers
                if (i >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((i / stages) & 1) ^ 1, flags)))
                    continue;  // aborted: the other waits end the same way
                tc_fence_after();
                put(s, v[h]);
                load_w(i + kAhead, v[h]);
                load_x(i + kAhead, v[h]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
        }
    }

    if constexpr (FUSE) {
        // ---- LoRA blocks: this CTA's share of the batch's (adapter, 8 columns) chunks ----
        if (warp >= 2) {
            const int chunks = a.R / 8;
            auto issue_b = [&](int b, int P_all) {  // the feature side of this CTA's block b
                const int p0 = (split + b * a.splits) * kDChunks, cnt = min(kDChunks, P_all - p0);
                uint64_t* bar = &lora_tma[b & 1];
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(cnt) * 2048);
                for (int j = 0; j < cnt; ++j) {
                    const int d = (p0 + j) / chunks, c = (p0 + j) - d * chunks;
                    tma_load_3d_cta(lora_sm + (b & 1) * lora_bytes + j * 2048, &tmB, bar, 0, c,
                                    dlist[d] * a.h_out + m_tile * kDM);
                }
            };
            if (warp >= 6) {
                // the batch's adapters, while the scale warps and the kernel ahead are at work (the
                // segments are older than that kernel)
                const int lt = threadIdx.x - 192;
                const bool st_ok = __ldcg(a.status) == LORA_OK;
                if (lt < 64) seen[lt] = 0;
                int slot[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = lt + 128 * h;
                    slot[h] = st_ok && t < n ? __ldcg(a.idx + t) : -1;
                    slot_sm[t] = slot[h];
                    badmap[t] = 0;
                }
                named_bar_sync(2, 128);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (slot[h] >= 0) atomicOr(&seen[slot[h] >> 5], 1u << (slot[h] & 31));
                named_bar_sync(2, 128);
                if (lt < 32) {  // words 2 lt and 2 lt + 1
                    const uint32_t w0 = seen[2 * lt], w1 = seen[2 * lt + 1];
                    int v = __popc(w0) + __popc(w1);
                    const int own = v;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, v, d);
                        if (lt >= d) v += o;
                    }
                    int at = v - own;
                    before[2 * lt] = at;
                    for (uint32_t m = w0; m; m &= m - 1) dlist[at++] = 2 * lt * 32 + __ffs(m) - 1;
                    before[2 * lt + 1] = at;
                    for (uint32_t m = w1; m; m &= m - 1) dlist[at++] = (2 * lt + 1) * 32 + __ffs(m) - 1;
                }
                named_bar_sync(2, 128);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    dl_sm[lt + 128 * h] =
                        slot[h] < 0 ? -1 : before[slot[h] >> 5] + __popc(seen[slot[h] >> 5] & ((1u << (slot[h] & 31)) - 1u));
            }
            const int lt = threadIdx.x - 64;  // 0..255
            auto count_blocks = [&](int P_all) {
                const int all = (P_all + kDChunks - 1) / kDChunks;
                return all > split ? (all - split - 1) / a.splits + 1 : 0;
            };
            if (threadIdx.x == 192) {
                const int P_all = (before[63] + __popc(seen[63])) * chunks, blocks = count_blocks(P_all);
                flags[1] = blocks;
                mbar_arrive(linfo);
                for (int b = 0; b < min(blocks, 2); ++b) issue_b(b, P_all);
            }
            named_bar_sync(3, 256);  // the scale warps join
            const int P_all = (before[63] + __popc(seen[63])) * chunks, blocks = count_blocks(P_all);
            pdl_wait();  // s
            bool ok = true;
            for (int b = 0; b < blocks; ++b) {
                const int lbuf = b & 1, p0 = (split + b * a.splits) * kDChunks;
                uint8_t* blk = lora_sm + lbuf * lora_bytes;
                if (b >= 2) {
                    // the block two before is consumed; its feature side may be overwritten
                    ok = __all_sync(0xffffffffu, mbar_wait(&lora_empty[lbuf], ((b >> 1) & 1) ^ 1, flags));
                    if (ok && threadIdx.x == 192) issue_b(b, P_all);
                }
                // token side: 32 bytes a token and chunk; several parts of one, or one part of several, at once
                if (ok) {
                    uint8_t* S = blk + kDChunks * 2048;
                    if (a.s_parts > 1)
                        build_tokens<T, 2, 4>(a, S, schunk, dl_sm, p0, chunks, lt, badmap, &flags[2]);
                    else
                        build_tokens<T, 4, 1>(a, S, schunk, dl_sm, p0, chunks, lt, badmap, &flags[2]);
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&lora_tma[lbuf], (b >> 1) & 1, flags));
                if (!ok) break;
#pragma unroll
                for (int jj = 0; jj < kDChunks / 2; ++jj) {
                    const int j = 2 * jj + (lt >> 7);
                    uint4* bp = reinterpret_cast<uint4*>(blk + j * 2048 + (lt & 127) * 16);
                    if (p0 + j >= P_all) {
                        *bp = make_uint4(0, 0, 0, 0);
                    } else {
                        const uint4 v = *bp;
                        if (nonfinite8<T>(v)) {
                            *bp = finite8<T>(v);
                            atomicOr(&badmap[(p0 + j) >> 5], 1u << ((p0 + j) & 31));
                            flags[2] = 1;
                        }
                    }
                }
                fence_proxy_async_smem();  // read by the tensor cores
                __syncwarp();
                if (lane == 0) mbar_arrive(&lora_full[lbuf]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(lora_done);
            if (!ok) {
                if (a.status) report_timeout_status(a.status);
                // boxes in flight land before the CTA leaves
                if (threadIdx.x == 192)
                    for (int b = 0; b < 2; ++b) {
                        const unsigned long long t0 = globaltimer();
                        while (!mbar_try_wait(&lora_tma[b], 0) && globaltimer() - t0 < kWaitLimitNs) {
                        }
                    }
            }
        }
    }

    bool store = false;
    if (warp >= 2) {
        pdl_wait();
        store = !a.status || __ldcg(a.status) == LORA_OK;
    }
    if (warp >= 2 && warp < 6) {
        const int row = (warp & 3) * 32 + lane, o = m_tile * kDM + row;
        const bool got = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, flags) && (!FUSE || mbar_wait(lora_done, 0, flags)));
        if (got) {
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            for (int c0 = 0; c0 < n_pad; c0 += 64) {  // one wait per 64 columns
                uint32_t r[64];
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c0 + 16 * q < n_pad) tmem_ld16(taddr + c0 + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&r[16 * q]));
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c0 + 16 * q < n_pad)
#pragma unroll
                        for (int c = 16 * q; c < 16 * q + 16; ++c) P[(c0 + c) * kDM + row] = __uint_as_float(r[c]);
            }
            if constexpr (FUSE) {
                if (flags[2] && o < a.h_out) {  // products left out of the blocks
                    const int chunks = a.R / 8;
                    for (int t = 0; t < n; ++t) {
                        if (dl_sm[t] < 0) continue;
                        for (int k8 = 0; k8 < chunks; ++k8) {
                            const int p = dl_sm[t] * chunks + k8;
                            if (!((badmap[p >> 5] >> (p & 31)) & 1u)) continue;
                            float sv[8];
                            sum_parts8(a.s_in + (size_t)t * a.R + k8 * 8, a.s_parts, (size_t)n * a.R, sv);
                            const uint4 bv = __ldg(reinterpret_cast<const uint4*>(
                                static_cast<const T*>(a.B) + ((size_t)slot_sm[t] * a.h_out + o) * a.R + k8 * 8));
                            P[t * kDM + row] = nonfinite_dot8<T>(bv, sv, P[t * kDM + row]);
                        }
                    }
                }
            }
            fence_proxy_async_smem();  // read by the bulk copies
        } else if (lane == 0) {
            flags[0] = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    // Each CTA adds up the partial sums of its share of the tokens, in split order, and stores them:
    // 8 features a thread, 16 neighbouring threads a token's 128.  The sums reach their owner by one
    // bulk copy from each other CTA (a token's row is 512 bytes, an owner's rows are contiguous) where a
    // receive buffer fits, else they are read remotely, which is slower (64 tokens, 4 CTAs: 1.9 us).
    bool good = flags[0] == 0;
    const int per = (n + a.splits - 1) / a.splits;
    const int t0 = min(n, split * per), cnt = min(n, t0 + per) - t0;
    float* rcv = P + (size_t)n_pad * kDM;  // [splits - 1][per][128]
    bool recv = true;
    if (a.splits > 1) {
        if (a.push && threadIdx.x == 64 && cnt > 0)
            mbar_arrive_expect_tx(rbar, static_cast<uint32_t>((a.splits - 1) * cnt * kDM * 4));
        cluster_sync();
        if (a.push) {
            const int dst = (int)threadIdx.x - 64;
            if (dst >= 0 && dst < a.splits && dst != split) {
                const int d0 = min(n, dst * per), dcnt = min(n, d0 + per) - d0;
                if (dcnt > 0)
                    bulk_s2cluster(mapa_shared(smem_u32(rcv + (size_t)(split < dst ? split : split - 1) * per * kDM),
                                               static_cast<uint32_t>(dst)),
                                   P + (size_t)d0 * kDM, static_cast<uint32_t>(dcnt * kDM * 4),
                                   mapa_shared(smem_u32(rbar), static_cast<uint32_t>(dst)));
            }
            __syncwarp();
            good = cluster_unaborted(flags, a.splits);  // sums of a CTA that gave up are no one's; read while the copies fly
            if (cnt > 0) recv = __all_sync(0xffffffffu, mbar_wait(rbar, 0, flags));
            cluster_arrive();  // (the last wait below: every copy out of this CTA has then landed)
        } else {
            good = cluster_unaborted(flags, a.splits);
        }
    }
    if (warp >= 2 && good && store && recv) {
        auto store8 = [&](int t, int o, const float (&v)[8]) {
            T* yp = y + (long long)t * a.ldy + o;
            alignas(16) T w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = from_f32<T>(v[i]);
            if (o + 8 <= a.h_out) {
#pragma unroll
                for (int i = 0; i < (int)(8 * sizeof(T) / 16); ++i)
                    reinterpret_cast<uint4*>(yp)[i] = reinterpret_cast<const uint4*>(w)[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (o + i < a.h_out) yp[i] = w[i];
            }
        };
        const int o8 = ((int)threadIdx.x & 15) * 8, o = m_tile * kDM + o8;
        if (!a.vec) {
            // rows off 16-byte boundaries: a feature a thread, neighbours side by side, eight tokens' sums at
            // once (204 x 105 x 2507 in float32: 20.5 us one token after the other, 12.4 so)
            const int f = (int)threadIdx.x & 127, of = m_tile * kDM + f;
            for (int u0 = ((int)threadIdx.x - 64) >> 7; u0 < cnt; u0 += 16) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = 0.f;
                for (int c = 0; c < a.splits; ++c)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int u = min(u0 + 2 * k, cnt - 1);
                        const float* own = P + (t0 + u) * kDM + f;
                        if (a.splits == 1 || (a.push && c == split))
                            v[k] += *own;
                        else if (a.push)
                            v[k] += rcv[((size_t)(c < split ? c : c - 1) * per + u) * kDM + f];
                        else
                            v[k] += ld_dsmem_f32(mapa_shared(smem_u32(own), static_cast<uint32_t>(c)));
                    }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (u0 + 2 * k < cnt && of < a.h_out) y[(long long)(t0 + u0 + 2 * k) * a.ldy + of] = from_f32<T>(v[k]);
            }
        } else if (a.splits == 1) {
            for (int t = ((int)threadIdx.x - 64) >> 4; t < n; t += 16) {
                const float4* own = reinterpret_cast<const float4*>(P + t * kDM + o8);
                const float4 lo = own[0], hi = own[1];
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                store8(t, o, v);
            }
        } else {
            for (int u = ((int)threadIdx.x - 64) >> 4; u < cnt; u += 16) {
                const float* own = P + (t0 + u) * kDM + o8;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
                for (int c0 = 0; c0 < a.splits; c0 += 4) {  // four CTAs' loads in flight
                    float4 lo[4], hi[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = min(c0 + k, a.splits - 1);
                        if (a.push) {
                            const float* p = c == split ? own : rcv + ((size_t)(c < split ? c : c - 1) * per + u) * kDM + o8;
                            lo[k] = reinterpret_cast<const float4*>(p)[0];
                            hi[k] = reinterpret_cast<const float4*>(p)[1];
                        } else {
                            const uint32_t at = mapa_shared(smem_u32(own), static_cast<uint32_t>(c));
                            lo[k] = ld_dsmem_f32x4(at);
                            hi[k] = ld_dsmem_f32x4(at + 16);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c0 + k < a.splits) {
                            v[0] += lo[k].x, v[1] += lo[k].y, v[2] += lo[k].z, v[3] += lo[k].w;
                            v[4] += hi[k].x, v[5] += hi[k].y, v[6] += hi[k].z, v[7] += hi[k].w;
                        }
                }
                store8(t0 + u, o, v);
            }
        }
    }
    if (!recv && a.status) report_timeout_status(a.status);
    // no CTA leaves while its partial sums may still be read or copied
    if (a.splits > 1) {
        if (!a.push) cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, a.tmem_cols);
}

template <typename T, bool FUSE>
static int launch_fp4_decode_t(const Fp4View& x, const Fp4View& w, void* y, long long ldy, int32_t* status, int early,
                               const Fp4DecodeLora* lora, cudaStream_t st) {
    Fp4DecodeArgs a;
    memset(&a, 0, sizeof(a));
    a.sx = x.scales;
    a.sw = w.scales;
    a.y = y;
    a.status = status;
    a.ldy = ldy;
    a.n = x.rows;
    a.n_pad = (x.rows + 15) / 16 * 16;
    a.h_out = w.rows;
    a.kt = x.ktiles;
    a.kb_total = x.ktiles / 2;
    a.early_w = early >= 1;
    a.early_x = early >= 2;
    // y is written 16 bytes at a time when every row starts on a 16-byte boundary
    a.vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (long long)sizeof(T)) % 16 == 0;
    const int m_tiles = (w.rows + kDM - 1) / kDM;
    a.splits = fp4_decode_splits(w.rows, w.cols);
    a.kb_per_split = (a.kb_total + a.splits - 1) / a.splits;
    PoolView pv;
    if (lora) {
        pv = *lora->pool;
        a.R = pv.R;
        a.s_parts = lora->s_parts;
        a.bf16 = pv.dtype == LORA_BF16;
        a.s_in = lora->s_in;
        a.idx = lora->idx;
        a.B = pv.B;
    }
    const size_t stage_bytes = kDWBytes + (size_t)a.n_pad * 128;
    const size_t lora_bytes = lora ? 2 * (size_t)kDChunks * (2048 + 2 * a.n_pad * 16) : 0;
    const size_t room = 227 * 1024 - kDScratch - kDBars - 1024;
    int stages = (int)((room - lora_bytes) / stage_bytes);
    stages = std::min({stages, 8, a.kb_per_split});
    a.stages = stages;
    // the stages and LoRA blocks are idle when the sums are parked in their place
    const int per = (x.rows + a.splits - 1) / a.splits;
    const size_t park = (size_t)a.n_pad * kDM * 4, rcv = (size_t)(a.splits - 1) * per * kDM * 4;
    a.push = a.splits > 1 && park + rcv <= room;
    a.ring_bytes = (int)((std::max(stages * stage_bytes + lora_bytes, park + (a.push ? rcv : 0)) + 1023) / 1024 * 1024);
    int cols = 32;
    while (cols < a.n_pad + 24 * stages) cols <<= 1;
    a.tmem_cols = cols;
    const size_t smem = (size_t)a.ring_bytes + kDScratch + kDBars + 1024;
    if (smem > 227 * 1024 || cols > 512) return set_error(LORA_EUNSUP, "internal: 4-bit decode plan");
    CUtensorMap mX, mW, mB;
    int rc = make_map_fp4(&mX, x.codes, x.pitch, x.rows, a.n_pad);
    if (!rc) rc = make_map_fp4(&mW, w.codes, w.pitch, w.rows, kDM);
    if (!rc && lora) rc = make_map_bchunks(&mB, pv.B, a.bf16, pv.R, (uint64_t)pv.S * pv.h_out);
    if (rc) return rc;
    if (!lora) mB = mW;  // not used
    static bool attr_set = false;
    if (!attr_set) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(fp4_decode_kernel<T, FUSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
        attr_set = true;
    }
    void* args[] = {(void*)&mW, (void*)&mX, (void*)&mB, (void*)&a};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(m_tiles, a.splits);
    cfg.blockDim = dim3(kDThreads);
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
    LORA_CUDA_TRY(cudaLaunchKernelExC(&cfg, (const void*)fp4_decode_kernel<T, FUSE>, args));
    count_launch();
    return LORA_OK;
}

}  // namespace tc

// CTAs (a cluster) that share K: as many as let every feature tile have an SM a CTA.
int fp4_decode_splits(int h_out, int h_in) {
    const int m_tiles = (h_out + tc::kDM - 1) / tc::kDM, steps = (h_in + 255) / 256;
    const int splits = std::min({std::max(1, num_sms() / m_tiles), 8, steps}), per = (steps + splits - 1) / splits;
    return (steps + per - 1) / per;
}

int launch_fp4_decode(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status,
                      int early, const Fp4DecodeLora* lora, cudaStream_t st) {
    if (lora && dtype == LORA_F16)
        return tc::launch_fp4_decode_t<__half, true>(x, w, y, ldy, status, early, lora, st);
    if (lora) return tc::launch_fp4_decode_t<__nv_bfloat16, true>(x, w, y, ldy, status, early, lora, st);
    switch (dtype) {
        case LORA_F32: return tc::launch_fp4_decode_t<float, false>(x, w, y, ldy, status, early, nullptr, st);
        case LORA_F16: return tc::launch_fp4_decode_t<__half, false>(x, w, y, ldy, status, early, nullptr, st);
        default: return tc::launch_fp4_decode_t<__nv_bfloat16, false>(x, w, y, ldy, status, early, nullptr, st);
    }
}

}  // namespace lora
