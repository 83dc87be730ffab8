// Products over an 8-bit weight on the tensor cores, whole-number sums kept exact.
//
// sm_103a's tensor cores take no 8-bit integers, but a code is a float16 number and a product of two codes
// is exact in float32, so is a sum of 1024 of them (1024 * 128 * 128 = 2^24), or of more where the tokens' codes
// are small: the kernel before this one leaves each token's largest sum of |code| over 256, which bounds the
// partial sums.  Codes go through tcgen05.mma kind::f16; every chunk of so many the accumulator is read into
// 32-bit integers and started again (normal data: 24 to 26 steps of 128 codes; with a few loud channels, as activations
// have them, some hundred).
//
// The weight is the MMA's M side (128 features a tile) and up to 256 tokens its N side.  The weight stays
// in bytes until it is on the SM: TMA brings 128 x 128 codes, sixteen warps turn them into float16 and store
// them to tensor memory as the MMA's A operand (tcgen05.st), so float16 weights never pass through shared
// memory.  A warp's turn (waits, loads, conversion, store) takes about 900 clocks for 32 features x 64 codes,
// a step of 128 codes from HBM 700: eight warps would not keep up.
//
// K is split over the CTAs of a thread-block cluster until the grid fills the GPU; each CTA finishes a share of
// the tokens, into whose shared memory the others store their sums (integers: any order gives the same).
//
// The LoRA term is added there in float32: y[t, o] = sx sw sum + s[t, :] . B[o, :].  Eight more warps compute it
// during the main loop for the tokens their CTA will finish.  Tokens come in the order of the segments, so
// neighbouring tokens share their adapter's rows of B.
//
// Measured (launches in a graph, the kernel that makes x's codes included): 16, 64, 256, 512 tokens 4096 x 4096 float16
// 10.5, 11.2, 17.9, 24.2 us; 256 x 4096 x 11008 32, of which the MMAs take 17: 86 tiles leave 66 of 152 SMs idle, and a
// split of K would need 172.  With adapters, 64 tokens over 100 of rank 8 14.6; of rank 64 30 (without their B 18); 200
// tokens 11008 x 4096 over 6 of rank 64 50, of which the shrink before it 12.  Small batches are a chain of latencies: the
// kernel ahead, its x through TMA, eight steps, the sums' way through the cluster.
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
constexpr int kIN = 256;          // tokens per tile, at most
constexpr int kIK = 128;          // codes of a step along K
constexpr int kIChunk = 8;        // steps between two readings of the accumulator, at least: 1024 codes
constexpr int kIWorkers = 16;     // warps 2-17: convert (half of them the even steps, half the odd), drain
constexpr int kIThreads = 64 + 32 * kIWorkers;  // warp 0 loads, 1 MMAs
constexpr int kILora = 256;       // more threads for the LoRA term
constexpr int kIASlots = 4;       // steps of the weight in tensor memory, 64 columns each
constexpr int kIACol = 256;       // behind two accumulators of up to 128 tokens, or one of more
constexpr int kIMostS = 64;       // columns of the shrink output staged at once, at most
constexpr uint32_t kIWBytes = kIM * kIK;
constexpr int kIBars = 384;
constexpr size_t kISmemMax = 227 * 1024;

struct I8TileArgs {
    void* y;
    int32_t* status;       // nullable
    const int32_t* perm;   // row of y of each row of x (nullable)
    const float* sx;
    const int* peak;
    const float* sw;
    long long ldy;
    int n, n_pad, h_out, kb_total, kb_per_split, splits, wstages, xstages, xk, early_x, release, vec, ring_bytes, alias, per, per_inv;
    // the LoRA term (FUSE)
    const SlotEntry* table;
    const void* B;
    const int32_t* idx;    // by token
    const float* s_in;     // [s_parts][n][R], by token
    int R, s_parts, s_cols;
};

// Eight columns of a row of B as they are in memory; zeros past `left`.
template <typename T> struct BRow {
    uint4 v;  // (16-bit pools: rows of B are whole 16-byte pieces)
    __device__ __forceinline__ void load(const T* p, int left) {
        v = left > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { unpack8<T>(v, f); }
};
template <> struct BRow<float> {
    float v[8];
    __device__ __forceinline__ void load(const float* p, int left) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? __ldg(p + e) : 0.f;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
    }
};

template <typename T, bool FUSE>
__global__ void __launch_bounds__(kIThreads + (FUSE ? kILora : 0), 1)
i8_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8TileArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    // stages of the weight's codes, which the warps that convert them free, and of the tokens', which the MMAs free
    const int ws = a.wstages, xs = a.xstages, n_pad = a.n_pad;
    const uint32_t x_bytes = static_cast<uint32_t>(n_pad) * 128 * a.xk;  // xk (1 or 2) boxes of 64 float16 columns
    uint8_t* xring = smem + ws * kIWBytes;
    // sums of the tokens this CTA finishes, from each CTA of the cluster [splits][per][128]; with alias in the ring,
    // once that is idle
    int* G = reinterpret_cast<int*>(smem + (a.alias ? 0 : a.ring_bytes));
    float* L = reinterpret_cast<float*>(smem + a.ring_bytes) + (a.alias ? 0 : a.splits * a.per * kIM);  // FUSE: [per][128] their LoRA terms
    float* S = L + (FUSE ? a.per * kIM : 0);                      // FUSE: [per][s_cols] shrink output
    int* tok_slot = reinterpret_cast<int*>(S + (FUSE ? a.per * a.s_cols : 0));  // FUSE: [per] slots of the CTA's tokens,
    int* tok_rank = tok_slot + (FUSE ? a.per : 0);               // FUSE: [per] and their ranks,
    int* row_sm = tok_rank + (FUSE ? a.per : 0);                 // [per] their rows of y,
    float* sx_sm = reinterpret_cast<float*>(row_sm + a.per);     // [per] and scales
    float* sw_sm = sx_sm + a.per;                                // [128]
    uint64_t* full_w = reinterpret_cast<uint64_t*>(smem_align(reinterpret_cast<uint8_t*>(sw_sm + kIM), 8));  // [8]
    uint64_t* empty_w = full_w + 8;           // [8] (8 of the warps)
    uint64_t* full_x = empty_w + 8;           // [4]
    uint64_t* empty_x = full_x + 4;           // [4]
    uint64_t* conv = empty_x + 4;             // [kIASlots] the step's weight is in tensor memory (8 of the warps)
    uint64_t* a_free = conv + kIASlots;       // [kIASlots] the slot's MMAs have completed
    uint64_t* acc_full = a_free + kIASlots;   // [2]
    uint64_t* acc_empty = acc_full + 2;       // [2] (16 warps)
    uint64_t* drained = acc_empty + 2;        // (after an abort) every MMA has completed
    uint64_t* cut = drained + 1;              // flags[2] is known
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cut + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);  // abort; a CTA of the cluster has aborted; steps a chunk

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m_tile = blockIdx.x, split = blockIdx.y, row0 = blockIdx.z * a.n_pad;
    const int n = min(a.n - row0, a.n_pad);
    const int kb0 = split * a.kb_per_split;
    const int nkb = min(a.kb_total, kb0 + a.kb_per_split) - kb0;
    // the tokens this CTA finishes
    const int t0 = min(n, split * a.per), cnt = min(n, t0 + a.per) - t0;

    // Each feature tile starts at another place along K (sums of whole numbers come in any order): together, the
    // CTAs would all read the same few lines of x at a time.
    const int rot = m_tile % nkb;
    auto column = [&](int i) {  // of step i
        const int k = i + rot;
        return (kb0 + (k < nkb ? k : k - nkb)) * kIK;
    };
    auto issue_w = [&](int i, int st) {
        mbar_arrive_expect_tx(&full_w[st], kIWBytes);
        tma_load_2d_cta(smem + st * kIWBytes, &tmW, &full_w[st], column(i), m_tile * kIM);
    };
    auto issue_x = [&](int i, int st) {
        uint8_t* dst = xring + st * x_bytes;
        mbar_arrive_expect_tx(&full_x[st], x_bytes);
        if (a.xk == 2) {
            tma_load_2d_cta(dst, &tmX, &full_x[st], column(i), row0);
            tma_load_2d_cta(dst + n_pad * 128, &tmX, &full_x[st], column(i) + 64, row0);
        } else {
            tma_load_2d_cta(dst, &tmX, &full_x[st], column(i >> 1) + (i & 1) * 64, row0);
        }
    };
    const int nkx = nkb * (3 - a.xk);  // the tokens' stages, 64 or 128 codes each
    const int pre_w = min(ws, nkb), pre_x = min(xs, nkx);
    const int nbuf = n_pad <= 128 ? 2 : 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ws; ++i) {
            mbar_init(&full_w[i], 1);
            mbar_init(&empty_w[i], 8);
        }
        for (int i = 0; i < xs; ++i) {
            mbar_init(&full_x[i], 1);
            mbar_init(&empty_x[i], 1);
        }
        for (int i = 0; i < kIASlots; ++i) {
            mbar_init(&conv[i], 8);
            mbar_init(&a_free[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kIWorkers);
        }
        mbar_init(drained, 1);
        mbar_init(cut, 1);
        flags[0] = flags[1] = 0;
        fence_barrier_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        // what is complete when this grid starts is loaded at once: the weight, or also x
        for (int i = 0; i < pre_w; ++i) issue_w(i, i);
        if (a.early_x)
            for (int i = 0; i < pre_x; ++i) issue_x(i, i);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (a.splits > 1 && !a.alias) cluster_arrive();  // (waited for before the first store into another CTA)
    if (a.release) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            if (!a.early_x) {
                pdl_wait();
                for (int i = 0; i < pre_x; ++i) issue_x(i, i);
            }
            // whichever of the two has a stage free next
            int iw = pre_w, ix = pre_x, sw = 0, sx = 0;
            uint32_t phw = 0, phx = 0;
            unsigned long long since = globaltimer();
            int last = iw + ix;
            for (uint32_t spin = 1; (iw < nkb || ix < nkx) && !flags[0]; ++spin) {
                if (iw < nkb && mbar_test(&empty_w[sw], phw)) {
                    issue_w(iw++, sw);
                    if (++sw == ws) sw = 0, phw ^= 1;
                }
                if (ix < nkx && mbar_test(&empty_x[sx], phx)) {
                    issue_x(ix++, sx);
                    if (++sx == xs) sx = 0, phx ^= 1;
                }
                if ((spin & 1023u) == 0) {
                    if (iw + ix != last) {
                        last = iw + ix;
                        since = globaltimer();
                    } else if (globaltimer() - since > kWaitLimitNs) {
                        flags[0] = 1;
                    }
                }
            }
            if (flags[0]) {  // give the copies in flight time to land
                if (a.status) report_timeout_status(a.status);
                const unsigned long long t = globaltimer();
                while (globaltimer() - t < kWaitLimitNs / 8) {
                }
            }
        }
        __syncwarp();
        // what the stores will need
        pdl_wait();
        const bool st_ok = !a.status || __ldcg(a.status) == LORA_OK;
        for (int e = lane; e < kIM; e += 32) sw_sm[e] = m_tile * kIM + e < a.h_out ? __ldg(a.sw + m_tile * kIM + e) : 0.f;
        for (int u = lane; u < cnt; u += 32) {
            const int r = row0 + t0 + u;
            sx_sm[u] = __ldcg(a.sx + r);
            if (!FUSE) row_sm[u] = a.perm && st_ok ? __ldcg(a.perm + r) : r;
        }
    } else if (warp == 1) {
        bool ok = true;
        const uint32_t idesc = idesc_f16(kIM, n_pad, false);
        // Steps a chunk: blocks of 256 codes whose products with 128 stay below 2^24 (two blocks less for those that
        // a chunk has a part of).  An accumulator of more than 128 tokens has no second one beside it, and reading
        // it holds the MMAs up: 200 x 11008 x 4096, chunks of 1024 codes 41 us, as long as the codes let them 33.
        int chunk_steps = kIChunk;
        if (nkb > kIChunk) {
            if (!a.early_x) pdl_wait();
            int top = 1;
            for (int t = lane; t < n; t += 32) top = max(top, __ldcg(a.peak + row0 + t));
            top = __reduce_max_sync(0xffffffffu, top);
            chunk_steps = max(kIChunk, 2 * ((1 << 17) / top - 2));
            if (lane == 0) {
                flags[2] = chunk_steps;
                mbar_arrive(cut);
            }
        }
        const int nchunks = (nkb + chunk_steps - 1) / chunk_steps;
        int i = 0, s = 0, slot = 0;
        uint32_t ph = 0, aph = 0;
        for (int c = 0; c < nchunks && ok; ++c) {
            const int buf = c % nbuf, end = min(nkb, (c + 1) * chunk_steps);
            const uint32_t acc = tmem + buf * n_pad;
            if (c >= nbuf) ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[buf], (c / nbuf & 1) ^ 1, flags));
            uint32_t more = 0;
            for (; i < end && ok; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full_x[s], ph, flags) && mbar_wait(&conv[slot], aph, flags));
                if (!ok) break;
                tc_fence_after();
                uint64_t xd = sdesc_sw128(smem_u32(xring + s * x_bytes));
                const uint32_t wa = tmem + kIACol + slot * 64;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f16_ta(acc, wa + k * 8, xd + k * 2, idesc, k > 0 ? 1u : more);
                    if (a.xk == 1) umma_commit(&empty_x[s]);
                }
                __syncwarp();
                more = 1;
                xd += n_pad * 8;
                if (a.xk == 1) {
                    if (++s == xs) s = 0, ph ^= 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_x[s], ph, flags));
                    if (!ok) break;
                    tc_fence_after();
                    xd = sdesc_sw128(smem_u32(xring + s * x_bytes));
                }
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f16_ta(acc, wa + 32 + k * 8, xd + k * 2, idesc, 1u);
                    umma_commit(&a_free[slot]);
                    umma_commit(&empty_x[s]);
                }
                __syncwarp();
                if (++s == xs) s = 0, ph ^= 1;
                if (++slot == kIASlots) slot = 0, aph ^= 1;
            }
            if (ok && elect_one()) umma_commit(&acc_full[buf]);
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0 && a.status) report_timeout_status(a.status);
            // every MMA issued above completes before the CTA may leave
            if (elect_one()) umma_commit(drained);
            const unsigned long long t = globaltimer();
            while (!mbar_try_wait(drained, 0) && globaltimer() - t < kWaitLimitNs) {
            }
            __syncwarp();
        }
    } else if (warp < 2 + kIWorkers) {
        // ---- codes to float16 in tensor memory: 32 features and 64 codes of every second step a warp; and the
        // accumulator, 32 features and every fourth 16 tokens a warp ----
        const int q = warp & 3, h = ((warp - 2) >> 2) & 1, set = (warp - 2) >> 3;
        const int row = q * 32 + lane;
        const uint32_t taddr = tmem + kIACol + h * 32 + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t sums = smem_u32(G) + (split * a.per * kIM + row) * 4;
        const int units = n_pad / 16;
        bool ok = true;
        int chunk = 0, chunk_steps = kIChunk, nchunks = 1;  // the next to drain; (known from step kIChunk on)
        bool started = a.splits == 1 || a.alias;
        int sum[kIN / 64][16];  // (indexed at run time: in local memory, touched once a chunk, not in registers)
        auto hand_over = [&](int u, const uint32_t* r) {  // to the CTAs that finish these 16 tokens
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = u * 16 + e, dst = (t * a.per_inv) >> 16;  // = t / per
                if (t < n) st_dsmem_u32(mapa_shared(sums + (t - dst * a.per) * kIM * 4, static_cast<uint32_t>(dst)), r[e]);
            }
        };
        auto drain = [&]() {
            const int buf = chunk % nbuf;
            ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], chunk / nbuf & 1, flags));
            if (!ok) return;
            tc_fence_after();
            const bool first = chunk == 0, last = ++chunk == nchunks;
            if (last && !started) {
                cluster_wait();  // every CTA of the cluster has started
                started = true;
            }
            const uint32_t aaddr = tmem + buf * n_pad + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int u = h * 2 + set, j = 0; u < units; u += 4, ++j) {
                uint32_t r[16];
                tmem_ld16(aaddr + u * 16, r);
                tmem_ld_wait();
                if (!first)
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = static_cast<uint32_t>(sum[j][e] + __float2int_rn(__uint_as_float(r[e])));
                else
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = static_cast<uint32_t>(__float2int_rn(__uint_as_float(r[e])));
                if (!last || (a.alias && a.splits > 1)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[j][e] = static_cast<int>(r[e]);
                } else if (a.splits == 1) {
                    // (the last accumulator is complete: every MMA has read its operands, the ring is idle)
#pragma unroll
                    for (int e = 0; e < 16; ++e) G[(u * 16 + e) * kIM + row] = static_cast<int>(r[e]);
                } else {
                    hand_over(u, r);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        };
        // step i has stage i % ws and slot i % kIASlots, both even numbers: a warp's steps share theirs with no others
        int s = set, slot = set, before = -1;
        uint32_t ph = 0, fph = 1;  // (the slots start free)
        uint4 v[4];
        auto read = [&]() {  // the warp's next codes, once they are there
            const uint8_t* wr = smem + s * kIWBytes + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(wr + (((h * 4 + c) ^ (row & 7)) << 4));
        };
        auto release = [&]() {  // (after their first use: the loads have returned)
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty_w[s]);
            if ((s += 2) >= ws) s -= ws, ph ^= 1;
        };
        auto announce = [&]() {  // the slot stored last, once the store has landed
            if (before < 0) return;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&conv[before]);
        };
        if (set < nkb) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full_w[s], 0, flags));
            if (ok) read();
        }
        auto learn = [&]() {  // the chunks: once, by step kIChunk
            if (nchunks > 1 || chunk_steps >= nkb) return;
            ok = __all_sync(0xffffffffu, mbar_wait(cut, 0, flags));
            if (!ok) return;
            chunk_steps = flags[2];
            nchunks = (nkb + chunk_steps - 1) / chunk_steps;
        };
        for (int i = set; i < nkb && ok; i += 2) {
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint2 f = i8_to_f16x4(w[e]);
                    r[c * 8 + e * 2] = f.x;
                    r[c * 8 + e * 2 + 1] = f.y;
                }
            }
            release();
            announce();  // (its latency was covered by the conversion)
            ok = __all_sync(0xffffffffu, mbar_wait(&a_free[slot], fph, flags));
            if (!ok) break;
            tc_fence_after();
            tmem_st32(taddr + slot * 64, r);
            before = slot;
            if ((slot += 2) >= kIASlots) slot -= kIASlots, fph ^= 1;
            // the chunk before is complete by now; or (one accumulator) holds the MMAs up, and enough is converted
            if (i >= kIChunk) learn();
            const bool done = ok && i >= (chunk + 1) * chunk_steps + (nbuf == 2 ? kIChunk / 2 : 2);
            const bool more = i + 2 < nkb;
            if (done || (more && !__all_sync(0xffffffffu, mbar_test(&full_w[s], ph)))) {
                announce();  // (the MMAs need not wait for what follows)
                before = -1;
            }
            if (done) drain();
            if (more && ok) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full_w[s], ph, flags));
                if (ok) read();
            }
        }
        if (ok) announce();
        if (ok) learn();
        while (ok && chunk < nchunks) drain();
        if (!started) cluster_wait();
        if (!ok && lane == 0) flags[0] = 1;
        if (a.alias && a.splits > 1) {
            cluster_sync();  // every CTA's MMAs have read their operands: the rings are idle
            if (ok)
#pragma unroll 1
                for (int u = h * 2 + set, j = 0; u < units; u += 4, ++j) {
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = static_cast<uint32_t>(sum[j][e]);
                    hand_over(u, r);
                }
        }
    } else if constexpr (FUSE) {
        const int lt = threadIdx.x - kIThreads;  // 0..255
        // (perm and the segments are older than the kernel ahead)
        const bool st_ok = !a.status || __ldcg(a.status) == LORA_OK;
        if (lt < cnt) {  // (per <= kILora)
            const int t = st_ok ? __ldcg(a.perm + row0 + t0 + lt) : 0;
            row_sm[lt] = t;
            const int slot = st_ok ? __ldcg(a.idx + t) : -1;
            tok_slot[lt] = slot;
            tok_rank[lt] = slot >= 0 ? a.table[slot].rank : 0;
        }
        // ---- the LoRA terms of this CTA's tokens: a feature a thread, half of the tokens, four at a time.  What
        // costs is the latency of B: its rows are held while the tokens' adapter is the same, and those of four
        // adapters are in flight together where it is not ----
        const int f = lt & 127, half = lt >> 7, o = m_tile * kIM + f, R = a.R, cols = a.s_cols;
        const int mid = (cnt + 1) / 2, ub = half ? mid : 0, ue = half ? cnt : mid;
        constexpr int CH = sizeof(T) == 2 ? 2 : 1;  // pieces of 8 columns at once
        pdl_wait();  // the shrink output
        const size_t part = (size_t)a.n * R;
        for (int j0 = 0; j0 < R; j0 += cols) {
            __syncwarp();
            named_bar_sync(2, kILora);
            for (int e = lt; e < cnt * cols; e += kILora) {
                const int u = e / cols, j = j0 + e - u * cols;
                float v = 0.f;
                if (j < tok_rank[u]) {
                    const float* sp = a.s_in + (size_t)row_sm[u] * R + j;
                    for (int p = 0; p < a.s_parts; ++p) v += __ldcg(sp + p * part);
                }
                S[e] = v;
            }
            named_bar_sync(2, kILora);
            if (o >= a.h_out) continue;
            for (int j = 0; j < min(cols, R - j0); j += 8 * CH) {
                BRow<T> b[4][CH];
                const T* Bo = static_cast<const T*>(a.B) + (size_t)o * R + j0 + j;
                auto load = [&](int k, int slot, int rank) {  // (columns past the rank are zeros)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        b[k][c].load(Bo + (size_t)max(slot, 0) * a.h_out * R + 8 * c, rank > j0 + j + 8 * c ? R - j0 - j - 8 * c : 0);
                };
                auto add = [&](int c, const float (&bf)[8], int u, float& acc) {
                    const float4* sp = reinterpret_cast<const float4*>(S + u * cols + j + 8 * c);
                    const float4 lo = sp[0], hi = sp[1];
                    const float sf[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc = fmaf(bf[e], sf[e], acc);
                };
                const int pieces = min(CH, (R - j0 - j + 7) / 8);
                int held = INT_MIN;
                for (int u0 = ub; u0 < ue; u0 += 4) {
                    float acc[4];
                    int slot[4];
                    bool same = true;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int u = min(u0 + k, ue - 1);
                        slot[k] = tok_slot[u];
                        acc[k] = j0 + j > 0 ? L[u * kIM + f] : 0.f;
                        same = same && slot[k] == slot[0];
                    }
                    if (same) {
                        if (slot[0] != held) load(0, slot[0], tok_rank[u0]);
                        held = slot[0];
                        if (held >= 0)
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                if (c >= pieces) break;
                                float bf[8];
                                b[0][c].get(bf);
#pragma unroll
                                for (int k = 0; k < 4; ++k) add(c, bf, min(u0 + k, ue - 1), acc[k]);
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) load(k, slot[k], tok_rank[min(u0 + k, ue - 1)]);
                        held = INT_MIN;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            if (c >= pieces) break;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float bf[8];
                                b[k][c].get(bf);
                                add(c, bf, min(u0 + k, ue - 1), acc[k]);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (u0 + k < ue) L[(u0 + k) * kIM + f] = acc[k];
                }
            }
        }
    }

    if (a.splits > 1 && (warp < 2 || warp >= 2 + kIWorkers)) {  // (as the workers have)
        if (a.alias) cluster_arrive();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    bool good = flags[0] == 0;
    if (a.splits > 1) {

        // sums of which a CTA gave up its part are no one's
        if (!good && threadIdx.x < a.splits)
            st_dsmem_u32(mapa_shared(smem_u32(const_cast<int*>(flags + 1)), threadIdx.x), 1u);
        cluster_sync();  // every CTA has added its sums
        good = good && flags[1] == 0;
    }
    pdl_wait();
    if (good && cnt > 0 && (!a.status || __ldcg(a.status) == LORA_OK)) {
        // ---- this CTA's share of the tokens ----
        T* y = static_cast<T*>(a.y);
        if (a.vec) {
            // 8 features a thread, 16 neighbouring threads a token's 128
            const int o8 = (threadIdx.x & 15) * 8, o = m_tile * kIM + o8;
            for (int u = threadIdx.x >> 4; u < cnt; u += blockDim.x / 16) {
                int v[8] = {};
                for (int c = 0; c < a.splits; ++c) {
                    const int4* p = reinterpret_cast<const int4*>(G + (c * a.per + u) * kIM + o8);
                    const int4 lo = p[0], hi = p[1];
                    v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
                    v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
                }
                alignas(16) T w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float r = i8_scaled(v[e], sx_sm[u], sw_sm[o8 + e]);
                    if constexpr (FUSE) r += L[u * kIM + o8 + e];
                    w[e] = from_f32<T>(r);
                }
                T* yp = y + (long long)row_sm[u] * a.ldy + o;
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
            // rows off 16-byte boundaries: neighbouring threads store neighbours
            for (int e = threadIdx.x; e < cnt * kIM; e += blockDim.x) {
                const int u = e / kIM, f = e % kIM, o = m_tile * kIM + f;
                int v = 0;
                for (int c = 0; c < a.splits; ++c) v += G[c * a.per * kIM + e];
                float r = i8_scaled(v, sx_sm[u], sw_sm[f]);
                if constexpr (FUSE) r += L[e];
                if (o < a.h_out) y[(long long)row_sm[u] * a.ldy + o] = from_f32<T>(r);
            }
        }
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Clusters of that many CTAs that the GPU holds at once: of 4 nearly a quarter of the SMs, of 8 far fewer than an eighth,
// as a cluster lies in one group of SMs.
static int max_clusters(int size) {
    static int held[9] = {};  // every variant takes most of an SM's shared memory: the same for each
    if (size == 1) return num_sms();
    if (!held[size]) {
        cudaLaunchConfig_t q;
        memset(&q, 0, sizeof(q));
        q.gridDim = dim3(1, size);
        q.blockDim = dim3(kIThreads + kILora);
        q.dynamicSmemBytes = kISmemMax;
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 1;
        qa[0].val.clusterDim.y = size;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int c = 0;
        if (cudaFuncSetAttribute(i8_tile_kernel<float, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kISmemMax) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&c, (const void*)i8_tile_kernel<float, true>, &q) != cudaSuccess || c < 1) {
            (void)cudaGetLastError();
            c = std::max(1, num_sms() / size / 2);
        }
        held[size] = c;
    }
    return held[size];
}

// How a launch cuts its work: tokens in groups of n_pad, K among `splits` CTAs, and the stages that leaves room for.
struct TilePlan {
    int n_pad, groups, splits, kb_per_split, per, alias, xk, xstages, wstages, s_cols, ring_bytes;
    size_t smem;
};
static bool tile_plan(int n, int m_tiles, int kb, bool fuse, int R, int groups, int splits, TilePlan& p) {
    p.n_pad = ((n + groups - 1) / groups + 15) / 16 * 16;
    p.groups = (n + p.n_pad - 1) / p.n_pad;
    p.kb_per_split = (kb + splits - 1) / splits;
    p.splits = (kb + p.kb_per_split - 1) / p.kb_per_split;
    p.per = (std::min(n, p.n_pad) + p.splits - 1) / p.splits;
    p.alias = p.splits == 1 || p.n_pad > 128;
    p.s_cols = !fuse ? 0 : p.per <= 64 ? std::min(kIMostS, (R + 15) / 16 * 16) : 16;
    const size_t words = (size_t)(p.alias ? 0 : p.splits * p.per * kIM) + (fuse ? p.per * (kIM + p.s_cols + 2) : 0) + 2 * p.per + kIM;
    const size_t tail = words * 4 + kIBars + 1024 + 16;
    // stages of x (at most 4; of 64 codes for more than 128 tokens), then of w (4, 6 or 8: an even number, as the
    // workers' halves alternate)
    p.xk = p.n_pad > 128 ? 1 : 2;
    const size_t x_bytes = (size_t)p.n_pad * 128 * p.xk;
    p.wstages = 0;
    for (int x = 4; x >= 2 && !p.wstages && tail < kISmemMax; --x) {
        const size_t room = kISmemMax - tail, left = room > x * x_bytes ? room - x * x_bytes : 0;
        p.xstages = x;
        p.wstages = (int)std::min<size_t>(left / kIWBytes / 2 * 2, 8);
        if (p.wstages < (x > 2 && p.xk == 2 ? 6 : 4) || (p.xk == 1 && x < 3)) p.wstages = 0;
    }
    p.ring_bytes = (int)std::max<size_t>(p.wstages * kIWBytes + p.xstages * x_bytes,
                                         p.alias ? (size_t)p.splits * p.per * kIM * 4 : 0);
    p.smem = p.ring_bytes + tail;
    return p.wstages && p.smem <= kISmemMax;
}
// What a plan takes, in units of 10 ns: rounds of the grid, a CTA's steps of 128 codes, and what does not depend on K.
// Above 128 tokens there is one accumulator and the sums cross the cluster once the rings are idle.  (4096 x 4096: groups
// of 128 tokens 13.3 us with 8 steps, 17.8 with 16, 24.3 with 32; of 256 22.3 with 8, 27.0 with 16.)
static long long tile_cost(const TilePlan& p, int m_tiles) {
    const long long clusters = (long long)m_tiles * p.groups, held = max_clusters(p.splits);
    const int n = p.n_pad;
    const int fix = n <= 128 ? 400 + 2 * n : 300 + (p.splits > 1 ? 4 : 2) * n, step = n <= 128 ? 45 : 45 + (n - 128) / 9;
    return (clusters + held - 1) / held * (fix + (long long)p.kb_per_split * step);
}

template <typename T, bool FUSE>
static int launch_tile_t(const I8Rows& x, const I8View& w, void* y, long long ldy, int32_t* status, bool early_x, bool release,
                         const I8Lora* lora, cudaStream_t st) {
    I8TileArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.status = status;
    a.perm = x.perm;
    a.sx = x.scales;
    a.peak = x.peak;
    a.sw = w.scales;
    a.ldy = ldy;
    a.n = x.rows;
    a.h_out = w.rows;
    a.kb_total = (int)((w.pitch + kIK - 1) / kIK);
    a.early_x = early_x;
    a.release = release;
    // y is written 16 bytes at a time when every row starts on a 16-byte boundary
    a.vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (long long)sizeof(T)) % 16 == 0;
    const int m_tiles = (w.rows + kIM - 1) / kIM;
    TilePlan best;
    long long cost = LLONG_MAX;
    for (int most = kIN; most >= 64; most /= 2)
        for (int splits = std::min(8, a.kb_total); splits >= 1; --splits) {
            TilePlan p;
            if (!tile_plan(x.rows, m_tiles, a.kb_total, FUSE, FUSE ? lora->pool->R : 0, (x.rows + most - 1) / most, splits, p)) continue;
            const long long c = tile_cost(p, m_tiles);
            if (c < cost) cost = c, best = p;
        }
    if (cost == LLONG_MAX || best.groups > 65535) return set_error(LORA_EUNSUP, "8-bit product of %d rows", x.rows);
    a.n_pad = best.n_pad;
    a.splits = best.splits;
    a.kb_per_split = best.kb_per_split;
    a.per = best.per;
    a.per_inv = 65535 / a.per + 1;  // t / per = t * per_inv >> 16 for t < 256
    a.alias = best.alias;
    a.xk = best.xk;
    a.xstages = best.xstages;
    a.wstages = best.wstages;
    a.s_cols = best.s_cols;
    a.ring_bytes = best.ring_bytes;
    if (lora) {
        const PoolView& pv = *lora->pool;
        a.table = pv.table;
        a.B = pv.B;
        a.idx = lora->idx;
        a.s_in = lora->s_in;
        a.R = pv.R;
        a.s_parts = lora->s_parts;
    }
    CUtensorMap mW, mX;
    int rc = make_map_fp4(&mW, w.codes, w.pitch, w.rows, kIM);  // (bytes in boxes of 128)
    if (!rc) rc = make_map(&mX, x.x16, 0, w.pitch, x.rows, a.n_pad);
    if (rc) return rc;
    static bool attr_set = false;
    if (!attr_set) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(i8_tile_kernel<T, FUSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kISmemMax));
        attr_set = true;
    }
    void* args[] = {(void*)&mW, (void*)&mX, (void*)&a};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(m_tiles, a.splits, best.groups);
    cfg.blockDim = dim3(kIThreads + (FUSE ? kILora : 0));
    cfg.dynamicSmemBytes = best.smem;
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

int launch_i8_tile(const I8Rows& x, const I8View& w, void* y, int dtype, long long ldy, int32_t* status, bool early_x,
                   bool release, const I8Lora* lora, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32:
            return lora ? tc::launch_tile_t<float, true>(x, w, y, ldy, status, early_x, release, lora, st)
                        : tc::launch_tile_t<float, false>(x, w, y, ldy, status, early_x, release, nullptr, st);
        case LORA_F16:
            return lora ? tc::launch_tile_t<__half, true>(x, w, y, ldy, status, early_x, release, lora, st)
                        : tc::launch_tile_t<__half, false>(x, w, y, ldy, status, early_x, release, nullptr, st);
        default:
            return lora ? tc::launch_tile_t<__nv_bfloat16, true>(x, w, y, ldy, status, early_x, release, lora, st)
                        : tc::launch_tile_t<__nv_bfloat16, false>(x, w, y, ldy, status, early_x, release, nullptr, st);
    }
}

}  // namespace lora
