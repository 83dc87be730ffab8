// Large batches (more than 256 tokens) over a 4-bit base weight: the product on CTA pairs, and the
// kernel before it that quantises x and computes the LoRA shrink in one read of x.
//
// The linear's tokens are taken in the order of the segments (sorted by adapter), so a tile of
// tokens meets few adapters whatever the batch's order; y rows go back to their own places.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "fp4_device.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace lora {
namespace tc {

using namespace ptx;

// ============================================================================================
// product: 256 x 256 tiles on CTA pairs (tcgen05 cta_group::2)
// ============================================================================================
// At 4 bits an operand byte carries 4 multiply-adds per output row, so a 128 x 256 tile per CTA
// would take operands in faster (about 100 bytes a clock and SM at the tensor cores' rate) than an
// SM receives them.  A pair of CTAs shares a 256 x 256 tile: CTA r stages token rows 128r.. and
// weight rows 128r.. (32 KB of codes a step of 256 along K instead of 48 KB), the even CTA issues
// M = 256 x N = 256 MMAs that read both halves, and each CTA's tensor memory receives its 128
// tokens x 256 features.
//
// Block scales reach tensor memory through registers: four warps read a step's 3 KB from shared
// memory and store it to their 32 lanes (tcgen05.st).  Copying it there by tcgen05.cp from the
// thread that issues the MMAs holds the tensor pipe: a step of four MMAs and six copies of 512 bytes
// took 815 clocks, the MMAs alone 512, about 50 clocks a copy.
//
// Tensor memory (512 columns): two accumulators of 256 columns that share 96 of them ([0, 256) and
// [160, 416)), and four sets of 24 scale columns.  The main loop of the next tile may start once
// the epilogue has taken the shared columns, which it takes first.
//
// The LoRA term is more K blocks of the same accumulator: for the distinct adapters d of the pair's
// 256 tokens, columns d * r_max + j hold s[t, j] on the token side (zero unless t uses d) and B_d[o, j]
// on the feature side, kind::f16, 16 columns a block, two block buffers.  s is float32 and goes in as two
// 16-bit parts (split8) that multiply the same B: in one, its rounding would add to y's.  Because those
// products reach every token of the tile, an infinity or NaN in one tenant's B would reach the other
// tenants' rows as 0 * inf: such elements are replaced by zeros here and the epilogue adds them to
// their own tokens alone, as it does what of s a float16 cannot hold.
//
// Warps: 0 loads codes, 1 issues MMAs (even CTA), 2-9 drain the accumulator, 10-13 build the LoRA
// blocks, 14-17 bring in the scales.
//
// Measured: 8191 x 11008 x 4096 to float32 in 121 us (112 on some boxes), 6.1 PFLOP/s, 63 % of the MMAs' own
// rate, 686 clocks a step where its MMAs take 512.  The likeliest bound is the shared-memory port, 128
// bytes a clock: a step's 32 KB of codes arrive and are read once by the MMAs (64 KB), its 3 KB of scales
// arrive and are read by each of four warps (15 KB), and y's pass adds 6 KB, 85 KB or 680 clocks.  Where
// K is short it is the epilogue's pass through shared memory: 16384 x 1024 x 4096 takes 46.7 us in bf16,
// 28 in a copy that left the pass out.
constexpr int kPM = 128;         // token rows per CTA
constexpr int kPN = 256;         // features per pair tile
constexpr int kPThreads = 576;
constexpr uint32_t kPXBytes = kPM * 128, kPWBytes = (kPN / 2) * 128;
constexpr uint32_t kPStageBytes = kPXBytes + kPWBytes;
constexpr int kPMaxStages = 6;
constexpr int kPScaleSlots = 5;                     // shared-memory slots of scales: 1 KB of x, 2 KB of w
constexpr uint32_t kPScaleBytes = 3 * 1024;
constexpr int kPScaleSets = 4;                      // tensor-memory sets of 24 columns
constexpr int kPScaleCol = 512 - 24 * kPScaleSets;
constexpr int kPAcc1 = kPScaleCol - kPN;            // first column of the second accumulator
constexpr int kPLoraChunk = kPM * 16;               // 8 columns of 128 rows, 16 bytes a row
constexpr int kPLoraBytes = 6 * kPLoraChunk;        // one block: 2 chunks of s's high parts, low parts, B
constexpr int kPScratch = 64 * 4 + 256 * 4 + 8;
// after the stages: scales, LoRA blocks (if any), y staging (8 warps of 1024 elements), the
// LoRA scratch, barriers
constexpr size_t pair_smem(int stages, bool fuse, size_t elt) {
    return (size_t)stages * kPStageBytes + kPScaleSlots * kPScaleBytes + (fuse ? 2 * kPLoraBytes : 0) + 8 * 1024 * elt +
           kPScratch + 256 + 1024;
}
constexpr size_t kSmemMax = 227 * 1024;
static_assert(kPAcc1 >= kPN - 128, "the shared columns are within the first 128 the epilogue takes");
static_assert(pair_smem(5, true, 2) <= kSmemMax && pair_smem(6, false, 2) <= kSmemMax && pair_smem(5, false, 4) <= kSmemMax,
              "shared memory of the pair kernel");

struct PairArgs {
    void* y;
    int32_t* status;         // nullable
    const int32_t* perm;     // row of y of each token row (nullptr: the same)
    const int32_t* idx;      // fuse: adapter slot by original token
    const float* s;          // fuse: [n][R] shrink output in token-row order
    const void* B;           // fuse: pool's B slab
    const uint8_t* sx;       // scale tiles of x and w
    const uint8_t* sw;
    long long ldy;
    int n, h_out, m_tiles, n_tiles, nkb, kt, stages;
    int R, fuse, bf16, early_w;
};

// A ring position: index and parity of its current use.
struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1;
        }
    }
};

// 16 bytes of T from float32 bits, each rounded once.
template <typename T> __device__ __forceinline__ uint4 round16(const uint32_t* r) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __float22half2_rn(f);
                memcpy(&w[i], &h, 4);
            } else {
                const __nv_bfloat162 h = __float22bfloat162_rn(f);
                memcpy(&w[i], &h, 4);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// VEC: y is written 16 bytes at a time (rows on 16-byte boundaries).  A kernel of its own for the other
// rows, for which the common one would spill registers (16384 x 4096 x 4096 bf16: 97.5 against 93.4 us).
template <typename T, bool VEC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
fp4_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const PairArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const int stages = a.stages;
    uint8_t* scale_sm = smem + stages * kPStageBytes;
    uint8_t* lora_sm = scale_sm + kPScaleSlots * kPScaleBytes;   // [2] blocks {token side, feature side}
    uint8_t* yst = lora_sm + (a.fuse ? 2 * kPLoraBytes : 0);     // [8 warps][1024]
    uint32_t* seen = reinterpret_cast<uint32_t*>(yst + 8 * 1024 * sizeof(T));  // [64] slots the tile's tokens name
    int* dlist = reinterpret_cast<int*>(seen + 64);              // [256] the tile's slots in order
    int* distinct = dlist + 256;                                 // [2] their number
    uint64_t* full = reinterpret_cast<uint64_t*>(distinct + 2);  // even CTA: codes of both halves, 8 scale warps
    uint64_t* empty = full + kPMaxStages;    // the even CTA's commits (multicast)
    uint64_t* acc_full = empty + kPMaxStages;  // [2] (multicast)
    uint64_t* ov_free = acc_full + 2;        // even CTA: the shared columns are drained (16 warps)
    uint64_t* lora_own = ov_free + 1;        // [2] a LoRA block of this CTA is written (4 warps)
    uint64_t* lora_peer = lora_own + 2;      // [2] even CTA: the odd CTA's block is written (relayed)
    uint64_t* lora_empty = lora_peer + 2;    // [2] (multicast)
    // by parity of the tile (the LoRA warps may be a tile ahead of the others):
    uint64_t* linfo = lora_empty + 2;        // [2] the tile's number of LoRA blocks is known
    uint64_t* epi_done = linfo + 2;          // [2] the epilogues (16 warps of both CTAs) and the odd CTA's relay are through
    uint64_t* lora_done = epi_done + 2;      // [2] the tile's LoRA blocks are written (8 warps of both CTAs)
    uint64_t* drained = lora_done + 2;       // even CTA: every MMA has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    // abort, -, then by parity of the tile: [2] 1 + the last tile whose blocks left products out, [2] LoRA blocks
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kPMaxStages + 16) * 8 + 28 <= 256, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int total = a.m_tiles * a.n_tiles;
    const int nkb = a.nkb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 9);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&lora_own[b], 4);
            mbar_init(&lora_peer[b], 1);
            mbar_init(&lora_empty[b], 1);
            mbar_init(&linfo[b], 1);
            mbar_init(&epi_done[b], rank == 1 ? 17 : 16);
            mbar_init(&lora_done[b], 8);
        }
        mbar_init(ov_free, 16);
        mbar_init(drained, 1);
        for (int i = 0; i < 6; ++i) flags[i] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW);
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
    // a product by itself releases nothing early: its y may be a weight that a 16-bit linear streams unwaited
    if (a.early_w) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            auto load_w = [&](int s, int kb, int n0) {
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPStageBytes);
                tma_load_2d_pair(smem + s * kPStageBytes + kPXBytes, &tmW, full0 + static_cast<uint32_t>(s) * 8u, kb * 128,
                                 n0 + static_cast<int>(rank) * (kPN / 2));
            };
            auto load_x = [&](int s, int kb, int m0) {
                tma_load_2d_pair(smem + s * kPStageBytes, &tmX, full0 + static_cast<uint32_t>(s) * 8u, kb * 128,
                                 m0 + static_cast<int>(rank) * kPM);
            };
            // the first tile's weight boxes go out before the kernels ahead have finished
            int pre = 0;
            if (a.early_w && pair < total) {
                pre = min(stages, nkb);
                for (int i = 0; i < pre; ++i) load_w(i, i, pair % a.n_tiles * kPN);
            }
            pdl_wait();
            int it = 0;
            Ring r;
            for (int tile = pair; tile < total && !flags[0]; tile += npairs) {
                const int m0 = tile / a.n_tiles * 2 * kPM, n0 = tile % a.n_tiles * kPN;
                for (int kb = 0; kb < nkb; ++kb, ++it, r.next(stages)) {
                    if (it >= stages && !mbar_wait(&empty[r.i], r.ph ^ 1, flags)) break;
                    if (it >= pre) load_w(r.i, kb, n0);
                    load_x(r.i, kb, m0);
                }
            }
            if (flags[0]) {  // aborted: give the copies in flight (both CTAs') time to land
                if (a.status) report_timeout_status(a.status);
                if (rank == 0)
                    for (int i = 0; i < stages; ++i) {
                        const unsigned long long t0 = globaltimer();
                        while (!mbar_try_wait(&full[i], 0) && globaltimer() - t0 < kWaitLimitNs / 8) {
                        }
                    }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc_lora = idesc_f16(2 * kPM, kPN, a.bf16 != 0);
            int it = 0, local = 0, lb = 0;
            Ring r;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += npairs, ++local) {
                const int buf = local & 1;
                const uint32_t acc = tmem + buf * kPAcc1;
                // the tile before has left the columns both accumulators share (and, the epilogue
                // taking tiles in order, the one before that has left this accumulator)
                if (local > 0 && !mbar_wait(ov_free, (local - 1) & 1, flags)) {
                    ok = false;
                    break;
                }
                for (int kb = 0; kb < nkb; ++kb, ++it, r.next(stages)) {
                    if (!mbar_wait(&full[r.i], r.ph, flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t xd = sdesc_sw128(smem_u32(smem + r.i * kPStageBytes));
                    const uint64_t wd = xd + (kPXBytes >> 4);
                    const uint32_t sfa = tmem + kPScaleCol + (it % kPScaleSets) * 24, sfb = sfa + 8;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_pair_mxf4(acc, xd + 2 * k, wd + 2 * k, idesc_mxf4(2 * kPM, kPN, (k & 1) * 2),
                                       sfa + 4 * (k >> 1), sfb + 8 * (k >> 1), (kb > 0 || k > 0) ? 1u : 0u);
                    umma_pair_commit(&empty[r.i], 0x3);
                }
                if (!ok) break;
                if (a.fuse) {
                    if (!mbar_wait(&linfo[buf], (local >> 1) & 1, flags)) {
                        ok = false;
                        break;
                    }
                    const int blocks = flags[4 + buf];
                    for (int b = 0; b < blocks; ++b, ++lb) {
                        const int lbuf = lb & 1;
                        if (!mbar_wait(&lora_own[lbuf], (lb >> 1) & 1, flags) ||
                            !mbar_wait_cluster(&lora_peer[lbuf], (lb >> 1) & 1, flags)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(lora_sm + lbuf * kPLoraBytes), ba = sa + 4 * kPLoraChunk;
#pragma unroll
                        for (int k = 0; k < 2; ++k)  // the high parts, the low ones
                            umma_pair_f16(acc, sdesc_chunks(sa + 2 * k * kPLoraChunk, kPLoraChunk),
                                          sdesc_chunks(ba, kPLoraChunk), idesc_lora, 1u);
                        umma_pair_commit(&lora_empty[lbuf], 0x3);
                    }
                    if (!ok) break;
                }
                umma_pair_commit(&acc_full[buf], 0x3);
            }
            if (!ok && a.status) report_timeout_status(a.status);
            // every MMA issued above has completed before the pair may tear down
            umma_pair_commit(drained, 0x1);
            const unsigned long long t0 = globaltimer();
            while (!mbar_try_wait(drained, 0) && globaltimer() - t0 < kWaitLimitNs) {
            }
        } else if (lane == 0 && a.fuse) {
            // odd CTA: tells the even one that a LoRA block is written.  A release at cluster scope waits
            // for every access of its thread, so it is this thread's and not the writers', whose next
            // loads it would wait for (600 tokens over 100 adapters of rank 16, s in one part: 76 against 65 us).
            const uint32_t peer0 = mapa_shared(smem_u32(lora_peer), 0);
            int local = 0, lb = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += npairs, ++local) {
                ok = mbar_wait(&linfo[local & 1], (local >> 1) & 1, flags);
                const int blocks = ok ? flags[4 + (local & 1)] : 0;
                for (int b = 0; b < blocks && ok; ++b, ++lb) {
                    ok = mbar_wait(&lora_own[lb & 1], (lb >> 1) & 1, flags);
                    if (ok) mbar_arrive_cluster(peer0 + static_cast<uint32_t>(lb & 1) * 8u);
                }
                if (ok) mbar_arrive(&epi_done[local & 1]);
            }
            if (!ok && a.status) report_timeout_status(a.status);
        }
    } else if (warp < 10) {
        // ---- epilogue: thread <-> token row (TMEM lane) of this CTA's half; two warps share a row,
        // taking alternate pieces of 128 bytes of y ----
        const int q = warp & 3, hv = (warp - 2) >> 2;
        constexpr int kCols = 128 / sizeof(T);          // features of a piece
        constexpr int kUnits = 64 / kCols;              // pieces a warp holds at once
        constexpr int kStaged = 1024 * sizeof(T) / 128; // rows staged at once
        constexpr int per = 16 / sizeof(T);
        uint8_t* ys = yst + (warp - 2) * (1024 * sizeof(T));
        const uint32_t ov_free0 = mapa_shared(smem_u32(ov_free), 0);
        const uint32_t other_epi = mapa_shared(smem_u32(epi_done), rank ^ 1);
        pdl_wait();
        const int status = a.status ? __ldcg(a.status) : LORA_OK;
        T* y = static_cast<T*>(a.y);
        int local = 0;
        for (int tile = pair; tile < total; tile += npairs, ++local) {
            const int buf = local & 1;
            const int m0 = tile / a.n_tiles * 2 * kPM + static_cast<int>(rank) * kPM, n0 = tile % a.n_tiles * kPN;
            const int row = m0 + q * 32 + lane;
            const int yrow = row < a.n ? (a.perm ? __ldcg(a.perm + row) : row) : -1;
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (local >> 1) & 1, flags))) break;
            tc_fence_after();
            bool any_bad = false;
            int slot = -1;
            if (a.fuse) {
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(&lora_done[buf], (local >> 1) & 1, flags))) break;
                any_bad = flags[2 + buf] == local + 1;
                if (any_bad && yrow >= 0 && status == LORA_OK) slot = __ldcg(a.idx + yrow);
            }
            const uint32_t taddr = tmem + buf * kPAcc1 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // the half of the columns that holds those both accumulators share comes first, 32 columns
                // at a time (64 spill)
                int c0[kUnits];
                uint4 w[kUnits][8];  // in y's type
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const int u = 2 * (half * kUnits + i) + hv;
                    const int cc = (buf == 0 ? kPN / kCols - 1 - u : u) * kCols;
                    c0[i] = n0 + cc;
#pragma unroll
                    for (int k = 0; k < kCols; k += 32) {
                        uint32_t r[32];
                        __syncwarp();
                        tmem_ld16(taddr + cc + k, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
                        tmem_ld16(taddr + cc + k + 16, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
                        tmem_ld_wait();
                        if (half == 0 && i == kUnits - 1 && k + 32 == kCols) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster_relaxed(ov_free0);
                        }
                        if constexpr (sizeof(T) == 2) {
                            if (any_bad && slot >= 0) {  // the products left out of the LoRA blocks
                                for (int c = 0; c < a.R; c += 8) {
                                    float sv[8];
                                    sum_parts8(a.s + (size_t)row * a.R + c, 1, 0, sv);
                                    const T* Bs = static_cast<const T*>(a.B) + ((size_t)slot * a.h_out + c0[i] + k) * a.R + c;
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (c0[i] + k + e < a.h_out)
                                            r[e] = __float_as_uint(
                                                nonfinite_dot8<T>(__ldg(reinterpret_cast<const uint4*>(Bs + (size_t)e * a.R)),
                                                                  sv, __uint_as_float(r[e])));
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += per) w[i][(k + e) / per] = round16<T>(&r[e]);
                    }
                }
                if (status != LORA_OK) continue;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    if (c0[i] >= a.h_out) continue;
                    // through shared memory (16-byte pieces permuted by row), so that eight neighbouring
                    // lanes write 128 consecutive bytes of a row of y.  (Whole 32-byte sectors straight from
                    // the registers were slower: 131 against 120 us for 8191 x 11008 x 4096 in float32.)
                    const int c = lane & 7, col = c0[i] + c * per;
#pragma unroll
                    for (int r0 = 0; r0 < 32; r0 += kStaged) {
                        __syncwarp();
                        if (lane >= r0 && lane < r0 + kStaged) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                *reinterpret_cast<uint4*>(ys + (lane - r0) * 128 + ((k ^ (lane & 7)) << 4)) = w[i][k];
                        }
                        __syncwarp();
                        if constexpr (!VEC) {
                            // rows off 16-byte boundaries: an element a lane, neighbours side by side, eight rows'
                            // reads at once (15323 x 66 x 3695 in float16: 85 us one row after the other, 55 so)
                            for (int k = 0; k < kStaged; k += 8) {
                                T v[8][kCols / 32];
#pragma unroll
                                for (int b = 0; b < 8; ++b)
#pragma unroll
                                    for (int h = 0; h < kCols / 32; ++h) {
                                        const int e = lane + 32 * h;
                                        v[b][h] = *reinterpret_cast<const T*>(ys + (k + b) * 128 + (((e / per) ^ b) << 4) +
                                                                              e % per * sizeof(T));
                                    }
#pragma unroll
                                for (int b = 0; b < 8; ++b) {
                                    const int yr = __shfl_sync(0xffffffffu, yrow, r0 + k + b);
#pragma unroll
                                    for (int h = 0; h < kCols / 32; ++h)
                                        if (yr >= 0 && c0[i] + lane + 32 * h < a.h_out)
                                            y[(long long)yr * a.ldy + c0[i] + lane + 32 * h] = v[b][h];
                                }
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < kStaged; k += 4) {
                                const int rr = k + (lane >> 3);
                                const int yr = __shfl_sync(0xffffffffu, yrow, r0 + rr);
                                const uint4 v = *reinterpret_cast<const uint4*>(ys + rr * 128 + ((c ^ (rr & 7)) << 4));
                                if (yr < 0) continue;
                                T* yp = y + (long long)yr * a.ldy + col;
                                if (col + per <= a.h_out) {
                                    *reinterpret_cast<uint4*>(yp) = v;
                                } else {
                                    alignas(16) T e8[per];
                                    *reinterpret_cast<uint4*>(e8) = v;
#pragma unroll
                                    for (int e = 0; e < per; ++e)
                                        if (col + e < a.h_out) yp[e] = e8[e];
                                }
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && a.fuse) {
                mbar_arrive(&epi_done[buf]);
                mbar_arrive_cluster_relaxed(other_epi + static_cast<uint32_t>(buf) * 8u);
            }
        }
    } else if (warp >= 14) {
        // ---- scales: the four warps copy steps ahead together, and each fills its own 32 lanes ----
        // A step of these warps has to stay shorter than the MMAs of a step (512 clocks), so the copies'
        // addresses only advance, and their issue overlaps the stores to tensor memory.  By the
        // load/store unit: TMA copies of 1 KB were slower (8191 x 11008 x 4096: 167 us as tensor boxes,
        // 184 us as bulk copies).
        constexpr int L = kPScaleSlots - 1;  // steps ahead
        const int q = warp & 3, st = threadIdx.x - 448;
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        const uint32_t taddr = tmem + kPScaleCol + (static_cast<uint32_t>(q * 32) << 16);
        // threads 0-63 copy x's 1 KB and the second of w's, threads 64-127 the first of w's
        int ltile = pair, lkb = 0, lslot = 0;  // next step to copy
        const uint8_t *pa = nullptr, *pb = nullptr;
        auto next_tile = [&]() {
            pa = pb = nullptr;  // tiles past the last row are left out: what they scale is not stored
            if (ltile >= total) return;
            const int m = ltile / a.n_tiles * 2 + static_cast<int>(rank), rt = ltile % a.n_tiles * 2;
            if (st >= 64) {
                pa = a.sw + (size_t)rt * a.kt * 512 + (st - 64) * 16;
            } else {
                if (m * 128 < a.n) pa = a.sx + (size_t)m * a.kt * 512 + st * 16;
                if ((rt + 1) * 128 < a.h_out) pb = a.sw + (size_t)(rt + 1) * a.kt * 512 + st * 16;
            }
        };
        auto copy_next = [&]() {
            uint8_t* dst = scale_sm + lslot * kPScaleBytes + st * 16;
            if (pa) cp_async16(dst, pa), pa += 1024;
            if (pb) cp_async16(dst + 2048, pb), pb += 1024;
            cp_async_commit();  // (a group each step, empty ones too)
            if (++lslot == kPScaleSlots) lslot = 0;
            if (++lkb == nkb) {
                lkb = 0;
                ltile += npairs;
                next_tile();
            }
        };
        pdl_wait();
        next_tile();
        for (int i = 0; i < L; ++i) copy_next();
        int slot = 0, set = 0, back = 0, warm = kPScaleSets;  // back: stage of the step kPScaleSets before
        uint32_t backph = 0;
        Ring cr;  // the stage last stored for
        cr.i = -1;
        bool ok = true;
        for (int tile = pair; tile < total; tile += npairs) {
            for (int kb = 0; kb < nkb; ++kb) {
                cp_async_wait<L - 1>();
                ok = named_bar_and(3, 128, ok);  // everyone's pieces of this step are there, the last step is read
                if (!ok) break;
                const uint4* sp = reinterpret_cast<const uint4*>(scale_sm + slot * kPScaleBytes) + lane;
                if (++slot == kPScaleSlots) slot = 0;
                const uint4 x0 = sp[0], x1 = sp[32];
                const uint4 w00 = sp[64], w01 = sp[96], w10 = sp[128], w11 = sp[160];  // [row tile][step half]
                // the step before is announced only now: its stores' latency overlapped the above
                if (cr.i >= 0) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive_cluster_relaxed(full0 + static_cast<uint32_t>(cr.i) * 8u);
                }
                cr.next(stages);
                // the set's last readers: the MMAs kPScaleSets steps before
                if (warm > 0) {
                    --warm;
                } else {
                    ok = __all_sync(0xffffffffu, mbar_wait(&empty[back], backph, flags));
                    if (++back == stages) {
                        back = 0;
                        backph ^= 1;
                    }
                    tc_fence_after();
                }
                if (ok) {
                    const uint32_t t = taddr + set * 24;
                    tmem_st8(t, x0, x1);
                    tmem_st8(t + 8, w00, w10);
                    tmem_st8(t + 16, w01, w11);
                }
                if (++set == kPScaleSets) set = 0;
                copy_next();
            }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0 && cr.i >= 0) mbar_arrive_cluster_relaxed(full0 + static_cast<uint32_t>(cr.i) * 8u);
        if (!ok && a.status) report_timeout_status(a.status);
        cp_async_wait<0>();
    } else if (a.fuse) {
        // ---- LoRA blocks ----
        const int lt = threadIdx.x - 320;  // 0..127: a token row and a feature of this CTA's half
        if constexpr (sizeof(T) == 2) {
            pdl_wait();
            const int status = a.status ? __ldcg(a.status) : LORA_OK;
            const uint32_t other_done = mapa_shared(smem_u32(lora_done), rank ^ 1);
            const uint32_t other_flags = mapa_shared(smem_u32(const_cast<int*>(flags)), rank ^ 1);
            const int chunks = a.R / 8;
            int local = 0, lb = 0;
            bool ok = true;
            for (int tile = pair; tile < total; tile += npairs, ++local) {
                const int m0 = tile / a.n_tiles * 2 * kPM, n0 = tile % a.n_tiles * kPN;
                // the slots of the pair's 256 tokens: this CTA's row lt, then the other CTA's
                int slot[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = m0 + static_cast<int>(rank ^ h) * kPM + lt;
                    slot[h] = -1;
                    if (row < a.n && status == LORA_OK) slot[h] = __ldcg(a.idx + __ldcg(a.perm + row));
                }
                if (lt < 64) seen[lt] = 0;
                // the epilogue has read this parity's flag of the tile two before (in both CTAs)
                if (local >= 2 && !mbar_wait(&epi_done[local & 1], ((local >> 1) & 1) ^ 1, flags)) ok = false;
                if (!named_bar_and(2, 128, ok)) break;  // all four warps leave together
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (slot[h] >= 0) atomicOr(&seen[slot[h] >> 5], 1u << (slot[h] & 31));
                named_bar_sync(2, 128);
                if (lt < 64) {
                    int at = 0;
                    for (int w = 0; w < lt; ++w) at += __popc(seen[w]);
                    for (uint32_t m = seen[lt]; m; m &= m - 1) dlist[at++] = lt * 32 + __ffs(m) - 1;
                    if (lt == 63) *distinct = at;
                }
                named_bar_sync(2, 128);
                const int P = *distinct * chunks;  // 8-column chunks of the tile's adapters
                const int blocks = (P + 1) / 2;
                if (lt == 0) {
                    flags[4 + (local & 1)] = blocks;
                    mbar_arrive(&linfo[local & 1]);
                }
                const int o = n0 + static_cast<int>(rank) * (kPN / 2) + lt;
                const float* srow = a.s + (size_t)(m0 + static_cast<int>(rank) * kPM + lt) * a.R;
                const T* Bcol = static_cast<const T*>(a.B) + (size_t)o * a.R;
                int d = 0, c = 0;  // the next chunk: columns 8c.. of adapter dlist[d]
                int sl = P > 0 ? dlist[0] : -1;
                struct Block {  // this thread's row and feature of a block
                    float4 s[2][2];
                    uint4 b[2];
                } even, odd;
                auto load = [&](Block& v) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool live = d * chunks + c < P;
                        const float4* sp = reinterpret_cast<const float4*>(srow + c * 8);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v.s[j][h] = live && sl == slot[0] ? __ldcg(sp + h) : make_float4(0.f, 0.f, 0.f, 0.f);
                        v.b[j] = live && o < a.h_out
                                     ? __ldg(reinterpret_cast<const uint4*>(Bcol + (size_t)sl * a.h_out * a.R + c * 8))
                                     : make_uint4(0, 0, 0, 0);
                        if (++c == chunks) {
                            c = 0;
                            ++d;
                            if (d * chunks < P) sl = dlist[d];
                        }
                    }
                };
                auto put = [&](Block& v) {
                    if (lb >= 2 && !__all_sync(0xffffffffu, mbar_wait(&lora_empty[lb & 1], ((lb >> 1) & 1) ^ 1, flags))) {
                        ok = false;
                        return;
                    }
                    uint8_t* blk = lora_sm + (lb & 1) * kPLoraBytes + lt * 16;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 &lo = v.s[j][0], &hi = v.s[j][1];
                        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        uint4 high, low;
                        bool left_out = split8<T>(f, high, low);
                        if (nonfinite8<T>(v.b[j])) {
                            v.b[j] = finite8<T>(v.b[j]);
                            left_out = true;
                        }
                        if (left_out) {  // raise both CTAs' flags of this tile
                            flags[2 + (local & 1)] = local + 1;
                            st_dsmem_u32(other_flags + 4 * (2 + (local & 1)), local + 1);
                        }
                        *reinterpret_cast<uint4*>(blk + j * kPLoraChunk) = high;
                        *reinterpret_cast<uint4*>(blk + (2 + j) * kPLoraChunk) = low;
                        *reinterpret_cast<uint4*>(blk + (4 + j) * kPLoraChunk) = v.b[j];
                    }
                    fence_proxy_async_smem();  // read by the tensor cores
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&lora_own[lb & 1]);
                    ++lb;
                };
                if (blocks > 0) load(even);
                if (blocks > 1) load(odd);
                for (int b = 0; b < blocks; b += 2) {  // two blocks in flight while a buffer is waited for
                    put(even);
                    if (!ok) break;
                    if (b + 2 < blocks) load(even);
                    if (b + 1 == blocks) break;
                    put(odd);
                    if (!ok) break;
                    if (b + 3 < blocks) load(odd);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&lora_done[local & 1]);
                    mbar_arrive_cluster(other_done + static_cast<uint32_t>(local & 1) * 8u);
                }
            }
            if (!ok && a.status) report_timeout_status(a.status);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves (or frees tensor memory) while its pair may still use it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Pairs the GPU holds at once (an SM left over in a group of SMs cannot host a pair).
template <typename T>
static int max_pairs() {
    static int pairs = 0;  // every variant takes all of an SM's shared memory: the same for each
    if (!pairs) {
        cudaLaunchConfig_t q;
        memset(&q, 0, sizeof(q));
        q.gridDim = dim3(2 * (num_sms() / 2));
        q.blockDim = dim3(kPThreads);
        q.dynamicSmemBytes = kSmemMax;
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 2;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, (const void*)fp4_pair_kernel<T, true>, &q) != cudaSuccess || c < 1) {
            (void)cudaGetLastError();
            c = num_sms() / 2;
        }
        pairs = std::min(c, num_sms() / 2);
    }
    return pairs;
}

template <typename T>
static int launch_pair_t(const Fp4View& x, const Fp4View& w, void* y, long long ldy, int32_t* status, bool early_w,
                         const Fp4Lora* lora, cudaStream_t st) {
    PairArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.status = status;
    a.ldy = ldy;
    a.n = x.rows;
    a.h_out = w.rows;
    a.m_tiles = (x.rows + 2 * kPM - 1) / (2 * kPM);
    a.n_tiles = (w.rows + kPN - 1) / kPN;
    a.nkb = x.ktiles / 2;
    a.kt = x.ktiles;
    if ((long long)a.m_tiles * a.n_tiles > INT_MAX / 2)
        return set_error(LORA_EUNSUP, "4-bit product of %d x %d outputs is too large", x.rows, w.rows);
    a.early_w = early_w;
    // six stages where neither the LoRA blocks nor float32 staging take the room of one
    a.stages = !lora && sizeof(T) == 2 ? 6 : 5;
    // rows of y are written 16 bytes at a time when every row starts on a 16-byte boundary
    const bool vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (long long)sizeof(T)) % 16 == 0;
    if (lora) {
        a.fuse = 1;
        a.perm = lora->perm;
        a.idx = lora->idx;
        a.s = lora->s;
        a.B = lora->B;
        a.R = lora->R;
        a.bf16 = std::is_same<T, __nv_bfloat16>::value;
    }
    a.sx = x.scales;
    a.sw = w.scales;
    CUtensorMap mX, mW;
    int rc = make_map_fp4(&mX, x.codes, x.pitch, x.rows, kPM);
    if (!rc) rc = make_map_fp4(&mW, w.codes, w.pitch, w.rows, kPN / 2);
    if (rc) return rc;
    static bool attr = false;
    if (!attr) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(fp4_pair_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax));
        LORA_CUDA_TRY(cudaFuncSetAttribute(fp4_pair_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax));
        attr = true;
    }
    const int pairs = (int)std::min<long long>((long long)a.m_tiles * a.n_tiles, max_pairs<T>());
    void* args[] = {(void*)&mX, (void*)&mW, (void*)&a};
    LORA_CUDA_TRY(launch_pdl(vec ? (const void*)fp4_pair_kernel<T, true> : (const void*)fp4_pair_kernel<T, false>, dim3(2 * pairs), dim3(kPThreads),
                             pair_smem(a.stages, a.fuse != 0, sizeof(T)), st, args));
    return LORA_OK;
}

// ============================================================================================
// before the product: x quantised and the LoRA shrink, one read of x
// ============================================================================================
// One CTA per 128 tokens in segment order and part of K.  The worker warps copy the tokens' rows of
// x to shared memory (cp.async, 128 columns a step, each thread its own 64 bytes), quantise them as
// the quantise kernel does, and the tensor cores multiply them with the A rows of the tile's adapters
// (TMA): the part's share of s[t, :] = (alpha / r) x[t] A^T, in float32.  (Loads to registers a step
// ahead spill, which waits for them at once: 58 us against 50 for 16384 x 4096, r_max 16.)  Tiles whose
// adapters need more accumulator columns than a pass holds take several passes over their columns.
// The parts of a tile are a thread-block cluster: they leave their shares in global memory, and after
// the cluster barrier each adds up some of the rows.
// With x already stored in 4 bits, the codes and scales are copied instead.  One read of x where a
// quantiser and a shrink would take two: 50 us for 16384 x 4096, 41 with no adapter in the batch (the
// quantiser alone 28).  That is 3 TB/s and 53 % of the issue slots, 63 % on the SMs that hold two CTAs:
// neither is full, and which of the two holds it is not settled.
constexpr int kQWorkers = 16;   // worker warps: with two CTAs an SM, 32 to hide their latencies
constexpr int kQThreads = 64 + 32 * kQWorkers;  // warp 0: A rows, warp 1: MMAs
constexpr uint32_t kQXBytes = 128 * 256;  // two 64-column swizzled halves
// Accumulator columns (A rows) per pass.  64 lets two CTAs share an SM; 256 (one CTA) where the grid does not
// fill the SMs twice anyway, or where 128 sorted tokens are likely to name more adapters than 64 columns
// hold, each pass reading x again.
inline int prep_cap(int n, int S, int R, int ctas) {
    const int per_adapter = std::max(1, n / std::max(1, std::min(n, S)));
    const int columns = std::min(S, 128 / per_adapter + 1) * R;
    return ctas <= num_sms() || columns > 64 ? 256 : std::max(64, (R + 15) / 16 * 16);
}
inline size_t prep_smem(int cap) { return 2 * ((size_t)kQXBytes + cap * 256) + 1024 + 128 * 4 + 64 * 8 + 128 * 4 + 256; }

struct PrepArgs {
    PoolView pool;
    SegView seg;
    const void* x;
    Fp4View q;                 // out: rows in segment order
    const uint8_t* xq_codes;   // x already stored, rows in token order (nullable)
    const uint8_t* xq_scales;
    float* parts_s;            // scratch: [parts][n][R]
    float* s;                  // out: [n][R], rows in segment order (the scratch itself where there is one part)
    int bf16, cap, steps, parts;  // steps: 128-column steps per part
};

template <typename T>
__global__ void __launch_bounds__(kQThreads, 2)
fp4_prepare_kernel(const __grid_constant__ CUtensorMap tmA, const PrepArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const uint32_t a_half = static_cast<uint32_t>(a.cap) * 128, stage_bytes = kQXBytes + 2 * a_half;
    int* slot_sm = reinterpret_cast<int*>(smem + 2 * stage_bytes);  // [128] slot of each row's token (-1: none)
    uint32_t* seen = reinterpret_cast<uint32_t*>(slot_sm + 128);    // [64]
    int* before = reinterpret_cast<int*>(seen + 64);                // [64]
    int* dlist = before + 64;                                       // [128]
    uint64_t* full = reinterpret_cast<uint64_t*>(dlist + 128);      // [2] the worker warps and the A rows
    uint64_t* empty = full + 2;                                     // [2]
    uint64_t* acc_full = empty + 2;
    uint64_t* acc_free = acc_full + 1;                              // 4 worker warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 1);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int m0 = blockIdx.x * 128;
    const int R = a.pool.R, h = a.pool.h_in;
    const int ch0 = blockIdx.y * a.steps;                      // this part's steps of 128 columns
    const int nch = min(a.q.ktiles, ch0 + a.steps) - ch0;
    const uint32_t tmem_cols = a.cap <= 64 ? 64 : a.cap <= 128 ? 128 : 256;
    const int l16 = lane & 15;
    // a worker's rows: r0 + 32 j; its first step of x is on its way before the tile's adapters are found
    const int r0 = (warp - 2) * 2 + (lane >> 4);
    int src[4];
    const T* x = static_cast<const T*>(a.x);
    // this thread's 16 bytes of row r0 + 32 j in a stage: a 64-column half, the chunk permuted by row
    uint8_t* own = smem + (l16 >> 3) * (kQXBytes / 2) + r0 * 128 + (((l16 & 7) ^ (r0 & 7)) << 4);
    auto fetch = [&](int ch, int s) {
        const int c = (ch0 + ch) * 128 + l16 * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool live = src[j] >= 0 && c < h;
            cp_async16_or_zero(own + s * stage_bytes + j * 32 * 128, x + (live ? (size_t)src[j] * h + c : 0), live);
        }
        cp_async_commit();
    };
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], kQWorkers + 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_free, 4);
        flags[0] = 0;
        fence_barrier_init();
        prefetch_tmap(&tmA);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    const bool run = __ldcg(a.seg.status) == LORA_OK;  // otherwise the product leaves y alone
    if (warp >= 2 && run) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = m0 + r0 + 32 * j;
            src[j] = r < a.seg.n ? __ldcg(a.seg.perm + r) : -1;
        }
        fetch(0, 0);
        fetch(nch > 1 ? 1 : 0, 1);  // (a part of one step starts its second pass in the other stage)
    }
    if (tid < 128) {
        const int t = run && m0 + tid < a.seg.n ? __ldcg(a.seg.perm + m0 + tid) : -1;
        slot_sm[tid] = t >= 0 ? __ldcg(a.seg.idx + t) : -1;
    } else if (tid < 192) {
        seen[tid - 128] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (tid < 128 && slot_sm[tid] >= 0) atomicOr(&seen[slot_sm[tid] >> 5], 1u << (slot_sm[tid] & 31));
    __syncthreads();
    if (tid < 32) {  // words 2 tid and 2 tid + 1
        const uint32_t w0 = seen[2 * tid], w1 = seen[2 * tid + 1];
        int v = __popc(w0) + __popc(w1);
        const int own = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (tid >= d) v += o;
        }
        int at = v - own;
        before[2 * tid] = at;
        for (uint32_t m = w0; m; m &= m - 1) dlist[at++] = 2 * tid * 32 + __ffs(m) - 1;
        before[2 * tid + 1] = at;
        for (uint32_t m = w1; m; m &= m - 1) dlist[at++] = (2 * tid + 1) * 32 + __ffs(m) - 1;
    }
    __syncthreads();
    const int D = before[63] + __popc(seen[63]);
    const int spp = a.cap / R;                     // adapters per pass
    const int passes = (D + spp - 1) / spp;        // 0: no token of the tile has an adapter

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int p = 0; p < passes && !flags[0]; ++p) {
                const int d0 = p * spp, dn = min(spp, D - d0);
                for (int ch = 0; ch < nch; ++ch, ++it) {
                    const int s = it & 1;
                    if (it >= 2 && !mbar_wait(&empty[s], ((it >> 1) & 1) ^ 1, flags)) break;
                    mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(dn * R * 256));
                    uint8_t* As = smem + s * stage_bytes + kQXBytes;
                    for (int d = 0; d < dn; ++d)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_2d_cta(As + hf * a_half + d * R * 128, &tmA, &full[s], (ch0 + ch) * 128 + hf * 64,
                                            dlist[d0 + d] * R);
                }
            }
            if (flags[0]) {
                report_timeout_status(a.seg.status);
                for (int i = max(0, it - 2); i < it; ++i) {
                    const unsigned long long t0 = globaltimer();
                    while (!mbar_try_wait(&full[i & 1], (i >> 1) & 1) && globaltimer() - t0 < kWaitLimitNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int p = 0; p < passes && ok; ++p) {
                const int cols = (min(spp, D - p * spp) * R + 15) / 16 * 16;  // up to 8 more than loaded: not read
                const uint32_t idesc = idesc_f16(128, cols, a.bf16 != 0);
                if (p > 0 && !mbar_wait(acc_free, (p - 1) & 1, flags)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int ch = 0; ch < nch; ++ch, ++it) {
                    const int s = it & 1;
                    if (!mbar_wait(&full[s], (it >> 1) & 1, flags)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t xa = smem_u32(smem + s * stage_bytes), aa = xa + kQXBytes;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        umma_f16(tmem, sdesc_sw128(xa + (k >> 2) * (kQXBytes / 2) + (k & 3) * 32),
                                 sdesc_sw128(aa + (k >> 2) * a_half + (k & 3) * 32), idesc, (ch > 0 || k > 0) ? 1u : 0u);
                    umma_commit(&empty[s]);
                }
                umma_commit(acc_full);
            }
            if (!ok) {
                report_timeout_status(a.seg.status);
                umma_commit(acc_full);
            }
        }
    } else if (run) {
        auto quantise = [&](int ch, const Raw8<T> (&v)[4]) {
            const int c = (ch0 + ch) * 128 + l16 * 8;
            const bool live = c / 32 < a.q.blocks;
            uint32_t codes[4], sw[4];
            if (a.xq_codes) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    codes[j] = sw[j] = 0;
                    if (src[j] < 0) continue;
                    if (live)
                        codes[j] = __ldg(reinterpret_cast<const uint32_t*>(a.xq_codes + (size_t)src[j] * a.q.pitch + c / 2));
                    sw[j] = __ldg(reinterpret_cast<const uint32_t*>(
                        a.xq_scales + ((size_t)(src[j] / 128) * a.q.ktiles + ch0 + ch) * 512 + (src[j] % 32) * 16 +
                        (src[j] % 128) / 32 * 4));
                }
            } else {
                quantise_rows<T, 4>(v, codes, sw, lane);
            }
            uint8_t* out = a.q.codes + (size_t)(m0 + r0) * a.q.pitch + c / 2;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live && src[j] >= 0) *reinterpret_cast<uint32_t*>(out + (size_t)(32 * j) * a.q.pitch) = codes[j];
            if (l16 == 0)
                *reinterpret_cast<uint4*>(a.q.scales + ((size_t)blockIdx.x * a.q.ktiles + ch0 + ch) * 512 + r0 * 16) =
                    make_uint4(sw[0], sw[1], sw[2], sw[3]);
        };
        const int rounds = max(passes, 1);  // the first round quantises
        const int row = (warp & 3) * 32 + lane;
        const int slot = slot_sm[row];
        const int dl = slot >= 0 ? before[slot >> 5] + __popc(seen[slot >> 5] & ((1u << (slot & 31)) - 1u)) : -1;
        const float scale = slot >= 0 ? a.pool.table[slot].scale : 0.f;
        int it = 0;
        bool ok = true;
        for (int p = 0; p < rounds && ok; ++p) {
            for (int ch = 0; ch < nch; ++ch, ++it) {
                const int s = it & 1;
                cp_async_wait<1>();  // this thread's bytes of the step
                Raw8<T> cur[4];
                if (p == 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        cur[j].v = *reinterpret_cast<const uint4*>(own + s * stage_bytes + j * 32 * 128);
                if (passes > 0) {
                    fence_proxy_async_smem();  // read by the tensor cores
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                }
                if (p == 0) quantise(ch, cur);
                // the step two ahead (the next pass starts over) into the same stage
                int next = ch + 2;
                if (next >= nch) next = p + 1 < rounds ? next - nch : -1;
                if (next >= nch) next = 0;  // a part of one step
                if (next >= 0) {
                    if (passes > 0 && !__all_sync(0xffffffffu, mbar_wait(&empty[s], (it >> 1) & 1, flags))) {
                        ok = false;
                        break;
                    }
                    fetch(next, s);
                } else {
                    cp_async_commit();
                }
            }
            if (passes == 0 || warp >= 6) continue;
            // ---- the pass's shrink output: thread <-> token row, the columns of its own adapter ----
            const bool got = __all_sync(0xffffffffu, ok && mbar_wait(acc_full, p & 1, flags));
            if (!got) break;
            tc_fence_after();
            const int d0 = p * spp, dn = min(spp, D - d0);
            const bool mine = dl >= d0 && dl < d0 + dn;
            const int col0 = (dl - d0) * R;
            const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            float* out = a.parts_s + ((size_t)blockIdx.y * a.seg.n + m0 + row) * R;
            for (int c0 = 0; c0 < dn * R; c0 += 16) {
                uint32_t r[16];
                __syncwarp();
                tmem_ld16(taddr + c0, r);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    const int j = c0 + e - col0;
                    if (!mine || j < 0 || j >= R) continue;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = scale * __uint_as_float(r[e + i]);
                    reinterpret_cast<float4*>(out + j)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4*>(out + j)[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_free);
        }
        cp_async_wait<0>();
        if (!ok) report_timeout_status(a.seg.status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, tmem_cols);
    if (a.parts > 1) {
        cluster_sync();  // every part's share is written
        const int chunks = R / 8, per = (128 + a.parts - 1) / a.parts;
        const int q0 = blockIdx.y * per, q1 = min(128, q0 + per);
        for (int e = q0 * chunks + tid; e < q1 * chunks; e += kQThreads) {
            const int row = e / chunks, c = e - row * chunks;
            if (slot_sm[row] < 0) continue;
            const size_t at = (size_t)(m0 + row) * R + c * 8;
            float v[8];
            sum_parts8(a.parts_s + at, a.parts, (size_t)a.seg.n * R, v);
            reinterpret_cast<float4*>(a.s + at)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(a.s + at)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

template <typename T>
static int launch_prepare_t(const PoolView& pv, const SegView& sv, const void* x, const Fp4View* xq, const Fp4View& q,
                            float* parts_s, float* s, cudaStream_t st) {
    PrepArgs a;
    a.pool = pv;
    a.seg = sv;
    a.x = x;
    a.q = q;
    a.xq_codes = xq ? xq->codes : nullptr;
    a.xq_scales = xq ? xq->scales : nullptr;
    a.s = s;
    a.bf16 = std::is_same<T, __nv_bfloat16>::value;
    const int parts = fp4_prepare_parts(sv.n, q.ktiles);
    a.steps = (q.ktiles + parts - 1) / parts;
    a.parts = parts;
    a.parts_s = parts > 1 ? parts_s : s;
    a.cap = prep_cap(sv.n, pv.S, pv.R, (sv.n + 127) / 128 * parts);
    CUtensorMap mA;
    const int rc = make_map(&mA, pv.A, a.bf16, pv.h_in, (uint64_t)pv.S * pv.R, pv.R);
    if (rc) return rc;
    static bool attr = false;
    if (!attr) {
        LORA_CUDA_TRY(cudaFuncSetAttribute(fp4_prepare_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)prep_smem(256)));
        attr = true;
    }
    void* args[] = {(void*)&mA, (void*)&a};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((sv.n + 127) / 128, parts);
    cfg.blockDim = dim3(kQThreads);
    cfg.dynamicSmemBytes = prep_smem(a.cap);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = parts;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    LORA_CUDA_TRY(cudaLaunchKernelExC(&cfg, (const void*)fp4_prepare_kernel<T>, args));
    count_launch();
    return LORA_OK;
}

}  // namespace tc

// K parts (a cluster): as many CTAs as the GPU holds at once, two an SM; a part is at least two steps
// of 128 columns, the last one what is left, at times a single step.
int fp4_prepare_parts(int n, int ktiles) {
    const int tiles = (n + 127) / 128;
    int parts = std::max(1, 2 * num_sms() / tiles);
    parts = std::min({parts, 8, ktiles / 2});
    const int steps = (ktiles + parts - 1) / parts;
    return (ktiles + steps - 1) / steps;
}

int launch_fp4_prepare(const PoolView& pv, const SegView& sv, const void* x, const Fp4View* xq, const Fp4View& q,
                       float* parts_s, float* s, cudaStream_t st) {
    if (pv.dtype == LORA_F16) return tc::launch_prepare_t<__half>(pv, sv, x, xq, q, parts_s, s, st);
    return tc::launch_prepare_t<__nv_bfloat16>(pv, sv, x, xq, q, parts_s, s, st);
}

int launch_fp4_pair(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status, bool early_w,
                    const Fp4Lora* lora, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32: return tc::launch_pair_t<float>(x, w, y, ldy, status, early_w, nullptr, st);
        case LORA_F16: return tc::launch_pair_t<__half>(x, w, y, ldy, status, early_w, lora, st);
        default: return tc::launch_pair_t<__nv_bfloat16>(x, w, y, ldy, status, early_w, lora, st);
    }
}

}  // namespace lora
