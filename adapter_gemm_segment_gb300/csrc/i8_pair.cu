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
// The LoRA term is one more accumulator of a tile that meets adapters.  Tokens come in the order of the
// segments, so a tile meets few: for its distinct adapters d, K columns d * r_max + j hold B_d[o, j] on the
// feature side and s[t, j] on the token side (zero unless t uses d), kind::tf32, 8 columns a block.  B is a
// tf32 number exactly; s goes in as two (22 bits), each multiplying the same B.  0 * inf would carry an
// infinity or NaN of one tenant's B to the other tokens of the tile: such elements are replaced by zeros and
// added to their own tokens by the warps that drain the accumulators.
//
// Warps: 0 loads, 1 issues MMAs (even CTA), 4-7 build LoRA blocks, 8-15 drain: lane <-> feature, every second
// 16 tokens.  y is stored from the registers: the MMAs' operands arrive (64 KB every 512 clocks) and are read at
// the rate of the shared-memory port, which would make staging there wait.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "fp4_device.cuh"
#include "i8_device.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace lora {
namespace tc {

using namespace ptx;

constexpr int kJM = 128;           // features per CTA
constexpr int kJMaxN = 256;        // tokens per pair tile, at most
constexpr int kJThreads = 512;
// registers a thread of the warpgroups 0, 1 and 2-3: together what the block is launched with, 128 a thread.  (With
// 192 the drain spills: the prefill batch of 16384 x 4096 x 4096 with rank 16 took 478 us instead of 437.)
constexpr int kJRegs0 = 56, kJRegs1 = 56, kJRegs2 = 200;
static_assert(kJRegs0 + kJRegs1 + 2 * kJRegs2 == 4 * 128, "register split");
constexpr int kJChunk = 16;        // steps of 64 codes between two readings of the accumulator
constexpr uint32_t kJWBytes = kJM * 128;
constexpr int kJMaxStages = 8;
constexpr int kJUnits = kJMaxN / 32;  // 16-token units of a drain warp, at most
// a LoRA block: 8 columns of B for 128 features, then of s in two parts for N / 2 <= 128 tokens
constexpr int kJBufs = 4;  // blocks ahead of the MMAs: a tile of two adapters of rank 16 takes four
constexpr int kJLoraB = kJM * 32, kJLoraBytes = kJLoraB + 2 * (kJMaxN / 2) * 32;
constexpr size_t kJTail = kJMaxN * 16 + 64 * 4 + 256 * 4 + 16 + 512 + 1024;
constexpr size_t kJSmemMax = 227 * 1024;

struct I8PairArgs {
    void* y;
    int32_t* status;       // nullable
    const int32_t* perm;   // row of y of each row of x (nullable without the LoRA term)
    const float* sx;
    const float* sw;
    long long ldy;
    int n, N, h_out, m_tiles, n_tiles, nkb, stages, release, pairs;
    // the LoRA term (FUSE)
    const SlotEntry* table;
    const void* B;
    const int32_t* idx;    // by token
    const float* s;        // [n][R], by token
    int R;
};

// s = hi + lo to 2^-23 of itself, both tf32 numbers; an infinity or NaN stays in hi.
__device__ __forceinline__ void split_tf32(float s, uint32_t& hi, uint32_t& lo) {
    const uint32_t b = __float_as_uint(s);
    if ((b & 0x7f800000u) == 0x7f800000u) {
        hi = b;
        lo = 0;
        return;
    }
    hi = (b + 0x1000u) & 0xffffe000u;
    if ((hi & 0x7f800000u) == 0x7f800000u) hi = b & 0xffffe000u;  // (it rounded up to an infinity)
    lo = (__float_as_uint(s - __uint_as_float(hi)) + 0x1000u) & 0xffffe000u;
}

// Adds to y what the LoRA blocks left out: the products of B's infinities and NaN.
template <typename T> __device__ __noinline__ void add_bad(const I8PairArgs& a, int slot, int row, int o) {
    const T* b = static_cast<const T*>(a.B) + ((size_t)slot * a.h_out + o) * a.R;
    float acc = 0.f;
    for (int j = 0; j < a.table[slot].rank; ++j) {
        const float f = to_f32<T>(b[j]);
        if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) acc = fmaf(f, a.s[(size_t)row * a.R + j], acc);
    }
    T* y = static_cast<T*>(a.y) + (long long)row * a.ldy + o;
    if (acc != 0.f) *y = from_f32<T>(to_f32<T>(*y) + acc);
}

template <typename T, bool FUSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kJThreads, 1)
i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8PairArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align(smem_raw, 1024);
    const int stages = a.stages, N = a.N;
    const uint32_t stage_bytes = kJWBytes + static_cast<uint32_t>(N) * 64;  // 128 features, N / 2 tokens of 64 float16
    uint8_t* lora_sm = smem + stages * stage_bytes;              // [kJBufs] blocks
    int* row_sm = reinterpret_cast<int*>(lora_sm + (FUSE ? kJBufs * kJLoraBytes : 0));  // [N] row of y of a token of the tile
    int* slot_sm = row_sm + kJMaxN;                              // [N] its adapter
    float* sx_sm = reinterpret_cast<float*>(slot_sm + kJMaxN);   // [N] its scale
    float* up_sm = sx_sm + kJMaxN;                               // [N] and what its product is multiplied by
    uint32_t* seen = reinterpret_cast<uint32_t*>(up_sm + kJMaxN);  // [64] slots the tile's tokens name
    int* dlist = reinterpret_cast<int*>(seen + 64);              // [256] in order
    int* distinct = dlist + 256;                                 // [2] their number
    uint64_t* full = reinterpret_cast<uint64_t*>(distinct + 4);  // even CTA: both CTAs' halves landed
    uint64_t* empty = full + kJMaxStages;      // (multicast)
    uint64_t* acc_full = empty + kJMaxStages;  // [2] (multicast)
    uint64_t* acc_empty = acc_full + 2;        // [2] even CTA (8 warps of both CTAs)
    uint64_t* lora_own = acc_empty + 2;        // [kJBufs] a LoRA block of this CTA is written (4 warps)
    uint64_t* lora_peer = lora_own + kJBufs;   // [kJBufs] even CTA: the odd CTA's block is written (relayed)
    uint64_t* lora_empty = lora_peer + kJBufs;  // [kJBufs] (multicast)
    // by parity of the tile (the warps that build blocks may be a tile ahead of the others):
    uint64_t* linfo = lora_empty + kJBufs;          // [2] the tile's number of LoRA blocks is known
    uint64_t* tile_done = linfo + 2;           // [2] it has been used (8 drain warps, the MMA or relay thread)
    uint64_t* drained = tile_done + 2;         // even CTA: every MMA has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    // abort, -, then by parity of the tile: [2] LoRA blocks, [2] 1 + the last tile whose blocks left products out
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kJMaxStages + 3 * kJBufs + 9) * 8 + 28 <= 512, "barrier area");

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
            mbar_init(&linfo[b], 1);
            mbar_init(&tile_done[b], 9);
        }
        for (int b = 0; b < kJBufs; ++b) {
            mbar_init(&lora_own[b], 4);
            mbar_init(&lora_peer[b], 1);
            mbar_init(&lora_empty[b], 1);
        }
        mbar_init(drained, 1);
        for (int i = 0; i < 6; ++i) flags[i] = 0;
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
    if (warp < 4) {
        registers_down<kJRegs0>();
        if (warp == 0 && lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            pdl_wait();
            int it = 0, s = 0;
            uint32_t ph = 0;
            for (int tile = pair; tile < total && !flags[0]; tile += npairs) {
                const int m0 = tile % a.m_tiles * 2 * kJM + static_cast<int>(rank) * kJM;
                const int n0 = tile / a.m_tiles * N + static_cast<int>(rank) * (N / 2);
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    if (it >= stages && !mbar_wait(&empty[s], ph ^ 1, flags)) break;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
                    const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                    tma_load_2d_pair(smem + s * stage_bytes, &tmW, bar, kb * 64, m0);
                    tma_load_2d_pair(smem + s * stage_bytes + kJWBytes, &tmX, bar, kb * 64, n0);
                    if (++s == stages) s = 0, ph ^= 1;
                }
            }
            if (flags[0]) {  // aborted: give the copies in flight (both CTAs') time to land
                if (a.status) report_timeout_status(a.status);
                const unsigned long long t0 = globaltimer();
                while (globaltimer() - t0 < kWaitLimitNs / 8) {
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_f16(2 * kJM, N, false), idesc_lora = idesc_tf32(2 * kJM, N);
            bool ok = true;
            int s = 0, chunk = 0, local = 0, lb = 0;
            uint32_t ph = 0;
            for (int tile = pair; tile < total && ok; tile += npairs, ++local) {
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
                if constexpr (FUSE) {
                    if (!ok) break;
                    if (!mbar_wait(&linfo[local & 1], (local >> 1) & 1, flags)) {
                        ok = false;
                        break;
                    }
                    const int blocks = flags[2 + (local & 1)];
                    mbar_arrive(&tile_done[local & 1]);
                    if (blocks == 0) continue;
                    const int buf = chunk & 1;
                    if (chunk >= 2 && !mbar_wait(&acc_empty[buf], ((chunk >> 1) & 1) ^ 1, flags)) {
                        ok = false;
                        break;
                    }
                    ++chunk;
                    for (int b = 0; b < blocks; ++b, ++lb) {
                        const int lbuf = lb % kJBufs;
                        if (!mbar_wait(&lora_own[lbuf], (lb / kJBufs) & 1, flags) ||
                            !mbar_wait_cluster(&lora_peer[lbuf], (lb / kJBufs) & 1, flags)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t ba = smem_u32(lora_sm + lbuf * kJLoraBytes), sa = ba + kJLoraB;
                        const uint32_t half = static_cast<uint32_t>(N) * 16;  // a part of s: N / 2 tokens
#pragma unroll
                        for (uint32_t k = 0; k < 2; ++k)
                            umma_pair_tf32(tmem + buf * N, sdesc_chunks(ba, kJM * 16), sdesc_chunks(sa + k * half, half / 2),
                                           idesc_lora, (b > 0 || k > 0) ? 1u : 0u);
                        umma_pair_commit(&lora_empty[lbuf], 0x3);
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
        } else if (FUSE && warp == 1 && lane == 0) {
            // odd CTA: tells the even one that a LoRA block is written.  (A release at cluster scope waits for every
            // access of its thread: this thread's, not the writers'.)
            const uint32_t peer0 = mapa_shared(smem_u32(lora_peer), 0);
            int local = 0, lb = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += npairs, ++local) {
                ok = mbar_wait(&linfo[local & 1], (local >> 1) & 1, flags);
                const int blocks = ok ? flags[2 + (local & 1)] : 0;
                if (ok) mbar_arrive(&tile_done[local & 1]);
                for (int b = 0; b < blocks && ok; ++b, ++lb) {
                    ok = mbar_wait(&lora_own[lb % kJBufs], (lb / kJBufs) & 1, flags);
                    if (ok) mbar_arrive_cluster(peer0 + static_cast<uint32_t>(lb % kJBufs) * 8u);
                }
            }
            if (!ok && a.status) report_timeout_status(a.status);
        }
    } else if (warp < 8) {
        registers_down<kJRegs1>();
        if constexpr (FUSE) {
            // ---- LoRA blocks: a feature of this CTA and a token of its half a thread ----
            const int lt = threadIdx.x - 128;
            pdl_wait();
            const bool st_ok = !a.status || __ldcg(a.status) == LORA_OK;
            const int chunks = a.R / 8;
            int local = 0, lb = 0;
            bool ok = true;
            for (int tile = pair; tile < total; tile += npairs, ++local) {
                const int n0 = tile / a.m_tiles * N;
                // the slots of the tile's tokens: this thread's of its CTA's half, then of the other's
                int slot[2], tok = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = n0 + static_cast<int>(rank ^ h) * (N / 2) + lt;
                    slot[h] = -1;
                    if (lt < N / 2 && r < a.n && st_ok) {
                        const int t = __ldcg(a.perm + r);
                        slot[h] = __ldcg(a.idx + t);
                        if (h == 0) tok = t;
                    }
                }
                const int own_rank = slot[0] >= 0 ? a.table[slot[0]].rank : 0;
                if (lt < 64) seen[lt] = 0;
                // this parity's count and flag, of the tile two before, have been used
                if (local >= 2 && !mbar_wait(&tile_done[local & 1], ((local >> 1) & 1) ^ 1, flags)) ok = false;
                if (!named_bar_and(4, 128, ok)) {  // all four warps leave together
                    ok = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (slot[h] >= 0) atomicOr(&seen[slot[h] >> 5], 1u << (slot[h] & 31));
                named_bar_sync(4, 128);
                if (lt < 64) {
                    int at = 0;
                    for (int w = 0; w < lt; ++w) at += __popc(seen[w]);
                    for (uint32_t m = seen[lt]; m; m &= m - 1) dlist[at++] = lt * 32 + __ffs(m) - 1;
                    if (lt == 63) *distinct = at;
                }
                named_bar_sync(4, 128);
                const int blocks = *distinct * chunks;
                if (lt == 0) {
                    flags[2 + (local & 1)] = blocks;
                    mbar_arrive(&linfo[local & 1]);
                }
                const int o = tile % a.m_tiles * 2 * kJM + static_cast<int>(rank) * kJM + lt;
                const float* srow = a.s + (size_t)tok * a.R;
                const T* Bcol = static_cast<const T*>(a.B) + (size_t)o * a.R;
                int d = 0, c = 0;  // the next block: columns 8c.. of adapter dlist[d]
                struct Block {     // this thread's token and feature of a block
                    float4 s[2];
                    uint4 b;
                } now, next;
                auto load = [&](Block& v) {
                    const int sl = dlist[d];
                    const bool mine = sl == slot[0] && c * 8 < own_rank;
                    const float4* sp = reinterpret_cast<const float4*>(srow + c * 8);
                    v.s[0] = v.s[1] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (mine) v.s[0] = __ldcg(sp), v.s[1] = __ldcg(sp + 1);
                    v.b = o < a.h_out ? __ldg(reinterpret_cast<const uint4*>(Bcol + (size_t)sl * a.h_out * a.R + c * 8))
                                      : make_uint4(0, 0, 0, 0);
                    // (columns past the rank: B's are zeros, s may not have been written)
                    if (mine && c * 8 + 8 > own_rank) {
                        float* f = reinterpret_cast<float*>(v.s);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c * 8 + e >= own_rank) f[e] = 0.f;
                    }
                    if (++c == chunks) c = 0, ++d;
                };
                if (blocks > 0) load(next);
                for (int b = 0; b < blocks; ++b, ++lb) {
                    now = next;
                    if (b + 1 < blocks) load(next);  // a block ahead
                    if (lb >= kJBufs && !__all_sync(0xffffffffu, mbar_wait(&lora_empty[lb % kJBufs], ((lb / kJBufs) & 1) ^ 1, flags))) {
                        ok = false;
                        break;
                    }
                    uint8_t* blk = lora_sm + (lb % kJBufs) * kJLoraBytes;
                    if (nonfinite8<T>(now.b)) {
                        now.b = finite8<T>(now.b);
                        flags[4 + (local & 1)] = local + 1;
                    }
                    float bf[8];
                    unpack8<T>(now.b, bf);
                    uint4* fb = reinterpret_cast<uint4*>(blk + lt * 16);
                    fb[0] = make_uint4(__float_as_uint(bf[0]), __float_as_uint(bf[1]), __float_as_uint(bf[2]), __float_as_uint(bf[3]));
                    fb[kJM] = make_uint4(__float_as_uint(bf[4]), __float_as_uint(bf[5]), __float_as_uint(bf[6]), __float_as_uint(bf[7]));
                    if (lt < N / 2) {
                        const float f[8] = {now.s[0].x, now.s[0].y, now.s[0].z, now.s[0].w,
                                            now.s[1].x, now.s[1].y, now.s[1].z, now.s[1].w};
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) split_tf32(f[e], hi[e], lo[e]);
                        uint4* sb = reinterpret_cast<uint4*>(blk + kJLoraB + lt * 16);
                        const int q = N / 2;  // rows of a chunk of 16 bytes
                        sb[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        sb[q] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                        sb[2 * q] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        sb[3 * q] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                    }
                    fence_proxy_async_smem();  // read by the tensor cores
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&lora_own[lb % kJBufs]);
                }
                if (!ok) flags[0] = 1;
            }
            if (!ok && a.status && lane == 0) report_timeout_status(a.status);
        }
    } else {
        registers_up<kJRegs2>();
        // ---- drain ----
        const int q = warp & 3, hv = (warp - 8) >> 2, lt = threadIdx.x - 256;
        const int units = N / 16;
        const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
        pdl_wait();
        const bool store = !a.status || __ldcg(a.status) == LORA_OK;
        T* y = static_cast<T*>(a.y);
        int chunk = 0, local = 0;
        bool ok = true;
        struct {
            int row, slot;
            float sx;
        } next = {-1, -1, 0.f};
        auto look_up = [&](int tile) {  // token lt of the tile
            const int r = tile / a.m_tiles * N + lt;
            const bool live = lt < N && r < a.n && store;
            next.row = !live ? -1 : a.perm ? __ldcg(a.perm + r) : r;
            next.sx = live ? __ldcg(a.sx + r) : 0.f;
            if constexpr (FUSE) next.slot = live ? __ldcg(a.idx + next.row) : -1;
        };
        if (pair < total) look_up(pair);
        for (int tile = pair; tile < total; tile += npairs, ++local) {
            const int o = tile % a.m_tiles * 2 * kJM + static_cast<int>(rank) * kJM + q * 32 + lane;
            named_bar_sync(2, 256);  // the tile before is through with the tokens' rows
            if (lt < N) {
                row_sm[lt] = next.row;
                // (a scale that its sum could carry past float32's range is taken down by a power of two, and the product
                // with sw up again: see i8_scaled.  With the LoRA term that is one instruction, as the addition by itself)
                const bool large = i8_large(next.sx);
                sx_sm[lt] = large ? next.sx * 0x1p-64f : next.sx;
                up_sm[lt] = large ? 0x1p64f : 1.f;
                if constexpr (FUSE) slot_sm[lt] = next.slot;
            }
            const float sw = o < a.h_out ? __ldg(a.sw + o) : 0.f;
            const bool lora = FUSE && !named_bar_and(2, 256, next.slot < 0);
            if constexpr (!FUSE) named_bar_sync(2, 256);
            if (tile + npairs < total) look_up(tile + npairs);
            bool large_sx = false;
            if constexpr (!FUSE) {
                for (int t = lane; t < N; t += 32) large_sx = large_sx || up_sm[t] != 1.f;
                large_sx = __any_sync(0xffffffffu, large_sx);
            }
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
            const int lbuf = chunk & 1;
            bool left_out = false;
            if (lora && ok) {
                ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[lbuf], (chunk >> 1) & 1, flags));
                ++chunk;
                tc_fence_after();
                left_out = flags[4 + (local & 1)] == local + 1;
            }
            // all eight warps leave together
            if (!named_bar_and(3, 256, ok)) {
                ok = false;
                break;
            }
            // values first, which leaves the LoRA accumulator to the next tile's MMAs, then the stores
            const uint32_t laddr = tmem + lbuf * N + (static_cast<uint32_t>(q * 32) << 16);
            auto values = [&](auto large) {
#pragma unroll
                for (int i = 0; i < kJUnits; ++i) {
                    const int u = 2 * i + hv;
                    if (u < units) {
                        uint32_t r[16];
                        if (lora) {
                            __syncwarp();
                            tmem_ld16(laddr + u * 16, r);
                            tmem_ld_wait();
                        }
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 sx = *reinterpret_cast<const float4*>(sx_sm + u * 16 + e);
                            const float4 up = large ? *reinterpret_cast<const float4*>(up_sm + u * 16 + e) : make_float4(1.f, 1.f, 1.f, 1.f);
                            const float s4[4] = {sx.x, sx.y, sx.z, sx.w}, u4[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float v = __int2float_rn(sum[i][e + k]) * s4[k] * sw;
                                sum[i][e + k] = __float_as_int(lora ? fmaf(v, u4[k], __uint_as_float(r[e + k])) : large ? v * u4[k] : v);
                            }
                        }
                    }
                }
            };
            if (FUSE || large_sx)
                values(std::true_type{});
            else
                values(std::false_type{});
            if constexpr (FUSE) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && lora) mbar_arrive_cluster_relaxed(acc_empty0 + static_cast<uint32_t>(lbuf) * 8u);
            }
#pragma unroll 1
            for (int i = 0; i < kJUnits; ++i) {
                const int u = 2 * i + hv;
                if (u >= units || !store) break;
                float v[16];
#pragma unroll
                for (int j = 0; j < kJUnits; ++j)
                    if (j == i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __int_as_float(sum[j][e]);
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int row = row_sm[u * 16 + e];
                        if (row >= 0 && o < a.h_out) y[(long long)row * a.ldy + o] = v[e];
                    }
                } else if (a.pairs) {
                    // neighbouring lanes exchange a value: an even lane then has two features of one token, an odd one of
                    // the next
                    const bool odd = lane & 1;
                    const int oe = o & ~1;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[e + 1], 1);
                        const uint32_t w = odd ? pack2<T>(other, v[e + 1]) : pack2<T>(v[e], other);
                        const int row = row_sm[u * 16 + e + (odd ? 1 : 0)];
                        if (row < 0) continue;
                        T* yp = y + (long long)row * a.ldy + oe;
                        if (oe + 1 < a.h_out)
                            *reinterpret_cast<uint32_t*>(yp) = w;
                        else if (oe < a.h_out)
                            *reinterpret_cast<uint16_t*>(yp) = static_cast<uint16_t>(w);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int row = row_sm[u * 16 + e];
                        if (row >= 0 && o < a.h_out) y[(long long)row * a.ldy + o] = from_f32<T>(v[e]);
                    }
                }
            }
            if constexpr (FUSE) {
                __syncwarp();
                if (left_out && store && o < a.h_out)
#pragma unroll 1
                    for (int t = 0; t < N; ++t)  // this warp's tokens: infinities and NaN onto what it has stored
                        if ((t / 16 & 1) == hv && slot_sm[t] >= 0) add_bad<T>(a, slot_sm[t], row_sm[t], o);
                __syncwarp();
                if (lane == 0) mbar_arrive(&tile_done[local & 1]);
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
    a.pairs = reinterpret_cast<uintptr_t>(y) % 4 == 0 && ldy % 2 == 0;  // 16-bit y: two features at a time
    // tokens a tile: what the rounds of all pairs take, with 48 tokens' time a tile for what does not shrink with it
    const int pairs = max_pairs();
    long long best = LLONG_MAX;
    for (int N = kJMaxN; N >= 96; N -= 32) {
        const long long tiles = (long long)a.m_tiles * ((x.rows + N - 1) / N), cost = (tiles + pairs - 1) / pairs * (N + 48);
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
    const size_t stage_bytes = kJWBytes + (size_t)a.N * 64, tail = kJTail + (FUSE ? kJBufs * kJLoraBytes : 0);
    a.stages = (int)std::min<size_t>((kJSmemMax - tail) / stage_bytes, kJMaxStages);
    CUtensorMap mW, mX;
    int rc = make_map(&mW, w.x16, 0, pitch, w.rows, kJM);
    if (!rc) rc = make_map(&mX, x.x16, 0, pitch, x.rows, a.N / 2);
    if (rc) return rc;
    void* args[] = {(void*)&mW, (void*)&mX, (void*)&a};
    LORA_CUDA_TRY(launch_pdl((const void*)i8_pair_kernel<T, FUSE>, dim3(2 * (unsigned)std::min<long long>(tiles, pairs)),
                             dim3(kJThreads), a.stages * stage_bytes + tail, st, args));
    return LORA_OK;
}

}  // namespace tc

int launch_i8_pair(const I8Rows& x, const I8Rows& w, void* y, int dtype, long long ldy, int32_t* status, bool release,
                   const I8Lora* lora, cudaStream_t st) {
    switch (dtype) {
        case LORA_F32: return tc::launch_pair_t<float, false>(x, w, y, ldy, status, release, nullptr, st);
        case LORA_F16:
            return lora ? tc::launch_pair_t<__half, true>(x, w, y, ldy, status, release, lora, st)
                        : tc::launch_pair_t<__half, false>(x, w, y, ldy, status, release, nullptr, st);
        default:
            return lora ? tc::launch_pair_t<__nv_bfloat16, true>(x, w, y, ldy, status, release, lora, st)
                        : tc::launch_pair_t<__nv_bfloat16, false>(x, w, y, ldy, status, release, nullptr, st);
    }
}

}  // namespace lora
