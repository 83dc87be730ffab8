// Launchers shared between the library's translation units (host side).
#pragma once
#include "common.cuh"

namespace lora {

// Shrink output layout: s_parts float32 arrays [n, r_max] (original token order); the shrink
// value of token t is scale_s * x[t] A_s^T = sum over parts p of s[p][t][:].  Rows of
// base-only tokens are not written.

// CUDA-core shrink.  Small batches of 16-bit data: one CTA per (sorted token, 8 adapter rows,
// 1024 input features), *s_parts = ceil(h_in / 1024).  tiled: one CTA per (segment, 64 tokens)
// through shared memory, *s_parts = 1.  float32: one warp per (token, rows), *s_parts = 1.
// xready: nonzero for the small-batch kernels ahead of a fused decode GEMM launched with the
// same value (GroupView::xready).
int launch_shrink(const PoolView& pv, const SegView& sv, const void* x, float* s_out, cudaStream_t st, bool tiled,
                  int* s_parts, int xready = 0);
int shrink_parts(const PoolView& pv, int n, bool tiled);
// Whether the small-batch shrink of 16-bit data takes the segmented kernel (A rows read once per
// work item) rather than the per-token one.
int shrink_segmented(const PoolView& pv, int n);
// The same for the slices of a group (16-bit data, not tiled): slice q's output starts at
// s_out + q * grp.s_stride.  One launch covers every slice.
int launch_shrink_group(const PoolView& pv, const GroupView& grp, const SegView& sv, const void* x, float* s_out,
                        cudaStream_t st, bool tiled, int* s_parts);

// Whether the fused tensor-core decode GEMM (n <= 256) holds every adapter's B rows a CTA can
// need in shared memory during its main loop (the variant policy keys on this).
int decode_fused_fits(const PoolView& pv, int n);

// y[t, :] += s[t, :] B_s^T (separate variant's residual kernel).
int launch_expand(const PoolView& pv, const SegView& sv, const float* s_in, int s_parts, void* y, cudaStream_t st);
// The same for the slices of a group (16-bit data): y has row stride grp.ldy, slice q owns
// columns [grp.col[q], grp.col[q + 1]).  One launch covers every slice.
int launch_expand_group(const PoolView& pv, const GroupView& grp, const SegView& sv, const float* s_in, int s_parts,
                        void* y, cudaStream_t st);

// CUDA-core base GEMM y = x W^T (+ fused expand when fuse).
int launch_gemm_simt(const PoolView& pv, const SegView& sv, const void* W, const void* x, const float* s_in,
                     int s_parts, void* y, bool fuse, cudaStream_t st);

// Tensor-core (tcgen05) base GEMM with optional fused expand.
//   decode path  (n <= 256): W tiles on the MMA M side, tokens on N, split-K across the CTAs
//                 of a thread-block cluster, reduced through distributed shared memory.
//   prefill path (n > 256):  token tiles on M (128), outputs on N (256), persistent CTAs.
int tc_supported(const PoolView& pv, int n);
// prefetch/prefetch_bytes: optional device range the decode kernel streams into L2 after its
// own loads (ignored by the prefill kernel).
// grp: output slices of a group (nullptr: the single linear of pv).  pv.h_out is then the
// concatenated width; y has row stride grp->ldy.  The prefill kernel applies every slice's
// LoRA term; the decode kernel takes one slice with fuse, or several without the LoRA term
// (a single slice may also be a column range of a wider y: pv.h_out < grp->ldy).
// xready: nonzero when the shrink kernel just before this fused decode GEMM was launched with
// the same value: the GEMM then streams its weight from its start and reads x once the shrink
// has published the value.
int launch_gemm_tc(const PoolView& pv, const SegView& sv, const void* W, const void* x, const float* s_in, int s_parts,
                   void* y, bool fuse, cudaStream_t st, const void* prefetch = nullptr, size_t prefetch_bytes = 0,
                   const GroupView* grp = nullptr, int xready = 0);

// The launch sequence of one LoRA-augmented linear (lora_linear_fwd and its variants), after the
// caller's arguments were checked; s_buf receives the shrink output.
int linear_fwd_impl(lora_pool_t pool, const void* W_dev, const void* x_dev, void* y_dev, const lora_segments* seg,
                    int variant, float* s_buf, const void* prefetch_dev, size_t prefetch_bytes, cudaStream_t st);

// Base GEMM y = x W^T (no LoRA term) with 256 W rows per CTA, two M=128 MMAs sharing each x
// tile, full K per CTA (batches of up to 256 tokens); y has row stride ldy.
int launch_gemm_tall(const PoolView& pv, const SegView& sv, const void* W, const void* x, void* y, int ldy,
                     cudaStream_t st);

// Grouped tcgen05 shrink for batches of more than 256 tokens (one CTA per 128-token tile).
int shrink_tc_supported(const PoolView& pv);
int launch_shrink_tc(const PoolView& pv, const SegView& sv, const void* x, float* s_out, cudaStream_t st);
// The same for the slices of a group in one launch (count * r_max <= 256): slice q's output
// starts at s_out + q * grp.s_stride.
int shrink_tc_group_supported(const PoolView& pv, int count);
int launch_shrink_tc_group(const PoolView& pv, const GroupView& grp, const SegView& sv, const void* x, float* s_out,
                           cudaStream_t st);

// A stored 4-bit matrix as the kernels see it (layout in lora.h).
struct Fp4View {
    uint8_t* codes;
    uint8_t* scales;
    int rows, cols;
    int blocks;     // blocks of 32 per row
    int ktiles;     // scale tiles per 128 rows (KT)
    size_t pitch;   // bytes per row of codes
};
inline Fp4View fp4_view(void* codes, void* scales, int rows, int cols) {
    Fp4View v;
    v.codes = static_cast<uint8_t*>(codes);
    v.scales = static_cast<uint8_t*>(scales);
    v.rows = rows;
    v.cols = cols;
    v.blocks = (cols - 1) / 32 + 1;
    v.ktiles = 2 * ((cols - 1) / 256 + 1);
    v.pitch = (size_t)v.blocks * 16;
    return v;
}
inline size_t fp4_codes_bytes(int rows, int cols) { return (size_t)rows * ((cols - 1) / 32 + 1) * 16; }
inline size_t fp4_scales_bytes(int rows, int cols) {
    return (size_t)((rows + 127) / 128) * (2 * ((cols - 1) / 256 + 1)) * 512;
}
int launch_fp4_quantize(const void* x, int dtype, long long ld, const Fp4View& q, cudaStream_t st);
// y = x w^T (dtype, row stride ldy).  status: nullable device word; y stays untouched unless it is
// LORA_OK.  early_w: every kernel that could have written w has completed when this grid starts (the
// products inside a linear; only these release the kernel behind them early).
// lora (nullable, 16-bit y): the LoRA term, for launch_fp4_pair with x's rows in the order of perm.
struct Fp4Lora {
    const int32_t* perm;  // token of each row of x
    const int32_t* idx;   // slot of each token
    const float* s;       // [n][R], rows like x's
    const void* B;
    int R;
};
// Up to 256 tokens.  early: every kernel that could have written w (1), or w and x (2), has completed when
// this grid starts; the rest is waited for.  lora: the pool, the slot of each token and the shrink output in K parts.
struct Fp4DecodeLora {
    const PoolView* pool;
    const int32_t* idx;
    const float* s_in;
    int s_parts;
};
int fp4_decode_splits(int h_out, int h_in);
int launch_fp4_decode(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status,
                      int early, const Fp4DecodeLora* lora, cudaStream_t st);
// The kernel before it for small batches: x quantised into q (nullptr: not) and the shrink output in
// *s_parts K parts, in one launch (pools of any type whose adapters the per-token shrink suits).
int launch_fp4_front(const PoolView& pv, const SegView& sv, const void* x, const Fp4View* q, float* s_out, int* s_parts,
                     cudaStream_t st);
// float32 pools: the shrink in K parts (s_out [f32_shrink_parts][n][R]), and y += s B^T.
int f32_shrink_parts(const PoolView& pv, int n);
int launch_f32_shrink(const PoolView& pv, const SegView& sv, const void* x, float* s_out, cudaStream_t st);
int launch_f32_expand(const PoolView& pv, const SegView& sv, const float* s_in, int s_parts, void* y, cudaStream_t st);
// More than 256 tokens.
int launch_fp4_pair(const Fp4View& x, const Fp4View& w, void* y, int dtype, long long ldy, int32_t* status, bool early_w,
                    const Fp4Lora* lora, cudaStream_t st);
// Quantises x (or copies xq) into q and writes the shrink output to s [n][R], rows of both in segment order;
// parts_s: scratch [fp4_prepare_parts][n][R], not used where that is one part.
int fp4_prepare_parts(int n, int ktiles);
int launch_fp4_prepare(const PoolView& pv, const SegView& sv, const void* x, const Fp4View* xq, const Fp4View& q,
                       float* parts_s, float* s, cudaStream_t st);

int num_sms();

}  // namespace lora
