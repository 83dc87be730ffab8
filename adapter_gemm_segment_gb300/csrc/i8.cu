// Entry points of the 8-bit integer matrices: sizes, checks of arguments, and the choice of kernels.
#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace lora {

// 128 x 128 x cols stays below 2^31
constexpr int kI8MaxCols = 131071;
// rows in tiles of up to 256, counted in 32 bits
constexpr int kI8MaxRows = INT_MAX - 255;

static int check_shape(int rows, int cols) {
    if (rows < 0 || cols < 1) return set_error(LORA_EINVAL, "8-bit matrix of %d x %d", rows, cols);
    if (cols > kI8MaxCols) return set_error(LORA_EUNSUP, "8-bit matrix of %d columns (at most %d)", cols, kI8MaxCols);
    if (rows > kI8MaxRows) return set_error(LORA_EUNSUP, "8-bit matrix of %d rows (at most %d)", rows, kI8MaxRows);
    return LORA_OK;
}

static int check_matrix(const lora_i8_matrix* m, const char* what) {
    if (!m) return set_error(LORA_EINVAL, "%s is NULL", what);
    const int rc = check_shape(m->rows, m->cols);
    if (rc || m->rows == 0) return rc;
    if (!m->codes_dev || !m->scales_dev) return set_error(LORA_EINVAL, "%s has no codes or scales", what);
    if ((reinterpret_cast<uintptr_t>(m->codes_dev) | reinterpret_cast<uintptr_t>(m->scales_dev)) % 256)
        return set_error(LORA_EINVAL, "%s: codes and scales must be 256-byte aligned", what);
    return LORA_OK;
}

static int check_dtype(int dtype) {
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return set_error(LORA_EINVAL, "bad dtype %d", dtype);
    return LORA_OK;
}

// A strided [rows, cols] array of dtype.
static int check_rows(const void* p, int dtype, int64_t ld, int rows, int cols, const char* what) {
    const int rc = check_dtype(dtype);
    if (rc) return rc;
    if (ld < cols) return set_error(LORA_EINVAL, "%s: row stride %lld below %d columns", what, (long long)ld, cols);
    if (rows == 0) return LORA_OK;
    if (!p) return set_error(LORA_EINVAL, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % dtype_size(dtype)) return set_error(LORA_EINVAL, "%s is misaligned", what);
    return LORA_OK;
}

// Whether an output [rows, cols] meets another array of the same element size, in elements other than (may: or in) the
// ones of the same index.  Distances in elements; lda, ldb >= cols.
static bool meets(const void* out, int64_t lda, const void* other, int64_t ldb, int rows, int cols, size_t elt, bool may) {
    if (!out || !other) return false;
    // (both are aligned to their element: the distance is a whole number of them)
    const int64_t d = (reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(other)) / (int64_t)elt, last = rows - 1;
    if (d > last * ldb + cols - 1 || -d > last * lda + cols - 1) return false;
    if (lda == ldb || rows == 1) {  // every row the same: out's row r is k rows and c columns behind other's
        if (d == 0) return !may;
        const int64_t k = d >= 0 ? d / ldb : -((-d + ldb - 1) / ldb), c = d - k * ldb;
        const int64_t behind = k >= 0 ? k : -k, next = k + 1 >= 0 ? k + 1 : -(k + 1);
        return (c < cols && behind <= last) || (c > ldb - cols && next <= last);
    }
    for (int64_t r = 0; r <= last; ++r) {
        const int64_t at = d + r * lda;  // of out's row r, from other's first element
        const int64_t k = at >= 0 ? at / ldb : -1, c = at - k * ldb;
        if (k >= 0 && k <= last && c < cols && !(may && k == r && c == 0)) return true;
        if (c > ldb - cols && k + 1 >= 0 && k + 1 <= last) return true;
        if (k > last) break;
    }
    return false;
}

static I8View view_of(const lora_i8_matrix* m) { return i8_view(m->codes_dev, m->scales_dev, m->rows, m->cols); }

// Up to this many tokens the dot products of i8_small.cu.  (4096 x 4096 float16, us, these / the tile kernel: 1 token
// 5.3 / 9.8, 8 tokens 6.9 / 10.3, 9 tokens 23.4 / 10.4; 8 tokens to 11008 features 17.2 / 19.5.)
constexpr int kI8Small = 8;

// Above this many tokens the pair kernel, for which the weight is turned into float16 first.  (Tile / pair, us: 512
// tokens 4096 x 4096 24.2 / 38.0, 11008 x 4096 48 / 86, 1024 x 1024 10.6 / 14.3, 4096 x 4096 over 100 adapters of rank 8
// 36.9 / 53.8.  Further up products still gain, 768 tokens 4096 x 4096 33 / 41, linears do not: 63 / 61.)
constexpr int kI8Tile = 512;

// What a product keeps in its workspace: x in float16 codes and its scales, and above kI8Tile rows the weight
// in float16 codes.
struct I8ProductWs {
    size_t scales_off, w_off, total;
};
static I8ProductWs product_ws(int n, int h_out, int h_in) {
    I8ProductWs L = {0, 0, 0};
    if (n <= kI8Small) return L;
    L.scales_off = align256((size_t)n * i8_pitch(h_in) * 2);
    L.w_off = L.scales_off + 2 * align256((size_t)n * 4);  // scales, peaks
    L.total = L.w_off + (n > kI8Tile ? align256((size_t)h_out * i8_pitch(h_in) * 2) : 0);
    return L;
}

// Batches of more than 512 tokens that may be spread over many adapters: the product in float32 into the workspace,
// the per-token or segmented shrink, and a segmented expand.  The tiles of the tensor-core shrink and of the pair kernel
// work through every adapter that they meet, and the host does not know which.  So: fewer than 16 tokens a slot; or
// fewer than 128 where y and the shrink's reads are small.  (us, separate / fused, 4096 x 4096: 513 tokens in no order
// over 6 adapters of rank 64 81 / 149, over 30 of rank 16 55 / 274, in runs of 512 over 6 of rank 64 85 / 75; 2048 tokens
// over 30 of rank 16 114 / 303, in runs of 64 over 30 of rank 8 103 / 106, in runs of 512 over 100 of rank 16 111 / 99;
// 4096 tokens in runs over 100 206 / 149.  8000 tokens 4096 x 256 over 100 of rank 8 93 / 442, in runs 90 / 81; 16384
// tokens 4096 x 88 in runs over 4 of rank 64 475 / 134.)
constexpr long long kI8SumElements = 32 << 20, kI8FewElements = 8 << 20, kI8ShrinkProducts = 1 << 29;
static bool separate(const PoolView& pv, int n) {
    const long long slots = std::min(n, pv.S), y = (long long)n * pv.h_out;
    return pv.dtype != LORA_F32 && n > kI8Tile &&
           ((n < 16 * slots && y <= kI8SumElements) ||
            (n < 128 * slots && y <= kI8FewElements && (long long)n * pv.R * pv.h_in <= kI8ShrinkProducts));
}
// The largest such batch of at most n tokens (0: none).
static int most_separate(const PoolView& pv, int n) {
    const int a = (int)std::min<long long>({(long long)n, 16LL * pv.S - 1, kI8SumElements / pv.h_out});
    const int b = (int)std::min<long long>({(long long)n, 128LL * pv.S - 1, kI8FewElements / pv.h_out,
                                            kI8ShrinkProducts / ((long long)pv.R * pv.h_in)});
    return std::max(separate(pv, a) ? a : 0, separate(pv, b) ? b : 0);
}

// Workspace of lora_i8_linear_fwd: the shrink output in its K parts, x's codes (in bytes for a few tokens,
// else in float16) and scales, the weight in float16 codes, the product where the expand is separate.
struct I8WsLayout {
    size_t codes_off, scales_off, w_off, y32_off, total;
};
static int ws_layout(lora_pool_t pool, int n, I8WsLayout* L) {
    if (n < 0) return set_error(LORA_EINVAL, "n_tokens < 0");
    const PoolView pv = pool_view(pool);
    if (pv.h_in > kI8MaxCols) return set_error(LORA_EUNSUP, "8-bit linear of %d features (at most %d)", pv.h_in, kI8MaxCols);
    // rows of shrink output over all K parts: at most what any batch of up to n tokens has (16-bit: at most
    // 256 / n parts up to 256 tokens; float32: 24 parts, and four CTAs an SM of 64 tokens)
    const long long m = std::max(n, 1);
    const long long rows = std::max(m, pv.dtype == LORA_F32 ? std::min(24 * m, 4LL * num_sms() * 64) : std::min(4 * m, 256LL));
    L->codes_off = align256((size_t)rows * pv.R * 4);
    const I8ProductWs P = product_ws(n, pv.h_out, pv.h_in);
    L->scales_off = L->codes_off + (n <= kI8Small ? align256((size_t)n * i8_pitch(pv.h_in)) : P.scales_off);
    L->w_off = L->scales_off + 2 * align256((size_t)n * 4);  // scales, peaks
    L->y32_off = L->w_off + P.total - P.w_off;
    L->total = L->y32_off + align256((size_t)most_separate(pv, n) * pv.h_out * 4);
    return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" {

int lora_i8_bytes(int rows, int cols, size_t* codes_bytes, size_t* scales_bytes) {
    if (!codes_bytes || !scales_bytes) return set_error(LORA_EINVAL, "codes_bytes/scales_bytes is NULL");
    const int rc = check_shape(rows, cols);
    if (rc) return rc;
    *codes_bytes = (size_t)rows * i8_pitch(cols);
    *scales_bytes = (size_t)rows * 4;
    return LORA_OK;
}

int lora_i8_quantize(const void* x_dev, int dtype, int64_t ld, const lora_i8_matrix* out, void* stream) {
    int rc = check_matrix(out, "out");
    if (rc) return rc;
    rc = check_rows(x_dev, dtype, ld, out->rows, out->cols, "x");
    if (rc) return rc;
    return launch_i8_quantize(x_dev, dtype, ld, view_of(out), static_cast<cudaStream_t>(stream));
}

int lora_i8_dequantize(const lora_i8_matrix* q, void* out_dev, int dtype, int64_t ld, void* stream) {
    int rc = check_matrix(q, "q");
    if (rc) return rc;
    rc = check_rows(out_dev, dtype, ld, q->rows, q->cols, "out");
    if (rc || q->rows == 0) return rc;
    return launch_i8_dequantize(view_of(q), out_dev, dtype, ld, static_cast<cudaStream_t>(stream));
}

int lora_i8_rmsnorm(const lora_i8_norm* p, void* stream) {
    if (!p) return set_error(LORA_EINVAL, "the arguments are NULL");
    int rc = check_dtype(p->dtype);
    if (!rc) rc = check_shape(p->rows, p->cols);
    if (rc) return rc;
    if (!(p->eps >= 1e-12f && p->eps <= 1.f)) return set_error(LORA_EINVAL, "eps %g outside [1e-12, 1]", (double)p->eps);
    if (!p->y_dev && !p->out) return set_error(LORA_EINVAL, "neither y nor out is wanted");
    if (p->residual_dev && !p->residual_out_dev) return set_error(LORA_EINVAL, "residual without residual_out");
    rc = check_rows(p->x_dev, p->dtype, p->ldx, p->rows, p->cols, "x");
    if (!rc) rc = check_rows(p->weight_dev, p->dtype, p->cols, p->rows ? 1 : 0, p->cols, "weight");
    if (!rc && p->residual_dev) rc = check_rows(p->residual_dev, p->dtype, p->ldr, p->rows, p->cols, "residual");
    if (!rc && p->residual_out_dev)
        rc = check_rows(p->residual_out_dev, p->dtype, p->ldro, p->rows, p->cols, "residual_out");
    if (!rc && p->y_dev) rc = check_rows(p->y_dev, p->dtype, p->ldy, p->rows, p->cols, "y");
    if (!rc && p->out) rc = check_matrix(p->out, "out");
    if (rc) return rc;
    if (p->rows > 0) {
        // a row is written while others are still read
        const size_t elt = dtype_size(p->dtype);
        const struct {
            const void *out, *other;
            int64_t lda, ldb;
            bool may;
            const char *what, *over;
        } pairs[] = {{p->residual_out_dev, p->x_dev, p->ldro, p->ldx, true, "residual_out", "x"},
                     {p->residual_out_dev, p->residual_dev, p->ldro, p->ldr, true, "residual_out", "residual"},
                     {p->y_dev, p->x_dev, p->ldy, p->ldx, true, "y", "x"},
                     {p->y_dev, p->residual_dev, p->ldy, p->ldr, true, "y", "residual"},
                     {p->y_dev, p->residual_out_dev, p->ldy, p->ldro, false, "y", "residual_out"}};
        for (const auto& q : pairs)
            if (meets(q.out, q.lda, q.other, q.ldb, p->rows, p->cols, elt, q.may))
                return set_error(LORA_EINVAL, "%s overlaps %s%s", q.what, q.over, q.may ? " without being the same array" : "");
    }
    if (p->out && (p->out->rows != p->rows || p->out->cols != p->cols))
        return set_error(LORA_EINVAL, "out is %d x %d, x %d x %d", p->out->rows, p->out->cols, p->rows, p->cols);
    if (p->rows == 0) return LORA_OK;
    return launch_i8_rmsnorm(*p, static_cast<cudaStream_t>(stream));
}

int lora_i8_matmul_workspace_bytes(int x_rows, int w_rows, int cols, size_t* bytes) {
    if (!bytes) return set_error(LORA_EINVAL, "bytes is NULL");
    int rc = check_shape(x_rows, cols);
    if (!rc) rc = check_shape(w_rows, cols);
    if (rc) return rc;
    *bytes = product_ws(x_rows, w_rows, cols).total;
    return LORA_OK;
}

int lora_i8_matmul(const lora_i8_matrix* x, const lora_i8_matrix* w, void* y_dev, int dtype, int64_t ldy, void* ws_dev,
                   size_t ws_bytes, void* stream) {
    int rc = check_matrix(x, "x");
    if (!rc) rc = check_matrix(w, "w");
    if (rc) return rc;
    if (x->cols != w->cols) return set_error(LORA_EINVAL, "x has %d columns, w %d", x->cols, w->cols);
    rc = check_rows(y_dev, dtype, ldy, w->rows ? x->rows : 0, w->rows, "y");
    if (rc || x->rows == 0 || w->rows == 0) return rc;
    const I8ProductWs L = product_ws(x->rows, w->rows, x->cols);
    if (L.total && !ws_dev) return set_error(LORA_EINVAL, "ws is NULL");
    if (reinterpret_cast<uintptr_t>(ws_dev) % 256) return set_error(LORA_EINVAL, "ws must be 256-byte aligned");
    if (ws_bytes < L.total)
        return set_error(LORA_ENOSPACE, "8-bit product workspace needs %zu bytes, got %zu", L.total, ws_bytes);
    const I8View xv = view_of(x), wv = view_of(w);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x->rows <= kI8Small) return launch_i8_small(xv, wv, y_dev, dtype, ldy, nullptr, /*early_w=*/false, nullptr, st);
    char* ws = static_cast<char*>(ws_dev);
    float* sx = reinterpret_cast<float*>(ws + L.scales_off);
    int* peak = reinterpret_cast<int*>(ws + L.scales_off + align256((size_t)x->rows * 4));
    rc = x->rows <= kI8Tile ? launch_i8_expand_small(xv, nullptr, nullptr, ws, sx, peak, st)
                            : launch_i8_expand(xv, nullptr, nullptr, ws, sx, st);
    if (rc) return rc;
    const I8Rows rows = {ws, sx, nullptr, x->rows, x->cols, peak};
    if (x->rows <= kI8Tile)
        return launch_i8_tile(rows, wv, y_dev, dtype, ldy, nullptr, /*early_x=*/false, /*release=*/false, nullptr, st);
    rc = launch_i8_expand(wv, nullptr, nullptr, ws + L.w_off, nullptr, st);
    if (rc) return rc;
    const I8Rows wrows = {ws + L.w_off, wv.scales, nullptr, w->rows, w->cols, nullptr};
    return launch_i8_pair(rows, wrows, y_dev, dtype, ldy, nullptr, /*release=*/false, nullptr, st);
}

int lora_i8_linear_workspace_bytes(lora_pool_t pool, int n_tokens, size_t* bytes) {
    if (!pool || !bytes) return set_error(LORA_EINVAL, "pool/bytes is NULL");
    I8WsLayout L;
    const int rc = ws_layout(pool, n_tokens, &L);
    if (rc) return rc;
    *bytes = L.total;
    return LORA_OK;
}

int lora_i8_linear_fwd(lora_pool_t pool, const lora_i8_matrix* w, const void* x_dev, const lora_i8_matrix* xq,
                       void* y_dev, const lora_segments* seg, void* ws_dev, size_t ws_bytes, void* stream) {
    if (!pool || !seg) return set_error(LORA_EINVAL, "pool/seg is NULL");
    const PoolView pv = pool_view(pool);
    const int n = seg->n_tokens;
    if (seg->n_slots != pv.S)
        return set_error(LORA_EINVAL, "segments were built for %d slots, pool has %d", seg->n_slots, pv.S);
    int rc = check_matrix(w, "w");
    if (rc) return rc;
    if (w->rows != pv.h_out || w->cols != pv.h_in)
        return set_error(LORA_EINVAL, "w is %d x %d, the pool's linear %d x %d", w->rows, w->cols, pv.h_out, pv.h_in);
    if (xq) {
        rc = check_matrix(xq, "xq");
        if (rc) return rc;
        if (xq->rows != n || xq->cols != pv.h_in)
            return set_error(LORA_EINVAL, "xq is %d x %d, x %d x %d", xq->rows, xq->cols, n, pv.h_in);
    }
    if (n == 0) return LORA_OK;
    if (!x_dev || !y_dev || !ws_dev) return set_error(LORA_EINVAL, "x/y/ws is NULL");
    const size_t align = pv.dtype == LORA_F32 ? 4 : 16;
    if ((reinterpret_cast<uintptr_t>(x_dev) | reinterpret_cast<uintptr_t>(y_dev)) % align)
        return set_error(LORA_EINVAL, "x/y must be %zu-byte aligned", align);
    if (reinterpret_cast<uintptr_t>(ws_dev) % 256) return set_error(LORA_EINVAL, "ws must be 256-byte aligned");
    I8WsLayout L;
    rc = ws_layout(pool, n, &L);
    if (rc) return rc;
    if (ws_bytes < L.total)
        return set_error(LORA_ENOSPACE, "8-bit linear workspace needs %zu bytes, got %zu", L.total, ws_bytes);
    char* ws = static_cast<char*>(ws_dev);
    float* s_buf = reinterpret_cast<float*>(ws);
    float* sx = reinterpret_cast<float*>(ws + L.scales_off);
    int* peak = reinterpret_cast<int*>(ws + L.scales_off + align256((size_t)n * 4));
    const SegView sv = seg_view(seg);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool few = n <= kI8Small;
    const bool front = n <= kI8Tile && (pv.dtype == LORA_F32 ? f32_front(pv, n) : !shrink_segmented(pv, n));
    char* codes = ws + L.codes_off;
    I8View xv, stored;
    if (xq) stored = view_of(xq);
    int s_parts = 1;
    if (front) {
        rc = launch_i8_front(pv, sv, x_dev, xq ? &stored : nullptr, codes, !few, sx, peak, s_buf, &s_parts, st);
    } else {
        if (!few)  // rows in the order of the segments
            rc = !xq            ? launch_i8_quantize_f16(x_dev, pv.dtype, n, pv.h_in, sv.perm, sv.status, codes, sx,
                                                         n <= kI8Tile ? peak : nullptr, st)
                 : n <= kI8Tile ? launch_i8_expand_small(stored, sv.perm, sv.status, codes, sx, peak, st)
                                : launch_i8_expand(stored, sv.perm, sv.status, codes, sx, st);
        else if (!xq)
            rc = launch_i8_quantize(x_dev, pv.dtype, pv.h_in, i8_view(codes, sx, n, pv.h_in), st);
        if (rc) return rc;
        if (pv.dtype == LORA_F32) {
            s_parts = f32_shrink_parts(pv, n);
            rc = launch_f32_shrink(pv, sv, x_dev, s_buf, st);
        } else if (n <= kI8Tile || separate(pv, n)) {
            // beside the kernel that makes x's codes, where there is one (200 tokens 11008 x 4096 rank 64: 57.1 us after
            // it, 55.4 beside it; 300 tokens over 100 adapters 4096 x 4096 rank 8: 56 and 48.5)
            rc = launch_shrink(pv, sv, x_dev, s_buf, st, /*tiled=*/false, &s_parts, /*xready=*/0, /*beside=*/!few || !xq);
        } else if (shrink_tc_supported(pv)) {
            rc = launch_shrink_tc(pv, sv, x_dev, s_buf, st);
        } else {
            rc = launch_shrink(pv, sv, x_dev, s_buf, st, /*tiled=*/true, &s_parts);
        }
    }
    if (rc) return rc;
    const I8View wv = view_of(w);
    const I8Lora lora = {&pv, sv.idx, s_buf, s_parts};
    if (few) {
        xv = xq ? stored : i8_view(codes, sx, n, pv.h_in);
        return launch_i8_small(xv, wv, y_dev, pv.dtype, pv.h_out, sv.status, /*early_w=*/true, &lora, st);
    }
    const I8Rows rows = {codes, sx, sv.perm, n, pv.h_in, peak};
    if (n <= kI8Tile)
        // x is complete before the product starts only where a float32 shrink, which waits for it, lies between
        return launch_i8_tile(rows, wv, y_dev, pv.dtype, pv.h_out, sv.status,
                              /*early_x=*/!front && pv.dtype == LORA_F32, /*release=*/true, &lora, st);
    rc = launch_i8_expand(wv, nullptr, nullptr, ws + L.w_off, nullptr, st);
    if (rc) return rc;
    const I8Rows wrows = {ws + L.w_off, wv.scales, nullptr, wv.rows, wv.cols, nullptr};
    if (pv.dtype == LORA_F32) {
        rc = launch_i8_pair(rows, wrows, y_dev, LORA_F32, pv.h_out, sv.status, /*release=*/true, nullptr, st);
        return rc ? rc : launch_f32_expand(pv, sv, s_buf, s_parts, y_dev, st);
    }
    if (separate(pv, n)) {
        float* y32 = reinterpret_cast<float*>(ws + L.y32_off);
        rc = launch_i8_pair(rows, wrows, y32, LORA_F32, pv.h_out, sv.status, /*release=*/true, nullptr, st);
        return rc ? rc : launch_sum_expand(pv, sv, s_buf, s_parts, y32, y_dev, st);
    }
    return launch_i8_pair(rows, wrows, y_dev, pv.dtype, pv.h_out, sv.status, /*release=*/true, &lora, st);
}

}  // extern "C"
