"""Matrices in 8-bit integers on the GPU against the float64 oracle.

Stored codes and scales are compared bit for bit: the definition leaves no freedom, and the norm holds its
row statistics closely enough (about 2^-44) that an element within that of a border of two codes does not
occur in these inputs.  A product's sum is a whole number and exact; its output is that sum rounded to
float32 and two float32 multiplications, then one rounding to its type: 3 * 2^-24 of itself and half a step
of the type.  The LoRA term adds float32 sums of h_in and of r_max products.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from oracle import i8_oracle as Q
from oracle import lora_oracle as O

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}  # half a subnormal step
F = 2.0 ** -24


def special_rows(rows, cols, dtype, seed=0):
    """Rows that meet every branch: ties, zeros, tiny and huge rows, infinities, NaN, -0."""
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 8, size=(rows, 1)))
    ties = rng.integers(-254, 255, size=(rows, cols)) / 2.0
    ties[:, 0] = 127
    kind = rng.integers(0, 8, size=(rows, 1))
    x = np.where(kind == 0, ties, x)
    x = np.where(kind == 1, 0.0, x)
    x = np.where(kind == 2, x * 2.0 ** (-16 if dtype == torch.float16 else -125), x)
    x = np.where(kind == 3, x * 2.0 ** (6 if dtype == torch.float16 else 118), x)
    x[rng.random((rows, cols)) < 0.05] = -0.0
    t = torch.from_numpy(x).to(dtype)
    if rows > 4:
        t[1, cols // 2] = float("inf")
        t[2, cols // 3] = float("nan")
        t[3, cols // 2] = torch.finfo(dtype).max
        t[4] = torch.finfo(dtype).smallest_normal / 8
    return t


def guarded_matrix(lib, rows, cols):
    """A stored matrix whose buffers are exactly as long as lora_i8_bytes says, between canaries."""
    m = lib.I8Matrix(rows, cols)
    nc, ns = lib.lora_i8_bytes(rows, cols)
    bufs = []
    for n in (nc, ns):
        full = torch.full((2 * 4096 + (n + 255) // 256 * 256,), 0x25, dtype=torch.int8, device="cuda")
        bufs.append((full, n))
    m.codes = bufs[0][0][4096:4096 + nc].view(rows, -1)
    m.scales = bufs[1][0][4096:4096 + ns].view(torch.float32)
    m.struct = lib.lora_i8_matrix(m.codes.data_ptr(), m.scales.data_ptr(), rows, cols)
    m.bufs = bufs
    return m


def check_stored(m, cols, codes, scales):
    got = m.codes.cpu().numpy()
    s = m.scales.cpu().numpy()
    assert np.array_equal(s, scales, equal_nan=True)
    assert np.array_equal(got[:, :cols], codes) and (got[:, cols:] == 0).all()
    for full, n in getattr(m, "bufs", ()):
        assert (full[:4096] == 0x25).all() and (full[4096 + n:] == 0x25).all()


SHAPES = [(1, 1, 0, 0), (1, 4096, 0, 0), (3, 31, 0, 0), (5, 33, 0, 1), (129, 257, 0, 0), (700, 255, 1, 0), (64, 1000, 24, 0),
          (900, 1009, 31, 3), (400, 4097, 0, 0), (400, 4104, 0, 0), (7, 11008, 8, 8), (350, 17000, 0, 0), (3, 70001, 0, 0),
          (320, 20008, 1, 0)]


def strided(rows, cols, pad, shift, dtype, fill=float("nan")):
    wide = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=dtype, device="cuda")
    return wide, wide[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad,shift", SHAPES)
def test_quantize_bytes_and_read_back(lib, dtype, rows, cols, pad, shift):
    src = special_rows(rows, cols, dtype)
    _, x = strided(rows, cols, pad, shift, dtype)
    x.copy_(src)
    m = guarded_matrix(lib, rows, cols)
    lib.lora_i8_quantize(x, m)
    codes, scales = Q.quantise(src)
    check_stored(m, cols, codes, scales)
    for out_dtype in DTYPES:
        out = torch.full((rows, cols + pad + 3), 7.0, dtype=out_dtype, device="cuda")
        lib.lora_i8_dequantize(m, out[:, :cols])
        with np.errstate(all="ignore"):
            want = codes.astype(np.float32) * scales[:, None]
        ref = torch.from_numpy(want).to(out_dtype)
        assert torch.equal(out[:, :cols].cpu().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
        assert (out[:, cols:] == 7.0).all()


def test_quantize_is_the_same_for_every_dtype(lib):
    x = (torch.randn(70, 300, generator=torch.Generator().manual_seed(1)) * 3).to(torch.bfloat16)
    x = x.to(torch.float16).to(torch.bfloat16)  # values every type holds
    out = []
    for dtype in DTYPES:
        m = lib.lora_i8_quantize(x.to(dtype).cuda(), lib.I8Matrix(70, 300))
        out.append((m.codes.clone(), m.scales.clone()))
    for c, s in out[1:]:
        assert torch.equal(c, out[0][0]) and torch.equal(s, out[0][1])


# ---- norm -----------------------------------------------------------------------------------------

def norm_inputs(rows, cols, dtype, seed):
    rng = np.random.default_rng([seed, rows, cols])
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 6, (rows, 1)))).to(dtype)
    res = torch.from_numpy(rng.standard_normal((rows, cols)) * 2).to(dtype)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).to(dtype)
    if rows > 3:
        x[0] = 0
        res[0] = 0
        x[1] = x[1] * 2.0 ** -10
        res[1] = 0
    return x, res, w


def check_norm(y, h, w, eps, dtype):
    ref = Q.rmsnorm(h, w, eps)
    err = np.abs(y.cpu().double().numpy() - ref)
    # r rounded to float32, the product h w (exact for 16-bit types), that product times r, the type's rounding
    assert (err <= (4 * F + UNIT[dtype]) * np.abs(ref) + TINY[dtype]).all()
    return ref


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad,shift", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(lib, dtype, rows, cols, pad, shift, residual):
    eps = 1e-5
    x0, res0, w0 = norm_inputs(rows, cols, dtype, 1)
    _, x = strided(rows, cols, pad, shift, dtype)
    x.copy_(x0)
    w = w0.cuda()
    m = guarded_matrix(lib, rows, cols)
    y = torch.full((rows, cols + 5), 7.0, dtype=dtype, device="cuda")
    h = x0
    if residual:
        wide, res = strided(rows, cols, pad, shift, dtype, 7.0)
        res.copy_(res0)
        lib.lora_i8_rmsnorm(x, w, eps, out=m, y=y[:, :cols], residual=res)  # in place
        h = (x0.double() + res0.double()).to(dtype)
        assert torch.equal(res.cpu(), h)
        assert (wide[:shift] == 7.0).all() and (wide[-8:] == 7.0).all()
        assert torch.equal(x.cpu(), x0)
    else:
        lib.lora_i8_rmsnorm(x, w, eps, out=m, y=y[:, :cols])
    ref = check_norm(y[:, :cols], h, w0, eps, dtype)
    assert (y[:, cols:] == 7.0).all()
    check_stored(m, cols, *Q.quantise(ref))
    # either output by itself gives the same
    m2, y2 = lib.I8Matrix(rows, cols), torch.empty(rows, cols, dtype=dtype, device="cuda")
    hd = h.cuda()
    lib.lora_i8_rmsnorm(hd, w, eps, out=m2)
    lib.lora_i8_rmsnorm(hd, w, eps, y=y2)
    assert torch.equal(m2.codes, m.codes) and torch.equal(m2.scales, m.scales) and torch.equal(y2, y[:, :cols])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [200, 4096, 9000])
def test_norm_special_rows(lib, dtype, cols):
    """Zeros, infinities and NaN, and rows whose squares overflow float32."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((7, cols))).to(dtype)
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, cols - 1] = float("nan")
    if dtype != torch.float16:
        x[3] *= 2.0 ** 120
        x[4] *= 2.0 ** 70
    x[5, 1:] = 0
    w = torch.ones(cols, dtype=dtype)
    w[3] = 0
    m, y = lib.I8Matrix(7, cols), torch.empty(7, cols, dtype=dtype, device="cuda")
    lib.lora_i8_rmsnorm(x.cuda(), w.cuda(), 1e-6, out=m, y=y)
    ok = [0, 3, 4, 5, 6]
    ref = check_norm(y[ok], x[ok], w, 1e-6, dtype)
    codes, scales = Q.quantise(ref)
    assert np.array_equal(m.codes[ok, :cols].cpu().numpy(), codes) and np.array_equal(m.scales[ok].cpu().numpy(), scales)
    assert m.scales[[1, 2]].isnan().all() and (m.codes[[1, 2]] == 0).all()
    assert y[1, 7].isnan() and y[2].isnan().all() and (y[1, :7] == 0).all()


def test_norm_outputs_over_their_inputs(lib):
    """residual_out and y over x, and a column window of a wider buffer."""
    x0, res0, w0 = norm_inputs(50, 264, torch.bfloat16, 5)
    w = w0.cuda()
    h = (x0.float() + res0.float()).bfloat16()
    m = lib.I8Matrix(50, 264)
    x = x0.cuda()
    lib.lora_i8_rmsnorm(x, w, 1e-5, out=m, residual=res0.cuda(), residual_out=x)
    assert torch.equal(x.cpu(), h)
    check_stored(m, 264, *Q.quantise(Q.rmsnorm(h, w0, 1e-5)))
    x = x0.cuda()
    lib.lora_i8_rmsnorm(x, w, 1e-5, y=x, residual=res0.cuda(), residual_out=torch.empty_like(x))
    check_norm(x, h, w0, 1e-5, torch.bfloat16)


# ---- product ----------------------------------------------------------------------------------------

def stored(lib, t):
    return lib.lora_i8_quantize(t.cuda(), lib.I8Matrix(t.shape[0], t.shape[1]))


def check_product(lib, x, w, dtype, pad=0):
    n, m = x.shape[0], w.shape[0]
    y = torch.full((n + 2, m + pad + 1), 7.0, dtype=dtype, device="cuda")
    yv = y[1:n + 1, :m]
    lib.lora_i8_matmul(stored(lib, x), stored(lib, w), yv)
    (cx, sx), (cw, sw) = Q.quantise(x), Q.quantise(w)
    ref = Q.sums(cx, cw).astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    err = np.abs(yv.cpu().double().numpy() - ref)
    assert (err <= (3 * F + UNIT[dtype]) * np.abs(ref) + TINY[dtype]).all()
    assert (y[0] == 7.0).all() and (y[n + 1] == 7.0).all() and (y[1:n + 1, m:] == 7.0).all()


def gauss(rows, cols, seed, dtype=torch.float32, scale=1.0):
    return (torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("k", [1, 15, 16, 17, 127, 128, 129, 1000, 1025, 2100])
@pytest.mark.parametrize("n,m,dtype", [(1, 1, 0), (1, 300, 1), (2, 129, 2), (3, 8, 0), (7, 129, 2), (8, 640, 1), (9, 130, 1),
                                       (17, 640, 1), (64, 128, 2), (100, 257, 0)])
def test_product_small_batches(lib, n, m, k, dtype):
    check_product(lib, gauss(n, k, 1), gauss(m, k, 2, scale=0.02), DTYPES[dtype], pad=m % 3)


@pytest.mark.parametrize("n,m,k,dtype", [(128, 512, 4096, 2), (129, 300, 700, 0), (200, 264, 1500, 1), (256, 1024, 1024, 2),
                                         (257, 100, 64, 1), (300, 513, 2048, 0), (777, 391, 1111, 2), (1500, 1003, 520, 1),
                                         (2050, 640, 130, 0), (5000, 77, 33, 2)])
def test_product_large_batches(lib, n, m, k, dtype):
    check_product(lib, gauss(n, k, 3), gauss(m, k, 4, scale=0.02), DTYPES[dtype], pad=(8 - m % 8) % 8 + 7)


@pytest.mark.parametrize("n", [1, 5, 16, 60, 130, 300, 700])
@pytest.mark.parametrize("k", [1024, 1100, 5000, 40000])
def test_sums_are_exact_at_their_largest(lib, n, k):
    """Every code -128 (which a caller may store) or 127: partial sums far past 2^24 stay whole."""
    m = 200
    rng = np.random.default_rng([n, k])
    x, w = lib.I8Matrix(n, k), lib.I8Matrix(m, k)
    cx = np.where(rng.random((n, 1)) < 0.5, -128, 127) * np.ones((1, k), np.int64)
    cw = np.where(rng.random((m, 1)) < 0.5, -128, 127) * np.ones((1, k), np.int64)
    cx[:, -3:] = rng.integers(-128, 128, (n, 3))
    cw[:, -3:] = rng.integers(-128, 128, (m, 3))
    for q, c in ((x, cx), (w, cw)):
        q.codes.zero_()
        q.codes[:, :k].copy_(torch.from_numpy(c.astype(np.int8)))
        q.scales.fill_(1.0)
    y = torch.empty(n, m, device="cuda")
    lib.lora_i8_matmul(x, w, y)
    ref = (cx @ cw.T).astype(np.float32)  # the float32 nearest the whole number
    assert np.array_equal(y.cpu().numpy(), ref)


@pytest.mark.parametrize("n", [10, 60, 200])
@pytest.mark.parametrize("k", [5001, 40000, 100000])
def test_sums_are_exact_where_tokens_codes_are_small(lib, n, k):
    """The smaller a batch's codes, the longer its sums stay in float32: every size of code at its largest sums, all
    of one sign, each an odd number."""
    m = 140
    rng = np.random.default_rng([n, k])
    w = lib.I8Matrix(m, k)
    cw = np.where(rng.random((m, 1)) < 0.5, -128, 127) * np.ones((1, k), np.int64)
    cw[:, -3:] = rng.integers(-128, 128, (m, 3))
    sign = np.where(rng.random((n, 1)) < 0.5, -1, 1)
    for c in (1, 3, 9, 13, 23, 41, 63, 101):
        cx = sign * c * np.ones((1, k), np.int64)
        if c == 13:
            cx[n // 2, k // 3: k // 3 + 300] = 127  # one token's codes are large, in three blocks
        if c == 3:
            cx[:, 100:k - 100] = 0
        x = lib.I8Matrix(n, k)
        for q, codes in ((x, cx), (w, cw)):
            q.codes.zero_()
            q.codes[:, :k].copy_(torch.from_numpy(codes.astype(np.int8)))
            q.scales.fill_(1.0)
        y = torch.empty(n, m, device="cuda")
        lib.lora_i8_matmul(x, w, y)
        ref = (cx @ cw.T).astype(np.float32)
        assert np.array_equal(y.cpu().numpy(), ref), c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k,slots,r_max", [(12, 20000, 2, 8), (40, 30001, 2, 8), (130, 20000, 3, 16), (200, 20008, 60, 8)])
@pytest.mark.parametrize("small", [0.02, 0.1, 0.4])
def test_linear_of_rows_with_few_large_values(lib, dtype, n, k, slots, r_max, small):
    """Rows whose scale is that of a few values: small codes along most of K."""
    if dtype != torch.float32:
        k = k // 8 * 8
    case = wl.random_case(k, n, k, 264, [r_max] * slots, r_max=r_max, dtype=dtype, p_base=0.5)
    x = case.x.float().sign() * (1 - 0.1 * torch.rand(n, k, generator=torch.Generator().manual_seed(k)))
    x[:, 1:] *= small
    x[:, k // 2: k // 2 + 5] = -1.0
    case.x = x.to(dtype)
    case.W = (case.W.float().abs() * case.x[0].float().sign()).to(dtype)  # (sums of one sign for the first token)
    check_linear(lib, case)


def test_a_row_gives_the_same_bits_in_every_batch(lib):
    x, w = gauss(700, 1300, 8), gauss(390, 1300, 9, scale=0.02)
    q = stored(lib, w)
    full = torch.empty(700, 390, device="cuda")
    lib.lora_i8_matmul(stored(lib, x), q, full)
    for n in (1, 2, 4, 8, 9, 33, 64, 100, 128, 129, 256, 257, 512):
        y = torch.empty(n, 390, device="cuda")
        lib.lora_i8_matmul(stored(lib, x[:n]), q, y)
        assert torch.equal(y, full[:n]), n


def test_scales_that_are_not_numbers_stay_in_their_row(lib):
    for n in (3, 40, 300):
        x, w = gauss(n, 200, 5), gauss(150, 200, 6)
        x[1, 5] = float("inf")
        w[7, 9] = float("nan")
        y = torch.empty(n, 150, device="cuda")
        lib.lora_i8_matmul(stored(lib, x), stored(lib, w), y)
        bad = y.isnan().cpu()
        want = torch.zeros(n, 150, dtype=torch.bool)
        want[1] = True
        want[:, 7] = True
        assert torch.equal(bad, want)


# ---- linear -----------------------------------------------------------------------------------------

def make_pool(lib, case):
    ad = case.adapters
    pool = lib.LoraPool(case.h_in, case.h_out, ad.r_max, ad.n_slots, case.dtype, "cuda")
    for s in range(ad.n_slots):
        pool.load_slot(s, ad.A[s].cuda(), ad.B[s].cuda(), ad.alphas[s])
    return pool


def linear_reference(case, codes=None):
    """(float64 y, bound on its error)."""
    cx, sx = Q.quantise(case.x) if codes is None else codes
    cw, sw = Q.quantise(case.W)
    base = Q.sums(cx, cw).astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    pool = O.pool_of_case(case)
    x = case.x.double().numpy()
    y, mag = base.copy(), np.zeros_like(base)
    for t, s in enumerate(case.idx.tolist()):
        if s < 0:
            continue
        y[t] += pool.scale[s] * (pool.B[s] @ (pool.A[s] @ x[t]))
        mag[t] = abs(pool.scale[s]) * (np.abs(pool.B[s]) @ (np.abs(pool.A[s]) @ np.abs(x[t])))
    # float32 sums of h_in and then r_max products, the scale, the sum over K parts; the base term's three
    # roundings, the addition, the type's rounding
    terms = case.h_in + case.adapters.r_max + 32
    bound = terms * F * mag + 3 * F * np.abs(base) + (F + UNIT[case.dtype]) * np.abs(y) + TINY[case.dtype]
    return y, bound


def check_linear(lib, case, **kw):
    pool = make_pool(lib, case)
    w = stored(lib, case.W)
    seg = pool.segment(case.idx.cuda())
    n = case.x.shape[0]
    y = torch.full((n + 2, case.h_out), 7.0, dtype=case.dtype, device="cuda")
    if (case.h_out * y.element_size()) % 16 and case.dtype != torch.float32:
        raise AssertionError("a test of 16-bit pools has 16-byte rows")
    x = case.x.cuda()
    pool.i8_linear(w, x, seg, y=y[1:n + 1])
    assert lib.lora_segment_status(seg) == lib.LORA_OK
    ref, bound = linear_reference(case)
    err = np.abs(y[1:n + 1].cpu().double().numpy() - ref)
    assert (err <= bound).all(), f"{(err / bound).max()}"
    assert (y[0] == 7.0).all() and (y[n + 1] == 7.0).all()
    # with x's stored form from outside: the same bits
    y2 = pool.i8_linear(w, x, seg, xq=stored(lib, case.x))
    assert torch.equal(y2, y[1:n + 1])
    pool.close()
    return y2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max,p_base", [
    (1, 64, 8, [8], 8, 0.0), (1, 4096, 136, [8, 8], 8, 0.0), (2, 264, 72, [1, 16], 16, 0.5), (5, 1000, 200, [3, 8, 24], 24, 0.2),
    (8, 512, 128, [8] * 20, 8, 0.1), (9, 256, 256, [64, 8], 64, 0.0), (16, 2056, 136, [16, 2], 16, 0.3), (40, 256, 384, [8, 16, 8], 16, 0.2),
    (64, 1024, 264, [8] * 100, 8, 0.1), (100, 3000, 128, [64, 8, 16], 64, 0.15), (128, 520, 520, [5] * 7, 8, 0.2),
    (129, 520, 136, [8, 256], 256, 0.2), (200, 1200, 264, [8, 16, 64] * 2, 64, 0.15), (256, 256, 264, [32] * 40, 32, 0.0),
    (257, 256, 264, [8, 16], 16, 0.2), (300, 1032, 392, [16] * 60, 16, 0.1), (700, 264, 520, [8, 64, 24], 64, 0.3),
    (1300, 520, 264, [16] * 9, 16, 1.0)])
def test_linear(lib, dtype, n, h_in, h_out, ranks, r_max, p_base):
    check_linear(lib, wl.random_case(n + h_in, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, p_base=p_base))


@pytest.mark.parametrize("n,h_in,h_out,r_max", [(3, 37, 5, 3), (20, 101, 33, 5), (150, 77, 131, 7), (400, 333, 91, 12)])
def test_linear_float32_odd_sizes(lib, n, h_in, h_out, r_max):
    check_linear(lib, wl.random_case(n, n, h_in, h_out, [r_max, 1, 2], r_max=r_max, dtype=torch.float32, p_base=0.2))


@pytest.mark.parametrize("n,slots,r_max", [(300, 100, 8), (900, 60, 64), (2000, 3, 256), (1700, 100, 24), (5000, 100, 8)])
def test_linear_many_adapters_in_large_batches(lib, n, slots, r_max):
    """The separate expand (few tokens a slot) and tiles of several adapters."""
    check_linear(lib, wl.random_case(n + slots, n, 136, 264, [max(1, r_max // (1 + s % 3)) for s in range(slots)], r_max=r_max,
                                     dtype=torch.bfloat16, p_base=0.1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max", [
    (130, 1000, 1304, [8] * 100, 8), (257, 2056, 136, [8] * 100, 8), (320, 520, 264, [64, 8, 16], 64), (400, 3000, 2056, [16] * 30, 16),
    (511, 1032, 520, [32, 24], 32), (512, 520, 4104, [8, 64], 64), (513, 520, 264, [8] * 100, 8)])
def test_linear_in_several_groups_of_tokens(lib, dtype, n, h_in, h_out, ranks, r_max):
    check_linear(lib, wl.random_case(n + h_in, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, p_base=0.1))


@pytest.mark.parametrize("n,m,k", [(48, 2056, 2048), (160, 4104, 4096), (256, 2048, 2100), (257, 1000, 1000), (320, 11008, 600), (384, 130, 40000),
                                   (511, 8, 1500), (512, 3000, 1024)])
def test_product_in_several_groups_of_tokens(lib, n, m, k):
    check_product(lib, gauss(n, k, 3), gauss(m, k, 4, scale=0.02), torch.float32, pad=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 7, 40, 130, 300, 700])
def test_adapters_that_are_not_finite_reach_their_own_tokens_only(lib, dtype, n):
    slots = 3 if n < 100 else 4
    case = wl.random_case(n, n, 264, 136, [8] * slots, r_max=8, dtype=dtype, p_base=0.1)
    case.idx[0] = 1
    ad = case.adapters
    clean = make_pool(lib, case)
    w, x = stored(lib, case.W), case.x.cuda()
    seg = clean.segment(case.idx.cuda())
    want = clean.i8_linear(w, x, seg).cpu()
    ad.B[1][5, 3] = float("inf")
    ad.B[1][9, 0] = float("nan")
    ad.A[slots - 1][2, 7] = float("nan")
    pool = make_pool(lib, case)
    got = pool.i8_linear(w, x, pool.segment(case.idx.cuda())).cpu()
    idx = case.idx
    ok = torch.ones_like(got, dtype=torch.bool)
    ok[idx == 1, 5] = False
    ok[idx == 1, 9] = False
    ok[idx == slots - 1] = False
    assert torch.equal(got[ok], want[ok])
    assert got[idx == slots - 1].isnan().all()
    assert got[idx == 1][:, 9].isnan().all() and not got[idx == 1][:, 5].isfinite().any()
    clean.close()
    pool.close()


@pytest.mark.parametrize("n", [1, 8, 9, 64, 200, 300])
def test_refused_batches_leave_y_untouched(lib, n):
    case = wl.random_case(n, n, 264, 136, [8, 8], r_max=8, dtype=torch.float16)
    pool = make_pool(lib, case)
    idx = case.idx.clone()
    idx[n // 2] = 7
    seg = pool.segment(idx.cuda())
    y = torch.full((n, 136), 7.0, dtype=torch.float16, device="cuda")
    pool.i8_linear(stored(lib, case.W), case.x.cuda(), seg, y=y)
    assert lib.lora_segment_status(seg) == lib.LORA_EIDX
    assert (y == 7.0).all()
    pool.close()


def test_empty_batches(lib):
    pool = lib.LoraPool(64, 32, 8, 2, torch.float16, "cuda")
    w = stored(lib, gauss(32, 64, 1))
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    seg = pool.segment(torch.empty(0, dtype=torch.int32, device="cuda"))
    assert pool.i8_linear(w, x, seg).shape == (0, 32)
    q = lib.lora_i8_quantize(x, lib.I8Matrix(0, 64))
    y = torch.empty(0, 32, device="cuda")
    lib.lora_i8_matmul(q, w, y)
    lib.lora_i8_dequantize(q, x)
    lib.lora_i8_rmsnorm(x, torch.ones(64, dtype=torch.float16, device="cuda"), 1e-5, out=q, y=x)
    pool.close()


def test_workspaces(lib):
    pool = lib.LoraPool(512, 256, 16, 100, torch.bfloat16, "cuda")
    last = 0
    for n in (0, 1, 2, 8, 9, 20, 64, 100, 256, 257, 300, 1000, 1599, 1600, 5000):
        need = lib.lora_i8_linear_workspace_bytes(pool.handle, n)
        assert need >= last
        last = need
    w = stored(lib, gauss(256, 512, 1))
    for n in (3, 30, 300):
        x = torch.zeros(n, 512, dtype=torch.bfloat16, device="cuda")
        seg = pool.segment(torch.full((n,), -1, dtype=torch.int32, device="cuda"))
        y = torch.empty(n, 256, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(lib.lora_i8_linear_workspace_bytes(pool.handle, n), dtype=torch.uint8, device="cuda")
        lib.lora_i8_linear_fwd(pool.handle, w, x, y, seg, ws)
        with pytest.raises(lib.LoraError) as e:
            lib.lora_i8_linear_fwd(pool.handle, w, x, y, seg, ws[:-1])
        assert e.value.code == lib.LORA_ENOSPACE
        with pytest.raises(lib.LoraError) as e:
            lib.lora_i8_linear_fwd(pool.handle, w, x, y, seg, ws, xq=lib.I8Matrix(n + 1, 512))
        assert e.value.code == lib.LORA_EINVAL
    with pytest.raises(lib.LoraError) as e:
        pool.i8_linear(stored(lib, gauss(255, 512, 1)), x, seg, y=y)
    assert e.value.code == lib.LORA_EINVAL
    pool.close()


# ---- together --------------------------------------------------------------------------------------

class Layer:
    """A norm with its residual and two projections over 8-bit bases that share its output."""

    def __init__(self, lib, h, dtype, seed, slots=5):
        self.lib, self.h = lib, h
        self.case = [wl.random_case(seed + i, 4, h, o, [8, 4, 8, 2, 8][:slots], r_max=8, dtype=dtype) for i, o in enumerate((h, 2 * h))]
        self.pools = [make_pool(lib, c) for c in self.case]
        self.W = [c.W for c in self.case]
        self.w = [stored(lib, c.W) for c in self.case]
        self.gamma = (1 + 0.1 * gauss(1, h, seed)[0]).to(dtype)
        self.g = self.gamma.cuda()

    def run(self, x, res, seg, q, y, out, stream=None):
        self.lib.lora_i8_rmsnorm(x, self.g, 1e-5, out=q, y=y, residual=res, stream=stream)
        for pool, w, o in zip(self.pools, self.w, out):
            pool.i8_linear(w, y, seg, xq=q, y=o, stream=stream)

    def buffers(self, n, dtype):
        lib = self.lib
        return (lib.I8Matrix(n, self.h), torch.empty(n, self.h, dtype=dtype, device="cuda"),
                [torch.empty(n, w.rows, dtype=dtype, device="cuda") for w in self.w])

    def reference(self, x, res, idx):
        h = (x.double() + res.double()).to(x.dtype)
        v = Q.rmsnorm(h, self.gamma, 1e-5)
        y = torch.from_numpy(v).to(x.dtype)
        codes = Q.quantise(v)
        return h, [linear_reference(wl.LinearCase("layer", y, W, c.adapters, idx), codes) for W, c in zip(self.W, self.case)]


@pytest.mark.parametrize("n", [1, 6, 50, 300])
def test_norm_and_projections(lib, n):
    """As they are used: the norm's codes and values go to the projections, on another stream than the default."""
    dtype = torch.bfloat16
    layer = Layer(lib, 256, dtype, 11)
    x, res = gauss(n, 256, 1).to(dtype), gauss(n, 256, 2, scale=2.0).to(dtype)
    idx = torch.randint(-1, 5, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
    stream = torch.cuda.Stream()
    q, y, out = layer.buffers(n, dtype)
    xd, rd, di = x.cuda(), res.cuda(), idx.cuda()
    torch.cuda.synchronize()
    seg = layer.pools[0].segment(di, stream=stream)
    layer.run(xd, rd, seg, q, y, out, stream=stream)
    stream.synchronize()
    h, refs = layer.reference(x, res, idx)
    assert torch.equal(rd.cpu(), h)
    for got, (ref, bound) in zip(out, refs):
        # y (the LoRA term's input) may round the other way where float32 and float64 differ: a unit of the LoRA term
        err = np.abs(got.cpu().double().numpy() - ref)
        assert (err <= 2 * bound + 2.0 ** -7 * np.abs(ref).max() * 0.01).all()
    for p in layer.pools:
        p.close()


@pytest.mark.parametrize("n,h_in,r_max", [(1, 512, 8), (8, 4096, 256), (8, 512, 8), (64, 4096, 64), (256, 2048, 32), (300, 1024, 16),
                                          (1500, 512, 16)])
@pytest.mark.parametrize("with_xq", [False, True])
def test_linears_of_what_was_just_written(lib, n, h_in, r_max, with_xq):
    """Kernels start before those ahead of them end: back to back, every call still sees its own x, and nothing that it
    shares with the call before is overwritten under that one."""
    case = wl.random_case(n, n, h_in, 264, [r_max] * 20, r_max=r_max, dtype=torch.bfloat16, p_base=0.1)
    pool = make_pool(lib, case)
    w, ones = stored(lib, case.W), torch.ones(h_in, dtype=torch.bfloat16, device="cuda")
    seg, ws = pool.segment(case.idx.cuda()), pool.i8_linear_workspace(n)
    xs = [(case.x.float() * f).roll(f, 0).to(torch.bfloat16).cuda() for f in (1, 2, 3, 4, 5)]
    x, q = torch.empty_like(xs[0]), lib.I8Matrix(n, h_in)

    def chain(wait):
        out = []
        for src in xs:
            lib.lora_i8_rmsnorm(src, ones, 1e-5, out=q, y=x)
            wait()
            out.append(pool.i8_linear(w, x, seg, xq=q if with_xq else None, ws=ws))
            wait()
        torch.cuda.synchronize()
        return out

    apart = chain(torch.cuda.synchronize)
    for _ in range(4):
        for a, b in zip(chain(lambda: None), apart):
            assert torch.equal(a, b)
    pool.close()


def test_two_graphs_and_an_eager_call_share_nothing(lib):
    """Two captured layers replayed on two streams at once, an eager call between them: each its own result."""
    dtype = torch.bfloat16
    layer = Layer(lib, 512, dtype, 21)
    runs = []
    for n, seed in ((20, 1), (300, 2)):
        x, res = gauss(n, 512, seed).to(dtype).cuda(), gauss(n, 512, seed + 7).to(dtype).cuda()
        idx = torch.randint(-1, 5, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()
        seg = layer.pools[0].segment(idx)
        want_res = res.clone()
        q, y, want = layer.buffers(n, dtype)
        layer.run(x, want_res, seg, q, y, want)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        q, y, out = layer.buffers(n, dtype)
        r = res.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.run(x, r, seg, q, y, out)
        runs.append((graph, stream, x, res, r, seg, q, y, out, want, want_res))
    eager = layer.buffers(20, dtype)
    for _ in range(20):
        for run in runs:
            run[4].copy_(run[3])
            for o in run[8]:
                o.zero_()
        er = runs[0][3].clone()
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        layer.run(runs[0][2], er, runs[0][5], *eager)
        torch.cuda.synchronize()
        for _, _, _, _, r, _, _, _, out, want, want_res in runs:
            assert torch.equal(r, want_res)
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(eager[2], runs[0][9]))
    for p in layer.pools:
        p.close()


def test_repeated_calls_give_the_same_bits(lib):
    for n in (1, 30, 200, 400, 3000):
        case = wl.random_case(n, n, 1032, 392, [16] * 10, r_max=16, dtype=torch.float16, p_base=0.2)
        pool = make_pool(lib, case)
        w, x = stored(lib, case.W), case.x.cuda()
        seg = pool.segment(case.idx.cuda())
        first = pool.i8_linear(w, x, seg)
        for _ in range(5):
            assert torch.equal(pool.i8_linear(w, x, seg), first)
        pool.close()


def test_weights_quantised_right_before_their_product(lib):
    """The products load their weight ahead of the kernel before them: a weight just stored is complete all the same."""
    x = gauss(64, 2048, 1, torch.bfloat16).cuda()
    for n in (2, 64):
        q = lib.lora_i8_quantize(x[:n], lib.I8Matrix(n, 2048))
        w = lib.I8Matrix(1024, 2048)
        y = torch.empty(n, 1024, device="cuda")
        pool = lib.LoraPool(2048, 1024, 8, 1, torch.bfloat16, "cuda")
        seg = pool.segment(torch.full((n,), -1, dtype=torch.int32, device="cuda"))
        for seed in range(6):
            W = torch.randn(1024, 2048, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()
            torch.cuda.synchronize()
            lib.lora_i8_quantize(W, w)
            lib.lora_i8_matmul(q, w, y)
            lib.lora_i8_quantize(-W, w)
            z = pool.i8_linear(w, x[:n], seg)
            # (whole-number sums: of products of values, 64 bits each, float64 would round sums that are 0)
            (cx, sx), (cw, sw) = Q.quantise(x[:n]), Q.quantise(W)
            ref = torch.from_numpy(Q.sums(cx, cw) * sx.astype(np.float64)[:, None] * sw.astype(np.float64))
            assert ((y.cpu().double() - ref).abs() <= 2.0 ** -20 * ref.abs() + 1e-30).all()
            assert ((z.cpu().double() + ref).abs() <= 2.0 ** -7.9 * ref.abs() + 1e-30).all()
        pool.close()


FIRST = """
import torch, sys
import adapter_gemm_segment_gb300 as lib
n = int(sys.argv[1])
g = torch.Generator("cuda").manual_seed(1)
W, x = torch.randn(264, 512, generator=g, device="cuda").half(), torch.randn(n, 512, generator=g, device="cuda").half()
w, q, y = lib.I8Matrix(264, 512), lib.I8Matrix(n, 512), torch.zeros(n, 264, device="cuda")
pool = lib.LoraPool(512, 264, 8, 1, torch.float16, "cuda")
seg = pool.segment(torch.full((n,), -1, dtype=torch.int32, device="cuda"))
ws, lws, z = torch.empty(1 << 24, dtype=torch.uint8, device="cuda"), pool.i8_linear_workspace(n), torch.zeros(n, 264, device="cuda").half()
ones, h = torch.ones(512, device="cuda").half(), torch.empty_like(x)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    lib.lora_i8_quantize(W, w)
    lib.lora_i8_rmsnorm(x, ones, 1e-5, out=q, y=h)
    lib.lora_i8_matmul(q, w, y, ws)
    pool.i8_linear(w, h, seg, xq=q, y=z, ws=lws)
graph.replay()
torch.cuda.synchronize()
first = y.clone(), z.clone()
assert first[0].abs().sum() > 0 and torch.equal(first[0].half(), first[1])
lib.lora_i8_matmul(q, w, y, ws)
pool.i8_linear(w, h, seg, xq=q, y=z, ws=lws)
torch.cuda.synchronize()
assert torch.equal(y, first[0]) and torch.equal(z, first[1])
"""


@pytest.mark.parametrize("n", [3, 60, 700])
def test_the_first_calls_of_a_process_under_capture(n):
    out = subprocess.run([sys.executable, "-c", FIRST, str(n)], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0, out.stderr[-2000:]


def test_the_layer_example_runs():
    out = subprocess.run([sys.executable, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "i8_layer.py"),
                          "--tokens", "12", "--prefill", "600", "--adapters", "3", "--hidden", "264", "--ff", "520"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("relative difference") == 10


# ---- offsets past 32 bits ---------------------------------------------------------------------------

def test_stored_matrices_past_32_bits(lib):
    """Codes past 2^31 bytes: the last rows are those of the last rows alone, through every kernel."""
    rows, cols = 18000, 121000
    g = torch.Generator("cuda").manual_seed(1)
    W = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    last = W[-300:].clone()
    w, wl_ = lib.lora_i8_quantize(W, lib.I8Matrix(rows, cols)), lib.lora_i8_quantize(last, lib.I8Matrix(300, cols))
    assert torch.equal(w.codes[-300:], wl_.codes) and torch.equal(w.scales[-300:], wl_.scales)
    back = lib.lora_i8_dequantize(w, torch.empty_like(W))
    assert torch.equal(back[-300:], lib.lora_i8_dequantize(wl_, torch.empty_like(last)))
    gain, q = torch.randn(cols, generator=g, device="cuda").bfloat16(), lib.I8Matrix(rows, cols)
    lib.lora_i8_rmsnorm(W, gain, 1e-5, out=q, y=back)
    ql, yl = lib.I8Matrix(300, cols), torch.empty_like(last)
    lib.lora_i8_rmsnorm(last, gain, 1e-5, out=ql, y=yl)
    assert torch.equal(q.codes[-300:], ql.codes) and torch.equal(q.scales[-300:], ql.scales) and torch.equal(back[-300:], yl)
    for n in (3, 40, 600):
        x = lib.lora_i8_quantize(W[:n], lib.I8Matrix(n, cols))
        y, z = torch.empty(n, rows, device="cuda"), torch.empty(n, 300, device="cuda")
        lib.lora_i8_matmul(x, w, y)
        lib.lora_i8_matmul(x, wl_, z)
        assert torch.equal(y[:, -300:], z), n
    # ... as the many tokens of a product
    y, z = torch.empty(rows, 300, device="cuda"), torch.empty(300, 300, device="cuda")
    lib.lora_i8_matmul(w, wl_, y)
    lib.lora_i8_matmul(wl_, wl_, z)
    assert torch.equal(y[-300:], z)


@pytest.mark.parametrize("n,m", [(2, 1200000000), (500, 4500000), (70001, 40008)])
def test_outputs_past_32_bits(lib, n, m):
    """y of more than 2^31 elements: its last rows and columns."""
    g = torch.Generator("cuda").manual_seed(2)
    x, w = lib.I8Matrix(n, 16), lib.I8Matrix(m, 16)
    for q in (x, w):
        q.codes.copy_(torch.randint(-127, 128, q.codes.shape, generator=g, device="cuda", dtype=torch.int8))
        q.scales.fill_(0.25)
    y = torch.empty(n, m, device="cuda", dtype=torch.float16)
    lib.lora_i8_matmul(x, w, y)
    rows, cols = torch.arange(max(0, n - 200), n, device="cuda"), torch.arange(m - 300, m, device="cuda")
    ref = (x.codes[rows].double() @ w.codes[cols].double().T) / 16
    assert torch.equal(y[rows[:, None], cols].double(), ref.half().double())
    assert y.flatten()[2 ** 31 - 5:2 ** 31 + 5].isfinite().all()


@pytest.mark.parametrize("n", [5, 60, 700])
def test_adapters_past_32_bits(lib, n):
    """B of more than 2^31 elements: the last features of the last slots."""
    S, R, h_in, h_out, m = 100, 64, 64, 400000, 256
    g = torch.Generator("cuda").manual_seed(3)
    A = [torch.randn(R, h_in, generator=g, device="cuda").bfloat16() * 0.1 for _ in range(S)]
    Bl = [torch.randn(m, R, generator=g, device="cuda").bfloat16() * 0.1 for _ in range(S)]
    big, small = lib.LoraPool(h_in, h_out, R, S, torch.bfloat16, "cuda"), lib.LoraPool(h_in, m, R, S, torch.bfloat16, "cuda")
    B = torch.zeros(h_out, R, device="cuda", dtype=torch.bfloat16)
    for s in range(S):
        B[-m:] = Bl[s]
        big.load_slot(s, A[s], B, 2.0 * R)
        torch.cuda.synchronize()
    small.load_slots(range(S), A, Bl, [2.0 * R] * S)
    torch.cuda.synchronize()
    W = torch.randn(h_out, h_in, generator=g, device="cuda").bfloat16()
    x = torch.randn(n, h_in, generator=g, device="cuda").bfloat16()
    idx = torch.randint(S - 4, S, (n,), generator=g, device="cuda", dtype=torch.int32)
    y = big.i8_linear(lib.lora_i8_quantize(W, lib.I8Matrix(h_out, h_in)), x, big.segment(idx))
    z = small.i8_linear(lib.lora_i8_quantize(W[-m:], lib.I8Matrix(m, h_in)), x, small.segment(idx))
    # the same sums, in another order at most: both rounded to the type, and 160 float32 terms that add up to about 41
    # in magnitude (2 * 64 * 0.064 of x . A each with 64 * 0.08 of B), 160 * 41 * 2^-24 = 4e-4
    assert ((y[:, -m:].float() - z.float()).abs() <= 2.0 ** -7 * z.float().abs() + 1e-3).all()
    assert z.float().abs().mean() > 1
    big.close()
    small.close()
