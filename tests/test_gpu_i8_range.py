"""The 8-bit operators at the ends of float32's range: a norm whose h * weight leaves it while the norm itself does
not, and a product whose sum times one scale does while the output does not."""
import numpy as np
import pytest
import torch

from oracle import i8_oracle as Q

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
WIDE = [torch.float32, torch.bfloat16]


def check_norm(lib, x, w, eps, shift=0):
    rows, cols = x.shape
    dtype = x.dtype
    buf = torch.zeros(rows * cols + shift, dtype=dtype, device="cuda")
    xd = buf[shift:].view(rows, cols)
    xd.copy_(x)
    m, y = lib.I8Matrix(rows, cols), torch.full((rows, cols), 7.0, dtype=dtype, device="cuda")
    lib.lora_i8_rmsnorm(xd, w.cuda(), eps, out=m, y=y)
    ref = Q.rmsnorm(x, w, eps)  # (float64 holds every product and square of float32 numbers)
    codes, scales = Q.quantise(ref)
    assert np.array_equal(m.scales.cpu().numpy(), scales)
    assert np.array_equal(m.codes[:, :cols].cpu().numpy(), codes) and (m.codes[:, cols:] == 0).all()
    # the product h w, the 1 / sqrt and their product rounded to float32, then to the type; below the normal range by
    # half a step of float32 and half a step of the type
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= (4 * F + UNIT[dtype]) * np.abs(ref) + TINY[dtype] + 2.0 ** -150).all()


def spread(rows, cols, seed):
    return np.random.default_rng([seed, rows, cols]).standard_normal((rows, cols))


SIZES = [(6, 40, 0), (5, 200, 1), (4, 4096, 0), (3, 9000, 3), (2, 70001, 0), (330, 520, 0)]


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("rows,cols,shift", SIZES)
@pytest.mark.parametrize("hexp,wexp", [(0, 110), (45, 95), (60, 100), (20, 120), (-60, -80), (-125, -8), (-20, -120), (40, -140), (-130, 20),
                                       (-140, 100), (-126, -149)])
def test_norm_of_products_outside_float32(lib, dtype, rows, cols, shift, hexp, wexp):
    """h * weight up to 2^170, or subnormal or zero in float32, where h / rms * weight is an ordinary number or a small
    one of the row's own."""
    x = torch.from_numpy(spread(rows, cols, 1) * 2.0 ** hexp).to(dtype)
    w = torch.from_numpy((1 + 0.2 * spread(1, cols, 2)[0]) * 2.0 ** wexp).to(dtype)
    check_norm(lib, x, w, 1e-6, shift)
    check_norm(lib, x, w, 1e-12, shift)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("cols,shift", [(64, 0), (200, 1), (4096, 0), (9000, 0)])
def test_norm_of_rows_that_span_the_range(lib, dtype, cols, shift):
    """Large elements with small weights beside small elements with large ones: their products are alike."""
    rng = np.random.default_rng(cols)
    e = rng.integers(-100, 101, cols).astype(np.float64)
    x = spread(6, cols, 3) * np.exp2(e)
    w = np.exp2(-e) * (1 + 0.2 * spread(1, cols, 4)[0])
    x[1] *= 2.0 ** 20
    x[2] *= 2.0 ** -30
    x[3, ::2] = 0
    x[4, :] = 0
    check_norm(lib, torch.from_numpy(x).to(dtype), torch.from_numpy(w).to(dtype), 1e-5, shift)
    x[4, 5] = 2.0 ** -140
    w[5] = 2.0 ** 127
    check_norm(lib, torch.from_numpy(x).to(dtype), torch.from_numpy(w).to(dtype), 1e-5, shift)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("cols,shift", [(200, 1), (2048, 0)])
@pytest.mark.parametrize("span", [3, 20, 45, 64, 90])
@pytest.mark.parametrize("hexp,wexp", [(60, 0), (0, 110), (-40, -60), (-100, 30), (30, -120)])
def test_norm_of_rows_of_every_span(lib, dtype, cols, shift, span, hexp, wexp):
    """Elements and weights spread over more and more powers of two, each by itself: from rows that one factor brings into
    range to rows that none does."""
    rng = np.random.default_rng([cols, span])

    def draw(rows, middle):
        e = np.clip(middle + rng.integers(-span, span + 1, (rows, cols)), -140, 118).astype(np.float64)
        return (1 + rng.random((rows, cols))) * np.exp2(e) * rng.choice([-1.0, 1.0], (rows, cols))

    x, w = draw(5, hexp), draw(1, wexp)[0]
    x[1, ::3] = 0
    x[2, 1:] = 0
    w[5] = 0
    check_norm(lib, torch.from_numpy(x).to(dtype), torch.from_numpy(w).to(dtype), 1e-5, shift)


@pytest.mark.parametrize("dtype", WIDE)
def test_norm_of_rows_that_are_not_finite_among_large_weights(lib, dtype):
    """An infinity in the weight or the row, beside products that overflow: NaN scale, codes 0, and the others' values."""
    x = torch.from_numpy(spread(5, 264, 5)).to(dtype)
    x[1, 3], x[2, 4] = float("inf"), float("nan")
    w = torch.from_numpy((1 + 0.1 * spread(1, 264, 6)[0]) * 2.0 ** 100).to(dtype)
    x[3] *= 2.0 ** 60
    m, y = lib.I8Matrix(5, 264), torch.empty(5, 264, dtype=dtype, device="cuda")
    lib.lora_i8_rmsnorm(x.cuda(), w.cuda(), 1e-6, out=m, y=y)
    ok = [0, 3, 4]
    ref = Q.rmsnorm(x[ok], w, 1e-6)
    codes, scales = Q.quantise(ref)
    assert np.array_equal(m.scales[ok].cpu().numpy(), scales) and np.array_equal(m.codes[ok, :264].cpu().numpy(), codes)
    assert m.scales[[1, 2]].isnan().all() and (m.codes[[1, 2]] == 0).all()
    assert y[1, 3].isnan() and (y[1, :3] == 0).all() and (y[1, 4:] == 0).all() and y[2].isnan().all()
    err = np.abs(y[ok].cpu().double().numpy() - ref)
    assert (err <= (4 * F + UNIT[dtype]) * np.abs(ref)).all()
    w[7] = float("inf")
    lib.lora_i8_rmsnorm(x.cuda(), w.cuda(), 1e-6, out=m, y=y)
    assert m.scales.isnan().all() and (m.codes == 0).all()
    assert y[0, 7].isinf() and y[3, 7].isinf() and y[0, :7].isfinite().all() and y[3, 8:].isfinite().all()


# ---- products ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 4, 8, 40, 200, 700])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("xexp,wexp", [(115, -130), (-130, 115), (100, -90), (120, -100)])
def test_products_of_a_large_and_a_small_scale(lib, n, odd, xexp, wexp):
    """The sum times x's scale is above float32's range, the output is not."""
    m, k = (257, 2100) if odd else (256, 2048)
    rng = np.random.default_rng([n, k])
    x, w = lib.I8Matrix(n, k), lib.I8Matrix(m, k)
    cx, cw = rng.integers(1, 128, (n, k)), rng.integers(1, 128, (m, k))  # sums of about 2^23
    sx = (2.0 ** xexp * (1 + rng.random(n))).astype(np.float32)
    sw = (2.0 ** wexp * (1 + rng.random(m))).astype(np.float32)
    sx[::2] = rng.random(len(sx[::2])).astype(np.float32)  # ordinary rows beside them
    for q, c, s in ((x, cx, sx), (w, cw, sw)):
        q.codes.zero_()
        q.codes[:, :k].copy_(torch.from_numpy(c.astype(np.int8)))
        q.scales.copy_(torch.from_numpy(s))
    y = torch.empty(n, m, device="cuda")
    lib.lora_i8_matmul(x, w, y)
    ref = Q.sums(cx, cw).astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    with np.errstate(over="ignore"):
        ref = np.where(np.abs(ref) > np.finfo(np.float32).max, np.inf, ref)
    got = y.cpu().double().numpy()
    # the sum, its product with one scale and with the other: three roundings
    assert np.array_equal(np.isinf(got), np.isinf(ref))
    ok = np.isfinite(ref)
    assert (np.abs(got[ok] - ref[ok]) <= 3 * F * np.abs(ref[ok]) + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("n,slots", [(3, 2), (40, 2), (200, 60), (700, 2), (700, 100)])
def test_linears_of_large_rows_and_small_weights(lib, dtype, n, slots):
    """x of 2^115 over weights of 2^-100: sums times x's scale pass 2^128."""
    h_in, h_out = 1024, 136
    x = torch.from_numpy(np.abs(spread(n, h_in, 7)) * 2.0 ** 115).to(dtype)
    W = torch.from_numpy((np.abs(spread(h_out, h_in, 8)) + 0.5) * 2.0 ** -100).to(dtype)
    x[0] = x[0] * 2.0 ** -115
    pool = lib.LoraPool(h_in, h_out, 8, slots, dtype, "cuda")
    # adapters of zeros: the LoRA term's paths, and a term that is 0
    zeros = [torch.zeros(8, h_in, dtype=dtype, device="cuda"), torch.zeros(h_out, 8, dtype=dtype, device="cuda")]
    pool.load_slots(range(slots), [zeros[0]] * slots, [zeros[1]] * slots, [8.0] * slots)
    idx = torch.randint(-1, slots, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
    w = lib.lora_i8_quantize(W.cuda(), lib.I8Matrix(h_out, h_in))
    seg = pool.segment(idx.cuda())
    y = pool.i8_linear(w, x.cuda(), seg)
    assert lib.lora_segment_status(seg) == lib.LORA_OK
    (cx, sx), (cw, sw) = Q.quantise(x), Q.quantise(W)
    ref = Q.sums(cx, cw).astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= (4 * F + UNIT[dtype]) * np.abs(ref)).all()
    pool.close()
