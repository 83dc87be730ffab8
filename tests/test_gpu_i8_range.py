"""The 8-bit operators at the ends of float32's range: a norm whose h * weight leaves it while the norm itself does
not."""
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
