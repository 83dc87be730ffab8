"""The 8-bit oracle against exact rational arithmetic and hand-worked rows."""
from fractions import Fraction

import numpy as np
import torch

from oracle import i8_oracle as Q


def brute(row):
    """Codes and scale of one row by fractions."""
    top = max(abs(Fraction(float(v))) for v in row)
    s = np.float32(float(top) / 127)
    # nearest float32 of top / 127, checked against its neighbours
    exact = top / 127
    cands = [np.nextafter(s, np.float32(0)), s, np.nextafter(s, np.float32(np.inf))]
    assert min(cands, key=lambda c: abs(Fraction(float(c)) - exact)) == s or top == 0
    out = []
    for v in row:
        if s == 0:
            out.append(0)
            continue
        q = Fraction(float(v)) / Fraction(float(s))
        out.append(max(-127, min(127, round(q))))  # (round of a fraction: ties to even)
    return out, s


def test_codes_and_scales_are_the_exact_ones():
    rng = np.random.default_rng(0)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        for kind in range(6):
            x = torch.from_numpy(rng.standard_normal((8, 37)) * 10.0 ** rng.integers(-4, 4)).to(dtype)
            if kind == 1:  # halves of a power-of-two scale: ties
                x = torch.from_numpy(rng.integers(-254, 255, (8, 37)) / 2.0).to(dtype)
                x[:, 0] = 127
            if kind == 2:
                x = x * (torch.finfo(dtype).smallest_normal if dtype != torch.float16 else 2.0 ** -18)
            if kind == 3:
                x = torch.zeros_like(x)
            if kind == 4:
                x[:, 3] = torch.finfo(dtype).max
            c, s = Q.quantise(x)
            for r in range(8):
                want, ws = brute(x[r].double().tolist())
                assert c[r].tolist() == want and s[r] == ws


def test_rows_that_are_not_finite():
    x = torch.ones(3, 5)
    x[0, 2] = float("inf")
    x[2, 4] = float("nan")
    c, s = Q.quantise(x)
    assert np.isnan(s[[0, 2]]).all() and (c[[0, 2]] == 0).all() and (c[1] == 127).all()


def test_norm_by_hand():
    h = torch.tensor([[3.0, 4.0]])
    v = Q.rmsnorm(h, torch.tensor([1.0, 2.0]), 0.0)
    assert np.allclose(v, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]], rtol=1e-15)
    assert Q.sums(np.array([[1, -2]], np.int8), np.array([[3, 4], [-127, 127]], np.int8)).tolist() == [[-5, -381]]
