"""How exactly the linear over a 4-bit base carries its shrink output s, over a base of zeros: y is then
the LoRA term alone, rounded once.

Error bound of an element, with low = s in float64, lowmag the same sum over magnitudes, and u half an
ulp of y's type: a float32 sum of h_in products, in steps of at least 16 of them or K / 128 long, is off
by (h_in / 16 + 8) 2^-22 lowmag at most; two 16-bit parts carry s to 2^-16 of itself (bfloat16) or 2^-22
and 2^-25 (float16); the R products with B add (R / 8 + 6) 2^-22 of their magnitudes; and y is rounded
once, u |y|.  One 16-bit part would carry bfloat16's s to 2^-8, as coarse as y itself."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
SPLIT = {torch.float16: (2.0 ** -22, 2.0 ** -25), torch.bfloat16: (2.0 ** -16, 0.0)}


def term_and_bound(case):
    x, idx, ad, dt = case.x.double().numpy(), case.idx.numpy(), case.adapters, case.dtype
    y, bound = np.zeros((case.n, case.h_out)), np.zeros((case.n, case.h_out))
    rel, absolute = SPLIT[dt]
    for s in range(ad.n_slots):
        t = np.nonzero(idx == s)[0]
        if t.size:
            A, B, f = ad.A[s].double().numpy(), ad.B[s].double().numpy(), ad.alphas[s] / ad.ranks[s]
            low, lowmag = f * (x[t] @ A.T), abs(f) * (np.abs(x[t]) @ np.abs(A).T)
            off = (case.h_in / 16 + 8) * 2.0 ** -22 * lowmag + rel * np.abs(low) + absolute
            y[t] = low @ B.T
            bound[t] = off @ np.abs(B).T + (ad.r_max / 8 + 6) * 2.0 ** -22 * (np.abs(low) @ np.abs(B).T)
    return y, bound + UNIT[dt] * np.abs(y) + TINY[dt]


def run(lib, case):
    pool = lib.LoraPool(case.h_in, case.h_out, case.adapters.r_max, case.adapters.n_slots, case.dtype, "cuda")
    for s in range(case.adapters.n_slots):
        pool.load_slot(s, case.adapters.A[s].cuda(), case.adapters.B[s].cuda(), case.adapters.alphas[s])
    w = lib.lora_fp4_quantize(torch.zeros_like(case.W).cuda(), lib.Fp4Matrix(case.h_out, case.h_in))
    y = pool.fp4_linear(w, case.x.cuda(), pool.segment(case.idx.cuda())).cpu().double().numpy()
    pool.close()
    return y


SIZES = [  # n, h_in, h_out, ranks, r_max, run: the per-token and the segmented shrink, every kind of product
    (1, 512, 264, [16], 16, 1), (9, 1024, 136, [8, 3], 8, 1), (60, 2048, 264, [16] * 4, 16, 1), (150, 2048, 136, [64, 8], 64, 1),
    (230, 512, 264, [16] * 3, 16, 20), (256, 512, 136, [8] * 2, 8, 1), (250, 2048, 136, [64] * 30, 64, 1),
    (300, 512, 264, [16, 5], 16, 100), (515, 768, 264, [64, 8, 16, 64], 64, 1), (400, 512, 136, [128, 24, 7], 128, 3),
    (600, 264, 520, [24] * 3, 24, 64), (700, 256, 136, [32] * 50, 32, 1)]


def build(seed, n, h_in, h_out, ranks, r_max, run, dtype, alphas=None):
    rng = np.random.default_rng([n, h_in, run])
    idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    idx[0] = 0
    return wl.random_case(seed, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, idx=idx, alphas=alphas)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_s_is_carried_more_finely_than_y(lib, size, dtype):
    case = build(61, *size, dtype)
    ref, bound = term_and_bound(case)
    err = np.abs(run(lib, case) - ref)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("size", SIZES)
def test_s_past_the_range_of_float16(lib, size):
    """One adapter's s passes 65504 while y stays below it."""
    ranks = size[3]
    alphas = [(2.0e5 if s == 0 else 2.0) * r for s, r in enumerate(ranks)]
    case = build(62, *size, torch.float16, alphas)
    ref, bound = term_and_bound(case)
    assert np.abs(ref).max() < 65504
    s = alphas[0] / ranks[0] * (case.x.double().numpy()[case.idx.numpy() == 0] @ case.adapters.A[0].double().numpy().T)
    assert np.abs(s).max() > 65520
    y = run(lib, case)
    assert np.isfinite(y).all()
    assert (np.abs(y - ref) <= bound).all(), (np.abs(y - ref) / bound).max()
