"""Prefill linears over a 4-bit base whose tiles of 128 tokens name more adapters than one pass of the
shrink's accumulator holds, at widths that the K split cuts unevenly (22, 36 and 28 steps of 128
columns; the last part is one step where 8 parts take three or five)."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from test_gpu_fp4 import check_linear
from test_gpu_fp4_lora_term import run as run_term, term_and_bound

pytestmark = pytest.mark.gpu

CASES = [  # n, h_in, ranks, r_max, run (0: Zipf-distributed adapters)
    (300, 2816, [64] * 12, 64, 1), (300, 2704, [64] * 9, 64, 1), (2000, 2816, [16] * 100, 16, 0), (300, 4608, [128] * 7, 128, 1),
    (4096, 2816, [64] * 8, 64, 300), (2600, 4608, [64] * 8, 64, 200), (5000, 2048, [64, 40, 64, 8, 64, 64], 64, 300),
    (8000, 1280, [128, 50] * 60, 128, 1), (300, 3584, [64] * 12, 64, 1), (700, 6400, [256, 100, 3], 256, 1)]


def build(case, dtype):
    n, h_in, ranks, r_max, run = case
    idx = None
    if run:
        rng = np.random.default_rng([n, h_in])
        idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    return wl.random_case(71, n, h_in, 136, ranks, r_max=r_max, dtype=dtype, idx=idx)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_lora_term_of_several_passes_over_uneven_parts(lib, case, dtype):
    c = build(case, dtype)
    ref, bound = term_and_bound(c)
    err = np.abs(run_term(lib, c) - ref)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] <= 700])
def test_linear_of_several_passes_over_uneven_parts(lib, case, dtype):
    c = build(case, dtype)
    assert torch.equal(check_linear(lib, c), check_linear(lib, c, with_xq=True))
