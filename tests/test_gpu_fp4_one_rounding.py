"""The linear over a 4-bit base rounds y once, whichever way the LoRA term joins the product.

Error bound: the product's float32 sums are off by (K / 64 + 2) 2^-22 of the magnitudes they add, the LoRA
term by the bound derived beside term_and_bound, their joining by R / 4 + 10 float32 steps at the
product's magnitude; y is rounded once, half an ulp.  A second rounding would add another half."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from oracle import fp4_oracle as Q
from test_gpu_fp4 import make_pool, stored
from test_gpu_fp4_lora_term import TINY, UNIT, term_and_bound

pytestmark = pytest.mark.gpu

SIZES = [  # n, h_in, h_out, ranks, r_max, run: many adapters for the batch, then few
    (250, 2048, 136, [64] * 30, 64, 1), (64, 512, 2056, [32, 5] * 60, 32, 1), (300, 512, 264, [16] * 40, 16, 1),
    (700, 256, 136, [32] * 50, 32, 1), (600, 1000, 1032, [24] * 100, 24, 7), (271, 256, 520, [8] * 17, 8, 1),
    (9, 1024, 136, [8, 3], 8, 1), (200, 512, 264, [16, 3], 16, 1), (600, 264, 520, [24] * 3, 24, 64)]


def build(size, dtype):
    n, h_in, h_out, ranks, r_max, run = size
    rng = np.random.default_rng([n, h_in, run])
    idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    case = wl.random_case(101, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, idx=idx)
    case.x[:] = case.x * 4  # a LoRA term of some weight beside the base
    return case


def reference(case):
    term, bound = term_and_bound(case)
    bound -= UNIT[case.dtype] * np.abs(term)
    xv, wv = Q.fake(case.x), Q.fake(case.W)
    base, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    ref = base + term
    steps = case.h_in / 64 + 2 + case.adapters.r_max / 4 + 10
    return ref, bound + steps * 2.0 ** -22 * mag + UNIT[case.dtype] * np.abs(ref) + TINY[case.dtype]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_y_is_rounded_once(lib, size, dtype):
    case = build(size, dtype)
    ref, bound = reference(case)
    pool = make_pool(lib, case)
    w, seg = stored(lib, case.W), pool.segment(case.idx.cuda())
    ws = torch.full((lib.lora_fp4_linear_workspace_bytes(pool.handle, case.n) + 2 * 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ybuf = torch.full((case.n + 2, case.h_out), 7.0, dtype=dtype, device="cuda")
    y = ybuf[1:-1]
    pool.fp4_linear(w, case.x.cuda(), seg, y=y, ws=ws[4096:-4096])
    assert lib.lora_segment_status(seg) == lib.LORA_OK
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= bound).all(), (err / bound).max()
    assert (ybuf[0] == 7.0).all() and (ybuf[-1] == 7.0).all()
    assert (ws[:4096] == 0xA5).all() and (ws[-4096:] == 0xA5).all()
    pool.close()


@pytest.mark.parametrize("slots,r_max,h_out", [(17, 16, 520), (100, 8, 4096), (3, 32, 64), (30, 24, 1 << 17), (2048, 8, 4096)])
def test_a_workspace_serves_every_smaller_batch(lib, slots, r_max, h_out):
    pool = lib.LoraPool(256, h_out, r_max, slots, torch.bfloat16, "cuda")
    counts = sorted(set(list(range(0, 1200)) + list(range(1200, 40000, 37)) + [16 * slots - 1, 16 * slots, 8191, 8192, 8193]))
    need = [lib.lora_fp4_linear_workspace_bytes(pool.handle, n) for n in counts]
    assert all(a <= b for a, b in zip(need, need[1:]))
    pool.close()


@pytest.mark.parametrize("n", [64, 300])
def test_nothing_is_stored_of_a_refused_batch(lib, n):
    case = wl.random_case(102, n, 512, 2056, [32] * 60, r_max=32, dtype=torch.bfloat16)
    pool = make_pool(lib, case)
    idx = case.idx.clone()
    idx[n // 2] = 60
    seg = pool.segment(idx.cuda())
    y = torch.full((n, 2056), 3.0, dtype=torch.bfloat16, device="cuda")
    pool.fp4_linear(stored(lib, case.W), case.x.cuda(), seg, y=y)
    assert lib.lora_segment_status(seg) == lib.LORA_EIDX
    assert (y == 3.0).all()
    pool.close()


def test_a_batch_without_adapters_is_the_product(lib):
    case = wl.random_case(103, 300, 512, 264, [16] * 40, r_max=16, dtype=torch.bfloat16, idx=np.full(300, -1, np.int32))
    pool = make_pool(lib, case)
    x, w = stored(lib, case.x), stored(lib, case.W)
    want = lib.lora_fp4_matmul(x, w, torch.empty(300, 264, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(pool.fp4_linear(w, case.x.cuda(), pool.segment(case.idx.cuda()), xq=x), want)
    pool.close()
