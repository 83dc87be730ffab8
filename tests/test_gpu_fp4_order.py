"""Calls over 4-bit matrices launched behind one another without waits: each reads what the ones before
it wrote, not what its buffers held earlier."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from test_gpu_fp4 import make_pool, stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max", [
    (1, 4096, 512, [8] * 3, 8), (24, 8192, 264, [16, 8], 16), (100, 1000, 136, [8] * 40, 8), (200, 8192, 512, [8, 3], 8),
    (64, 2048, 10000, [8] * 9, 8), (256, 4096, 264, [8] * 30, 8)])
def test_linear_takes_the_x_of_its_own_call(lib, dtype, n, h_in, h_out, ranks, r_max):
    """The workspace holds another x's stored form, or NaN scales, when the call is launched."""
    case = wl.random_case(81, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, p_base=0.2)
    pool = make_pool(lib, case)
    w, seg = stored(lib, case.W), pool.segment(case.idx.cuda())
    xs = [case.x.cuda(), (-3 * case.x.flip(0)).cuda()]
    want = []
    for x in xs:  # from x stored beforehand
        want.append(pool.fp4_linear(w, x, seg, xq=lib.lora_fp4_quantize(x, lib.Fp4Matrix(n, h_in))))
        torch.cuda.synchronize()
    ws = pool.fp4_linear_workspace(n)
    got = [torch.empty(n, h_out, dtype=dtype, device="cuda") for _ in range(20)]
    ws.fill_(255)
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        pool.fp4_linear(w, xs[i % 2], seg, y=y, ws=ws)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    for i in range(10):
        ws.fill_(255)
        assert torch.equal(pool.fp4_linear(w, xs[i % 2], seg, y=got[0], ws=ws), want[i % 2])
    pool.close()
