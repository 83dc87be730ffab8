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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 64, 256])
@pytest.mark.parametrize("between", [False, True])
def test_a_weight_read_back_is_whole_when_a_linear_streams_it(lib, dtype, n, between):
    """lora_linear_fwd behind the read-back of its weight, whose contents change with every call; between:
    another product launched between the two."""
    h_in, h_out = 4096, 11008
    case = wl.random_case(82, n, h_in, 64, [8], r_max=8, dtype=dtype, p_base=0.2)
    pool = lib.LoraPool(h_in, h_out, 8, 1, dtype, "cuda")
    pool.load_slot(0, torch.zeros(8, h_in, dtype=dtype, device="cuda"), torch.zeros(h_out, 8, dtype=dtype, device="cuda"), 8.0)
    seg, x = pool.segment(case.idx.cuda()), case.x.cuda()
    g = torch.Generator(device="cuda").manual_seed(n)
    forms = [lib.lora_fp4_quantize(torch.randn(h_out, h_in, generator=g, device="cuda"), lib.Fp4Matrix(h_out, h_in))
             for _ in range(2)]
    W = torch.empty(h_out, h_in, dtype=dtype, device="cuda")
    small = lib.lora_fp4_quantize(torch.randn(8, 64, device="cuda"), lib.Fp4Matrix(8, 64))
    out = torch.empty(8, 8, device="cuda")
    want = []
    for q in forms:
        lib.lora_fp4_dequantize(q, W)
        torch.cuda.synchronize()
        want.append(pool.linear(W, x, seg).clone())
        torch.cuda.synchronize()
    got = [torch.empty(n, h_out, dtype=dtype, device="cuda") for _ in range(12)]
    for i, y in enumerate(got):
        lib.lora_fp4_dequantize(forms[i % 2], W)
        if between:
            lib.lora_fp4_matmul(small, small, out)
        pool.linear(W, x, seg, y=y)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    pool.close()


@pytest.mark.parametrize("rows", [100, 1000])
def test_a_product_is_whole_when_a_linear_streams_it_as_its_weight(lib, rows):
    """lora_linear_fwd over the y of lora_fp4_matmul (both its kernels), launched behind it."""
    dtype, k, h_in, n = torch.bfloat16, 512, 4096, 32
    pool = lib.LoraPool(h_in, rows // 8 * 8, 8, 1, dtype, "cuda")
    rows = rows // 8 * 8
    seg = pool.segment(torch.full((n,), -1, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(rows)
    make = lambda r: lib.lora_fp4_quantize(torch.randn(r, k, generator=g, device="cuda"), lib.Fp4Matrix(r, k))  # noqa: E731
    left, right = [make(rows) for _ in range(2)], make(h_in)
    x = torch.randn(n, h_in, generator=g, device="cuda").to(dtype)
    W = torch.empty(rows, h_in, dtype=dtype, device="cuda")
    want = []
    for q in left:
        lib.lora_fp4_matmul(q, right, W)
        torch.cuda.synchronize()
        want.append(pool.linear(W, x, seg).clone())
        torch.cuda.synchronize()
    got = [torch.empty(n, rows, dtype=dtype, device="cuda") for _ in range(12)]
    for i, y in enumerate(got):
        lib.lora_fp4_matmul(left[i % 2], right, W)
        pool.linear(W, x, seg, y=y)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    pool.close()
