"""The 8-bit operators' contracts above 512 tokens, where the CTA-pair product takes over: with the LoRA term fused
(few adapters for the batch's size), added by a separate expand (many), and over float32 pools."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from oracle import i8_oracle as Q
from test_gpu_i8 import Layer, check_linear, gauss, linear_reference, make_pool, stored

pytestmark = pytest.mark.gpu

# (dtype, slots): the fused product, the separate expand (700 tokens, fewer than 16 a slot), float32's own
ROUTES = [(torch.float16, 2), (torch.bfloat16, 100), (torch.float32, 2), (torch.float32, 100)]


@pytest.mark.parametrize("n", [513, 700, 2100])
@pytest.mark.parametrize("dtype,slots", ROUTES)
@pytest.mark.parametrize("with_xq", [False, True])
def test_refused_batches_leave_y_untouched(lib, n, dtype, slots, with_xq):
    case = wl.random_case(n, n, 264, 136, [8] * slots, r_max=8, dtype=dtype)
    pool = make_pool(lib, case)
    idx = case.idx.clone()
    idx[n // 2] = slots
    seg = pool.segment(idx.cuda())
    y = torch.full((n, 136), 7.0, dtype=dtype, device="cuda")
    pool.i8_linear(stored(lib, case.W), case.x.cuda(), seg, xq=stored(lib, case.x) if with_xq else None, y=y)
    assert lib.lora_segment_status(seg) == lib.LORA_EIDX
    assert (y == 7.0).all()
    # the same workspace serves the next batch
    want, bound = linear_reference(case)
    got = pool.i8_linear(stored(lib, case.W), case.x.cuda(), pool.segment(case.idx.cuda()))
    assert (np.abs(got.cpu().double().numpy() - want) <= bound).all()
    pool.close()


def test_scales_that_are_not_numbers_stay_in_their_row(lib):
    for n in (700, 3000):
        x, w = gauss(n, 200, 5), gauss(150, 200, 6)
        x[1, 5] = float("inf")
        x[n - 1, 0] = float("nan")
        w[7, 9] = float("nan")
        y = torch.empty(n, 150, device="cuda")
        lib.lora_i8_matmul(stored(lib, x), stored(lib, w), y)
        want = torch.zeros(n, 150, dtype=torch.bool)
        want[[1, n - 1]] = True
        want[:, 7] = True
        assert torch.equal(y.isnan().cpu(), want)


@pytest.mark.parametrize("dtype,slots", ROUTES)
def test_adapters_that_are_not_finite_reach_their_own_tokens_only(lib, dtype, slots):
    n = 900
    case = wl.random_case(n, n, 264, 136, [8] * slots, r_max=8, dtype=dtype, p_base=0.1)
    case.idx[0], case.idx[1] = 1, 0
    ad = case.adapters
    clean = make_pool(lib, case)
    w, x = stored(lib, case.W), case.x.cuda()
    want = clean.i8_linear(w, x, clean.segment(case.idx.cuda())).cpu()
    ad.B[1][5, 3] = float("inf")
    ad.B[1][9, 0] = float("nan")
    ad.A[0][2, 7] = float("nan")
    pool = make_pool(lib, case)
    got = pool.i8_linear(w, x, pool.segment(case.idx.cuda())).cpu()
    idx = case.idx
    ok = torch.ones_like(got, dtype=torch.bool)
    ok[idx == 1, 5] = False
    ok[idx == 1, 9] = False
    ok[idx == 0] = False
    assert torch.equal(got[ok], want[ok])
    assert got[idx == 0].isnan().all()
    assert got[idx == 1][:, 9].isnan().all() and not got[idx == 1][:, 5].isfinite().any()
    clean.close()
    pool.close()


def crowded(n, h_in, h_out, slots, dtype, seed):
    """A batch whose first tokens, in the order of the segments, each have an adapter of their own, and whose other
    tokens share the last one."""
    case = wl.random_case(seed, n, h_in, h_out, [8, 3, 16, 1] * (slots // 4), r_max=16, dtype=dtype)
    idx = torch.full((n,), slots - 1, dtype=torch.int32)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))
    idx[order[:slots - 1]] = torch.arange(slots - 1, dtype=torch.int32)
    case.idx = idx
    return case


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,h_out,slots", [
    (1500, 264, 8), (5200, 264, 40),  # from 128 tokens a slot on the expand is fused, whatever the tokens name
    (5000, 1704, 256)])               # and from 16 on where y is large: a tile of 256 tokens over 256 adapters
def test_tiles_that_meet_many_adapters(lib, dtype, n, h_out, slots):
    check_linear(lib, crowded(n, 72, h_out, slots, dtype, n))


def test_tiles_of_many_adapters_that_are_not_finite(lib):
    """Infinities and NaN in some of the 39 adapters of a tile: their own tokens only."""
    n, slots, h_out = 5200, 40, 264
    case = crowded(n, 72, h_out, slots, torch.bfloat16, 3)
    clean = make_pool(lib, case)
    w, x = stored(lib, case.W), case.x.cuda()
    want = clean.i8_linear(w, x, clean.segment(case.idx.cuda())).cpu()
    bad = [3, 17, 38]
    for i, s in enumerate(bad):
        case.adapters.B[s][7 + i, 0] = (float("inf"), float("nan"), -float("inf"))[i]
    pool = make_pool(lib, case)
    got = pool.i8_linear(w, x, pool.segment(case.idx.cuda())).cpu()
    ok = torch.ones_like(got, dtype=torch.bool)
    for i, s in enumerate(bad):
        ok[case.idx == s, 7 + i] = False
        assert not got[case.idx == s, 7 + i].isfinite().any()
    assert torch.equal(got[ok], want[ok])
    clean.close()
    pool.close()


@pytest.mark.parametrize("n", [600, 1500])
def test_norm_and_projections(lib, n):
    """The norm's codes and values go to the projections, on another stream than the default."""
    dtype = torch.bfloat16
    layer = Layer(lib, 256, dtype, 11)
    x, res = gauss(n, 256, 1).to(dtype), gauss(n, 256, 2, scale=2.0).to(dtype)
    idx = torch.randint(-1, 5, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
    stream = torch.cuda.Stream()
    q, y, out = layer.buffers(n, dtype)
    xd, rd, di = x.cuda(), res.cuda(), idx.cuda()
    torch.cuda.synchronize()
    layer.run(xd, rd, layer.pools[0].segment(di, stream=stream), q, y, out, stream=stream)
    stream.synchronize()
    # the product over what the norm left, and that against the oracle
    h = (x.double() + res.double()).to(dtype)
    assert torch.equal(rd.cpu(), h)
    codes = Q.quantise(Q.rmsnorm(h, layer.gamma, 1e-5))
    assert np.array_equal(q.codes.cpu().numpy(), codes[0]) and np.array_equal(q.scales.cpu().numpy(), codes[1])
    for got, W, c in zip(out, layer.W, layer.case):
        ref, bound = linear_reference(wl.LinearCase("layer", y.cpu(), W, c.adapters, idx), codes)
        assert (np.abs(got.cpu().double().numpy() - ref) <= bound).all()
    for p in layer.pools:
        p.close()


def test_two_graphs_and_an_eager_call_share_nothing(lib):
    """Two captured layers replayed on two streams at once, an eager call between them: each its own result."""
    dtype = torch.bfloat16
    layer = Layer(lib, 512, dtype, 21)
    runs = []
    for n, seed in ((700, 1), (1300, 2)):
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
    eager = layer.buffers(700, dtype)
    for _ in range(10):
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


@pytest.mark.parametrize("dtype,slots", ROUTES)
def test_weights_quantised_right_before_their_product(lib, dtype, slots):
    """Back to back: the weight just stored is turned into float16 by the call, whole."""
    n, h_in, h_out = 700, 1024, 520
    case = wl.random_case(5, n, h_in, h_out, [8] * slots, r_max=8, dtype=dtype, p_base=0.2)
    pool = make_pool(lib, case)
    x, seg = case.x.cuda(), pool.segment(case.idx.cuda())
    q = lib.lora_i8_quantize(x, lib.I8Matrix(n, h_in))
    Ws = [(torch.randn(h_out, h_in, generator=torch.Generator().manual_seed(s)) * 0.02).to(dtype).cuda() for s in range(4)]
    apart = []
    for W in Ws:
        w = stored(lib, W)
        torch.cuda.synchronize()
        y = torch.empty(n, h_out, device="cuda")
        lib.lora_i8_matmul(q, w, y)
        torch.cuda.synchronize()
        z = pool.i8_linear(w, x, seg)
        torch.cuda.synchronize()
        apart.append((y, z))
    w = lib.I8Matrix(h_out, h_in)
    ws = torch.empty(lib.lora_i8_matmul_workspace_bytes(n, h_out, h_in), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        ys = [torch.empty(n, h_out, device="cuda") for _ in Ws]
        zs = [torch.empty(n, h_out, device="cuda", dtype=dtype) for _ in Ws]
        torch.cuda.synchronize()
        for W, y, z in zip(Ws, ys, zs):
            lib.lora_i8_quantize(W, w)
            lib.lora_i8_matmul(q, w, y, ws)
            pool.i8_linear(w, x, seg, y=z)
        torch.cuda.synchronize()
        for y, z, (a, b) in zip(ys, zs, apart):
            assert torch.equal(y, a) and torch.equal(z, b)
    pool.close()
