"""Microscaled 4-bit matrices on the GPU against the float64 oracle.

Stored bytes are compared bit for bit (the format leaves no freedom).  The product of two stored
matrices accumulates values that are exact in float32: an output is the sum of K / 64 partial sums,
each added with a relative error of at most 2^-22 of the magnitudes involved, then rounded to its
type once.  The LoRA term adds the rounding of s to the pool's 16-bit type and, where it is added in
a second pass, one more rounding of y.
"""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from oracle import fp4_oracle as Q

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}  # half a subnormal step


def special_rows(rows, cols, dtype, seed=0):
    """Rows that meet every branch: zeros, tiny and huge blocks, ties, infinities, NaN, -0."""
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols))
    x *= np.exp2(rng.integers(-20, 10, size=(rows, (cols + 31) // 32)).repeat(32, 1)[:, :cols])
    grid = rng.choice([0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], size=(rows, cols))
    x = np.where(rng.random((rows, cols)) < 0.2, grid * rng.choice([-1, 1], size=(rows, cols)), x)
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x[rng.random((rows, cols)) < 0.02] = -0.0
    kind = rng.integers(0, 12, size=(rows, (cols + 31) // 32)).repeat(32, 1)[:, :cols]
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, x * 2.0 ** -120, x)
    t = torch.from_numpy(x).to(dtype)
    if rows * cols > 40:
        t.view(-1)[rows * cols // 2] = float("inf")
        t.view(-1)[rows * cols // 3] = float("nan")
        t[0, 0] = torch.finfo(dtype).max
        t[-1, -1] = torch.finfo(dtype).smallest_normal / 4
    return t


def guarded_matrix(lib, rows, cols):
    """A stored matrix whose buffers are exactly as long as lora_fp4_bytes says, between canaries."""
    m = lib.Fp4Matrix(rows, cols)
    nc, ns = lib.lora_fp4_bytes(rows, cols)
    bufs = []
    for n in (nc, ns):
        full = torch.full((2 * 4096 + (n + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda")
        bufs.append((full, n))
    m.codes, m.scales = (b[4096:4096 + n] for b, n in bufs)
    m.struct = lib.lora_fp4_matrix(m.codes.data_ptr(), m.scales.data_ptr(), rows, cols)
    m.bufs = bufs
    return m


def check_guards(m):
    for full, n in m.bufs:
        assert (full[:4096] == 0xA5).all() and (full[4096 + n:] == 0xA5).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (1, 4096, 0, 0), (3, 31, 0, 0), (5, 33, 0, 1), (128, 256, 0, 0), (129, 257, 0, 0), (127, 255, 1, 0),
    (64, 1000, 24, 0), (257, 1009, 31, 3), (33, 96, 8, 8), (200, 512, 0, 1)])
def test_quantize_bytes(lib, dtype, rows, cols, pad, shift):
    src = special_rows(rows, cols, dtype)
    wide = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    x = wide[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    x.copy_(src)
    m = guarded_matrix(lib, rows, cols)
    lib.lora_fp4_quantize(x, m)
    codes, scales = Q.quantise(src)
    assert np.array_equal(m.codes.cpu().numpy(), Q.pack_codes(codes))
    assert np.array_equal(m.scales.cpu().numpy(), Q.pack_scales(scales, cols))
    check_guards(m)
    # read back, into every type
    want = Q.values(codes, scales, cols)
    for out_dtype in DTYPES:
        out = torch.full((rows, cols + pad + 3), 7.0, dtype=out_dtype, device="cuda")
        lib.lora_fp4_dequantize(m, out[:, :cols])
        ref = torch.from_numpy(want).to(out_dtype)
        assert torch.equal(out[:, :cols].cpu().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
        assert (out[:, cols:] == 7.0).all()


def test_every_code_and_scale_reads_back(lib):
    """All 16 codes under all 256 scale bytes."""
    m = lib.Fp4Matrix(256, 32)
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    m.codes.copy_(torch.from_numpy(Q.pack_codes(codes)))
    m.scales.copy_(torch.from_numpy(Q.pack_scales(scales, 32)))
    want = torch.from_numpy(Q.values(codes, scales, 32))
    for dtype in DTYPES:
        out = torch.empty(256, 32, dtype=dtype, device="cuda")
        lib.lora_fp4_dequantize(m, out)
        assert torch.equal(out.cpu().nan_to_num(nan=-1.0), want.to(dtype).nan_to_num(nan=-1.0))


def test_quantize_is_the_same_for_every_dtype(lib):
    x = (torch.randn(70, 300, generator=torch.Generator().manual_seed(1)) * 3).to(torch.bfloat16)
    x = x.to(torch.float16).to(torch.bfloat16)  # values every type holds
    out = []
    for dtype in DTYPES:
        m = lib.Fp4Matrix(70, 300)
        lib.lora_fp4_quantize(x.to(dtype).cuda(), m)
        out.append((m.codes, m.scales))
    for c, s in out[1:]:
        assert torch.equal(c, out[0][0]) and torch.equal(s, out[0][1])


# ---- product ------------------------------------------------------------------------------------

def stored(lib, t):
    return lib.lora_fp4_quantize(t.cuda(), lib.Fp4Matrix(t.shape[0], t.shape[1]))


def product_bound(xv, wv, ref, dtype):
    k = xv.shape[1]
    mag = np.abs(xv) @ np.abs(wv).T
    return (k / 64 + 2) * 2.0 ** -22 * mag + UNIT[dtype] * np.abs(ref) + TINY[dtype]


def check_product(lib, x, w, dtype, pad=0):
    n, m = x.shape[0], w.shape[0]
    y = torch.full((n + 2, m + pad + 1), 7.0, dtype=dtype, device="cuda")
    yv = y[1:n + 1, :m]
    lib.lora_fp4_matmul(stored(lib, x), stored(lib, w), yv)
    xv, wv = Q.fake(x), Q.fake(w)
    ref = xv @ wv.T
    err = np.abs(yv.cpu().double().numpy() - ref)
    assert (err <= product_bound(xv, wv, ref, dtype)).all()
    assert (y[0] == 7.0).all() and (y[n + 1] == 7.0).all() and (y[1:n + 1, m:] == 7.0).all()


@pytest.mark.parametrize("k", [1, 32, 33, 255, 256, 257, 520, 1000])
@pytest.mark.parametrize("n,m,dtype", [(1, 1, 0), (1, 300, 1), (7, 129, 2), (16, 8, 0), (17, 640, 1), (64, 128, 2)])
def test_product_small_batches(lib, n, m, k, dtype):
    g = torch.Generator().manual_seed(n * 1000 + k)
    check_product(lib, torch.randn(n, k, generator=g), torch.randn(m, k, generator=g), DTYPES[dtype])


@pytest.mark.parametrize("n,m,k,dtype,pad", [
    (65, 257, 300, 0, 0), (127, 500, 1000, 1, 3), (128, 256, 512, 2, 0), (129, 255, 2048, 0, 5), (200, 4096, 1024, 2, 0),
    (255, 136, 64, 1, 0), (256, 1000, 4096, 2, 7), (257, 256, 256, 0, 0), (300, 513, 777, 1, 0), (513, 1200, 1536, 2, 0),
    (700, 2049, 100, 0, 1), (1025, 300, 3000, 2, 3), (4096, 520, 512, 1, 0)])
def test_product(lib, n, m, k, dtype, pad):
    g = torch.Generator().manual_seed(n + m + k)
    check_product(lib, torch.randn(n, k, generator=g), torch.randn(m, k, generator=g) * 0.02, DTYPES[dtype], pad)


@pytest.mark.parametrize("n", [3, 100, 400])
def test_product_long_sums(lib, n):
    """Products of one sign: the sums grow, so lost low bits would show."""
    g = torch.Generator().manual_seed(n)
    x, w = torch.rand(n, 11008, generator=g) + 0.5, torch.rand(70, 11008, generator=g) + 0.5
    check_product(lib, x, w, torch.float32)


@pytest.mark.parametrize("n", [5, 70, 300])
def test_nan_blocks_stay_in_their_rows(lib, n):
    g = torch.Generator().manual_seed(n)
    x, w = torch.randn(n, 640, generator=g), torch.randn(200, 640, generator=g)
    clean = torch.empty(n, 200, device="cuda")
    lib.lora_fp4_matmul(stored(lib, x), stored(lib, w), clean)
    x2, w2 = x.clone(), w.clone()
    x2[n // 2, 100] = float("nan")
    x2[0, 639] = float("inf")
    w2[150, 0] = -float("inf")
    y = torch.empty(n, 200, device="cuda")
    lib.lora_fp4_matmul(stored(lib, x2), stored(lib, w2), y)
    bad = torch.zeros(n, 200, dtype=torch.bool, device="cuda")
    bad[n // 2] = bad[0] = True
    bad[:, 150] = True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad], clean[~bad])


def test_product_results_do_not_depend_on_the_call(lib):
    """The same call twice, and after another product has used the chip: the same bits."""
    g = torch.Generator().manual_seed(3)
    x, w = stored(lib, torch.randn(150, 4096, generator=g)), stored(lib, torch.randn(1024, 4096, generator=g))
    a, b = (torch.empty(150, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.lora_fp4_matmul(x, w, a)
    big = stored(lib, torch.randn(2000, 512, generator=g))
    lib.lora_fp4_matmul(big, big, torch.empty(2000, 2000, device="cuda"))
    lib.lora_fp4_matmul(x, w, b)
    assert torch.equal(a, b)


# ---- the LoRA-augmented linear over a 4-bit base ---------------------------------------------------

def make_pool(lib, case):
    ad = case.adapters
    pool = lib.LoraPool(case.h_in, case.h_out, ad.r_max, ad.n_slots, case.dtype, "cuda")
    for s in range(ad.n_slots):
        pool.load_slot(s, ad.A[s].cuda(), ad.B[s].cuda(), ad.alphas[s])
    return pool


def lora_parts(case):
    """(LoRA term, sum of its products' magnitudes) in float64."""
    x, idx, ad = case.x.double().numpy(), case.idx.numpy(), case.adapters
    term, mag = np.zeros((case.n, case.h_out)), np.zeros((case.n, case.h_out))
    for s in range(ad.n_slots):
        t = np.nonzero(idx == s)[0]
        if t.size:
            A, B = ad.A[s].double().numpy(), ad.B[s].double().numpy()
            low = ad.alphas[s] / ad.ranks[s] * (x[t] @ A.T)
            lowmag = abs(ad.alphas[s] / ad.ranks[s]) * (np.abs(x[t]) @ np.abs(A).T)
            term[t] = low @ B.T
            mag[t] = np.abs(low) @ np.abs(B).T + 2.0 ** -10 * (lowmag @ np.abs(B).T)
    return term, mag


def check_linear(lib, case, with_xq=False, zero_base=False):
    pool = make_pool(lib, case)
    W = torch.zeros_like(case.W) if zero_base else case.W
    w = stored(lib, W)
    x = case.x.cuda()
    seg = pool.segment(case.idx.cuda())
    n = case.n
    ybuf = torch.full((n + 2, case.h_out), 7.0, dtype=case.dtype, device="cuda")
    y = ybuf[1:n + 1]
    ws_full = torch.full((lib.lora_fp4_linear_workspace_bytes(pool.handle, n) + 2 * 4096,), 0xA5, dtype=torch.uint8,
                         device="cuda")
    ws = ws_full[4096:-4096]
    xq = stored(lib, case.x) if with_xq else None
    lib.lora_fp4_linear_fwd(pool.handle, w, x, y, seg, ws, xq)
    assert lib.lora_segment_status(seg) == lib.LORA_OK
    xv, wv = Q.fake(case.x), Q.fake(W)
    base = xv @ wv.T
    term, mag = lora_parts(case)
    ref = base + term
    u = UNIT[case.dtype]
    bound = product_bound(xv, wv, base, case.dtype) + 2 * u * np.abs(ref) + 3 * u * mag + 2.0 ** -18 * mag + TINY[case.dtype]
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= bound).all(), (err - bound).max()
    assert (ybuf[0] == 7.0).all() and (ybuf[n + 1] == 7.0).all()
    assert (ws_full[:4096] == 0xA5).all() and (ws_full[-4096:] == 0xA5).all()
    pool.close()
    return y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max", [
    (1, 256, 256, [8], 8), (1, 4096, 512, [8] * 5, 8), (2, 72, 40, [3, 8], 8), (16, 512, 384, [8, 16, 4], 16),
    (17, 1000, 136, [16] * 6, 16), (64, 1024, 1024, [8] * 40, 8), (63, 520, 264, [8, 24, 17], 24),
    (100, 768, 512, [64, 8, 16, 64], 64), (129, 256, 640, [40, 1], 40), (200, 2048, 256, [8, 8, 16, 16, 64, 64], 64),
    (256, 512, 520, [16] * 100, 16), (48, 512, 384, [256, 100, 8], 256)])
def test_linear_decode(lib, dtype, n, h_in, h_out, ranks, r_max):
    case = wl.random_case(41, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, p_base=0.15)
    check_linear(lib, case)
    check_linear(lib, case, zero_base=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max,run", [
    (257, 256, 256, [8], 8, 1), (300, 1000, 264, [16, 5], 16, 100), (600, 512, 776, [24] * 3, 24, 64),
    (1000, 264, 520, [8] * 100, 8, 1), (515, 768, 256, [64, 8, 16, 64], 64, 1), (900, 512, 1032, [16] * 30, 16, 256),
    (384, 320, 256, [128, 7], 128, 1), (400, 512, 384, [256, 100, 8], 256, 3)])
def test_linear_prefill(lib, dtype, n, h_in, h_out, ranks, r_max, run):
    rng = np.random.default_rng([n, run])
    idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    case = wl.random_case(43, n, h_in, h_out, ranks, r_max=r_max, dtype=dtype, idx=idx)
    check_linear(lib, case)
    check_linear(lib, case, zero_base=True)


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("pattern", ["none", "one", "last"])
def test_linear_token_patterns(lib, n, pattern):
    """No token with an adapter; one adapter for all; only the last token with one."""
    idx = np.full(n, -1, np.int32)
    if pattern == "one":
        idx[:] = 2
    elif pattern == "last":
        idx[-1] = 1
    case = wl.random_case(44, n, 512, 384, [8, 16, 8], r_max=16, dtype=torch.bfloat16, idx=idx)
    check_linear(lib, case)


@pytest.mark.parametrize("n", [1, 64, 300])
@pytest.mark.parametrize("dtype", DTYPES)
def test_shared_stored_x_gives_the_same_bits(lib, n, dtype):
    case = wl.random_case(45, n, 768, 512, [8, 16], r_max=16, dtype=dtype)
    a = check_linear(lib, case)
    b = check_linear(lib, case, with_xq=True)
    assert torch.equal(a, b)


@pytest.mark.parametrize("n,r_max", [(9, 8), (150, 64), (400, 16), (400, 128)])
@pytest.mark.parametrize("poison", ["A", "B"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_broken_adapter_reaches_only_its_tokens(lib, n, r_max, poison, value):
    """An infinity or NaN in one tenant's adapter leaves every other token's row as it was."""
    ranks = [r_max, max(1, r_max // 2), r_max]
    idx = (np.arange(n) % 4 - 1).astype(np.int32)
    case = wl.random_case(46, n, 512, 264, ranks, r_max=r_max, dtype=torch.bfloat16, idx=idx)
    w, x = stored(lib, case.W), case.x.cuda()

    def run():
        pool = make_pool(lib, case)
        y = pool.fp4_linear(w, x, pool.segment(case.idx.cuda()))
        torch.cuda.synchronize()
        pool.close()
        return y

    clean = run()
    getattr(case.adapters, poison)[1].view(-1)[7] = value
    dirty = run()
    others = torch.from_numpy(idx != 1).cuda()
    assert torch.equal(dirty[others], clean[others])
    mine = dirty[~others]
    if poison == "A":
        assert not torch.isfinite(mine).all()
    else:  # one element of B: one output feature
        o = 7 // case.adapters.ranks[1]
        assert not torch.isfinite(mine[:, o]).all()
        keep = torch.arange(264, device="cuda") != o
        assert torch.equal(mine[:, keep], clean[~others][:, keep])


@pytest.mark.parametrize("n", [12, 300])
def test_a_broken_token_reaches_only_its_row(lib, n):
    case = wl.random_case(47, n, 512, 264, [16, 8], r_max=16, dtype=torch.float16, p_base=0.3)
    pool = make_pool(lib, case)
    w, seg = stored(lib, case.W), pool.segment(case.idx.cuda())
    clean = pool.fp4_linear(w, case.x.cuda(), seg)
    x = case.x.clone()
    x[n // 2, 77] = float("inf")
    dirty = pool.fp4_linear(w, x.cuda(), seg)
    assert torch.isnan(dirty[n // 2]).all()
    keep = torch.arange(n, device="cuda") != n // 2
    assert torch.equal(dirty[keep], clean[keep])
    pool.close()


@pytest.mark.parametrize("n", [5, 64, 300])
def test_invalid_idx_leaves_y_untouched(lib, n):
    case = wl.random_case(48, n, 256, 264, [8, 8], r_max=8, dtype=torch.bfloat16)
    pool = make_pool(lib, case)
    idx = case.idx.clone()
    idx[n - 1] = 2
    seg = pool.segment(idx.cuda())
    y = torch.full((n, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    pool.fp4_linear(stored(lib, case.W), case.x.cuda(), seg, y=y)
    assert lib.lora_segment_status(seg) == lib.LORA_EIDX
    assert (y == 3.0).all()
    pool.close()


def test_linear_refusals_and_no_tokens(lib):
    case = wl.random_case(49, 20, 256, 264, [8, 8], r_max=8, dtype=torch.bfloat16)
    pool = make_pool(lib, case)
    seg = pool.segment(case.idx.cuda())
    w, x = stored(lib, case.W), case.x.cuda()
    y = torch.full((20, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = pool.fp4_linear_workspace(20)

    def refuses(code, **kw):
        a = dict(w=w, x=x, y=y, seg=seg, ws=ws, xq=None)
        a.update(kw)
        with pytest.raises(lib.LoraError) as e:
            lib.lora_fp4_linear_fwd(pool.handle, a["w"], a["x"], a["y"], a["seg"], a["ws"], a["xq"])
        assert e.value.code == code

    refuses(lib.LORA_EINVAL, w=lib.Fp4Matrix(264, 255))
    refuses(lib.LORA_EINVAL, w=lib.Fp4Matrix(256, 256))
    refuses(lib.LORA_EINVAL, xq=lib.Fp4Matrix(19, 256))
    refuses(lib.LORA_EINVAL, x=x.view(-1)[1:])
    refuses(lib.LORA_EINVAL, y=y.view(-1)[1:])
    refuses(lib.LORA_EINVAL, ws=ws[16:])
    refuses(lib.LORA_ENOSPACE, ws=ws[:lib.lora_fp4_linear_workspace_bytes(pool.handle, 20) - 1])
    other = lib.LoraPool(256, 264, 8, 3, torch.bfloat16, "cuda")
    refuses(lib.LORA_EINVAL, seg=other.segment(torch.full((20,), -1, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    assert (y == 3.0).all()
    empty = pool.segment(torch.empty(0, dtype=torch.int32, device="cuda"))
    out = pool.fp4_linear(w, x[:0], empty)
    assert out.shape == (0, 264)
    with pytest.raises(ValueError):
        lib.lora_fp4_quantize(case.x, lib.Fp4Matrix(20, 256))  # host memory
    with pytest.raises(ValueError):
        lib.lora_fp4_quantize(x.t(), lib.Fp4Matrix(256, 20))  # rows not contiguous
    with pytest.raises(ValueError):
        lib.lora_fp4_quantize(x.double(), lib.Fp4Matrix(20, 256))
    pool.close()


@pytest.mark.parametrize("n", [1, 64, 300])
def test_other_stream_and_graph_replay(lib, n):
    """On a side stream behind the producer of x, and captured once and replayed on new inputs."""
    case = wl.random_case(50, n, 1024, 520, [8, 16, 8], r_max=16, dtype=torch.float16)
    pool = make_pool(lib, case)
    w, x = stored(lib, case.W), case.x.cuda()
    ref = pool.fp4_linear(w, x, pool.segment(case.idx.cuda())).clone()
    other = pool.fp4_linear(w, 2 * x, pool.segment(case.idx.cuda())).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xs, y = torch.empty_like(x), torch.empty_like(ref)
    idx, ws, segws = case.idx.cuda(), pool.fp4_linear_workspace(n), pool.segment_workspace(n)
    with torch.cuda.stream(side):
        for _ in range(3):
            xs.zero_()
            xs.copy_(x)
            seg = pool.segment(idx, segws)
            pool.fp4_linear(w, xs, seg, y=y, ws=ws)
        side.synchronize()
        assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seg = pool.segment(idx, segws)
        pool.fp4_linear(w, xs, seg, y=y, ws=ws)
        pool.fp4_linear(w, xs, seg, y=y, ws=ws)
    for scale, want in ((1, ref), (2, other), (1, ref)):
        xs.copy_(x * scale)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    pool.close()


def test_chained_linears(lib):
    """Each linear reads what the one before it wrote, launched without waits in between."""
    case = wl.random_case(51, 64, 512, 512, [8, 16, 8], r_max=16, dtype=torch.bfloat16)
    pool = make_pool(lib, case)
    w = stored(lib, case.W)
    seg = pool.segment(case.idx.cuda())
    ws = pool.fp4_linear_workspace(64)
    bufs = [torch.empty(64, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def chain(sync):
        bufs[0].copy_(case.x)
        for i in range(6):
            pool.fp4_linear(w, bufs[i % 2], seg, y=bufs[(i + 1) % 2], ws=ws)
            if sync:
                torch.cuda.synchronize()
        return bufs[0].clone()

    slow = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), slow)
    pool.close()


def test_large_offsets(lib):
    """Elements past the 2^31st byte of x, codes and y are addressed with 64 bits."""
    rows, cols = 70000, 16640  # 2.3 GB of float16, 1.16 G elements
    x = torch.zeros(rows, cols, dtype=torch.float16, device="cuda")
    x[-1] = 3.0
    x[-2, -1] = -6.0
    m = lib.lora_fp4_quantize(x, lib.Fp4Matrix(rows, cols))
    x.fill_(1.0)
    lib.lora_fp4_dequantize(m, x)
    assert (x[-1] == 3.0).all() and x[-2, -1] == -6.0 and (x[-3] == 0).all() and x[-2, :-1].abs().max() == 0
    del x
    w = stored(lib, torch.ones(16640, 64))
    big = stored(lib, torch.ones(70000, 64))
    y = torch.empty(70000, 16640, dtype=torch.bfloat16, device="cuda")
    lib.lora_fp4_matmul(big, w, y)
    assert (y[-1] == 64).all() and bool((y.sum(1, dtype=torch.float32) == 64.0 * 16640).all())


# ---- sizes at which the calls above change their path --------------------------------------------

@pytest.mark.parametrize("n,m,k,dtype,pad", [
    (225, 136, 300, 0, 0), (240, 1000, 8192, 1, 1), (240, 300, 8200, 2, 0), (256, 1, 33, 0, 0), (65, 9736, 256, 2, 0),
    (64, 9736, 256, 1, 0), (100, 11008, 130, 0, 3), (224, 264, 512, 1, 0)])
def test_product_between_small_and_large(lib, n, m, k, dtype, pad):
    g = torch.Generator().manual_seed(n + m + k)
    check_product(lib, torch.randn(n, k, generator=g), torch.randn(m, k, generator=g) * 0.02, DTYPES[dtype], pad)


HEAVY = [  # n, h_in, ranks, r_max, run: small batches with many rows of A, and of few or many adapters
    (64, 2048, [64, 8, 32], 64, 1), (200, 2048, [64, 8, 16, 64, 33, 1], 64, 1), (129, 11008, [40] * 3, 40, 43),
    (256, 4096, [8], 8, 256), (250, 1000, [256, 100], 256, 1), (33, 1032, [256, 3], 256, 2), (256, 520, [128, 64, 1], 128, 7),
    (250, 2048, [64] * 30, 64, 1)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,h_in,ranks,r_max,run", HEAVY)
def test_linear_small_batches_of_high_rank(lib, dtype, n, h_in, ranks, r_max, run):
    rng = np.random.default_rng([n, h_in])
    idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    case = wl.random_case(51, n, h_in, 264, ranks, r_max=r_max, dtype=dtype, idx=idx)
    a = check_linear(lib, case)
    assert torch.equal(a, check_linear(lib, case, with_xq=True))
    check_linear(lib, case, zero_base=True)


@pytest.mark.parametrize("n,h_in,slots,r_max", [(200, 2048, 3, 64), (250, 2048, 30, 64), (300, 512, 40, 16), (700, 256, 100, 32)])
@pytest.mark.parametrize("poison", ["A", "B", "x"])
def test_a_broken_input_stays_with_its_tokens(lib, n, h_in, slots, r_max, poison):
    """A NaN in one tenant's adapter, or in one token, at the sizes of the paths above."""
    idx = (np.arange(n) % (slots + 1) - 1).astype(np.int32)
    case = wl.random_case(52, n, h_in, 136, [r_max] * slots, r_max=r_max, dtype=torch.float16, idx=idx)
    w = stored(lib, case.W)

    def run():
        pool = make_pool(lib, case)
        y = pool.fp4_linear(w, case.x.cuda(), pool.segment(case.idx.cuda()))
        torch.cuda.synchronize()
        pool.close()
        return y

    clean = run()
    if poison == "x":
        case.x[n - 2, 5] = float("nan")
        own = np.arange(n) == n - 2
    else:
        getattr(case.adapters, poison)[1].view(-1)[3] = float("nan")
        own = idx == 1
    dirty = run()
    others = torch.from_numpy(~own).cuda()
    assert torch.equal(dirty[others], clean[others])
    assert torch.isnan(dirty[~others]).any(dim=1).all()


@pytest.mark.parametrize("n,h_in,slots,r_max", [(200, 2048, 3, 64), (256, 4096, 2, 8), (300, 512, 40, 16)])
@pytest.mark.parametrize("what", ["none", "last", "invalid"])
def test_patterns_at_those_sizes(lib, n, h_in, slots, r_max, what):
    idx = np.full(n, -1, np.int32)
    if what == "last":
        idx[-1] = slots - 1
    case = wl.random_case(53, n, h_in, 136, [r_max] * slots, r_max=r_max, dtype=torch.bfloat16, idx=idx)
    if what != "invalid":
        check_linear(lib, case)
        return
    pool = make_pool(lib, case)
    bad = case.idx.clone()
    bad[0] = slots
    seg = pool.segment(bad.cuda())
    y = torch.full((n, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    pool.fp4_linear(stored(lib, case.W), case.x.cuda(), seg, y=y)
    assert lib.lora_segment_status(seg) == lib.LORA_EIDX
    assert (y == 3.0).all()
    pool.close()


@pytest.mark.parametrize("n,h_in,h_out,ranks,r_max,run", [
    (6000, 64, 1031, [40, 7, 33], 41, 100), (9000, 40, 392, [8] * 3, 8, 1), (5000, 300, 776, [256, 16], 256, 512),
    (40, 3000, 136, [8] * 2, 8, 1), (300, 5000, 72, [20] * 9, 20, 3)])
def test_linear_float32_tiles(lib, n, h_in, h_out, ranks, r_max, run):
    """Several feature tiles a CTA of the float32 expand, and many K parts of its shrink."""
    rng = np.random.default_rng([n, h_out])
    idx = np.repeat(rng.integers(-1, len(ranks), size=(n + run - 1) // run), run)[:n]
    case = wl.random_case(54, n, h_in, h_out, ranks, r_max=r_max, dtype=torch.float32, idx=idx)
    check_linear(lib, case)
    check_linear(lib, case, zero_base=True)


@pytest.mark.parametrize("h_in,h_out,slots,r_max,dtype", [
    (1024, 64, 4, 256, 0), (4096, 4096, 100, 8, 0), (2048, 512, 30, 64, 1), (8192, 256, 3, 16, 2), (64, 64, 1, 8, 0)])
def test_a_workspace_serves_every_smaller_batch(lib, h_in, h_out, slots, r_max, dtype):
    pool = lib.LoraPool(h_in, h_out, r_max, slots, DTYPES[dtype], "cuda")
    counts = list(range(0, 2000)) + list(range(2000, 50000, 61)) + [1 << 17]
    need = [lib.lora_fp4_linear_workspace_bytes(pool.handle, n) for n in sorted(counts)]
    assert all(a <= b for a, b in zip(need, need[1:]))
    pool.close()


def test_one_workspace_for_batches_of_many_sizes(lib):
    """Batches of every path in a workspace sized for the largest."""
    case = wl.random_case(55, 700, 1024, 136, [8, 24, 64], r_max=64, dtype=torch.float32, p_base=0.2)
    pool = make_pool(lib, case)
    w, ws = stored(lib, case.W), pool.fp4_linear_workspace(700)
    for n in (700, 1, 64, 200, 300, 513):
        x, seg = case.x[:n].cuda(), pool.segment(case.idx[:n].cuda())
        assert torch.equal(pool.fp4_linear(w, x, seg, ws=ws), pool.fp4_linear(w, x, seg))
    pool.close()
