"""Cases of the microscaled 4-bit operators: what is timed and against which plain form.

The multi-LoRA linear streams a frozen base weight; held in microscaled 4-bit floating point
(MXFP4: 32 consecutive elements of a row share one power-of-two scale, every element is one of
0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) it takes 4.25 bits an element instead of 16.

  roundtrip   quantise rows, then read them back (both calls of one pass)
  readback    read a stored 4-bit matrix back
  matmul      y = Xq Wq^T of two stored 4-bit matrices
  linear      y = Q(x) Wq^T + (alpha/r) (x A_s^T) B_s^T: the LoRA-augmented linear over a 4-bit
              base, every token naming its adapter slot s (or none)

Shapes are those of the 7B-shaped layer the benchmark uses (4096 and 11008 wide, 1 to 64 tokens
at decode, 256 for a large batch, 32 x 512 tokens of prefill, 100 adapters of rank 8 or 16, mixed
ranks padded to 64).
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decode token's activations: two calls whose latency is all that counts
        dict(name="roundtrip_token", op="roundtrip", rows=1, cols=4096, ld=4096, dtype="f16"),
        # a column window of a wider float32 buffer: odd width, the last block is not whole
        dict(name="roundtrip_window", op="roundtrip", rows=257, cols=1009, ld=1040, dtype="f32"),
        # the activations of a prefill batch (32 requests of 512 tokens)
        dict(name="roundtrip_prefill", op="roundtrip", rows=16384, cols=4096, ld=4096, dtype="bf16"),
        # a small ragged matrix read back
        dict(name="readback_small", op="readback", rows=100, cols=1000, dtype="f32"),
        # the up projection's weight read back, as for merging an adapter into it
        dict(name="readback_weight", op="readback", rows=11008, cols=4096, dtype="bf16"),
        # one decode token without an adapter through q_proj
        dict(name="matmul_token", op="matmul", n=1, h_in=4096, h_out=4096, dtype="f16"),
        # a 256-token decode batch through the up projection
        dict(name="matmul_batch", op="matmul", n=256, h_in=4096, h_out=11008, dtype="bf16"),
        # a prefill batch through the down projection, float32 out, a token count off every tile
        dict(name="matmul_prefill", op="matmul", n=8191, h_in=11008, h_out=4096, dtype="f32"),
        # one decode token with its adapter
        dict(name="linear_token", op="linear", n=1, h_in=4096, h_out=4096, slots=100, r_max=8, mixed=False,
             run=1, p_base=0.0, dtype="f16"),
        # the decode batch of the benchmark: 64 tokens, 100 adapters, 10 % without one
        dict(name="linear_decode", op="linear", n=64, h_in=4096, h_out=4096, slots=100, r_max=8, mixed=False,
             run=1, p_base=0.1, dtype="f16"),
        # adapters of ranks 8, 16 and 64 in one batch, through the down projection
        dict(name="linear_mixed", op="linear", n=200, h_in=11008, h_out=4096, slots=6, r_max=64, mixed=True,
             run=1, p_base=0.15, dtype="bf16"),
        # the prefill batch of the benchmark: 32 requests of 512 tokens, one adapter each
        dict(name="linear_prefill", op="linear", n=16384, h_in=4096, h_out=4096, slots=100, r_max=16, mixed=False,
             run=512, p_base=0.0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["roundtrip", "readback", "matmul", "matmul", "linear", "linear", "linear"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("roundtrip", "readback"):
        cols = _log(rng, 1, 11008)
        rows = _log(rng, 1, max(1, min(16384, 16384 * 4096 // cols)))
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype)
        if op == "roundtrip":
            case["ld"] = cols + rng.choice([0, 0, 1, 8, 24, 100])
        return case
    if op == "matmul":
        h_in = _log(rng, 32, 11008)
        h_out = _log(rng, 8, 11008)
        n = _log(rng, 1, min(16384, 16384 * 4096 * 4096 // (h_in * h_out)))
        return dict(op=op, n=n, h_in=h_in, h_out=h_out, dtype=dtype)
    h_in = max(8, _log(rng, 64, 11008) // 8 * 8)
    h_out = max(8, _log(rng, 64, 11008) // 8 * 8)
    n = _log(rng, 1, min(16384, 16384 * 4096 * 4096 // (h_in * h_out)))
    r_max = rng.choice([8, 16, 24, 32, 64])
    return dict(op=op, n=n, h_in=h_in, h_out=h_out, slots=_log(rng, 1, 100), r_max=r_max,
                mixed=rng.choice([True, False]), run=rng.choice([1, 1, 7, 64, 512]),
                p_base=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)


def _stored(rows, cols):
    """Bytes of a stored matrix: 16 bytes of codes and one of scale a block of 32."""
    return rows * ((cols + 31) // 32) * 17


def work(case):
    es = ES[case["dtype"]]
    if case["op"] in ("roundtrip", "readback"):
        r, c = case["rows"], case["cols"]
        if case["op"] == "readback":
            return {"bytes": _stored(r, c) + r * c * es, "flops": r * c}
        # the rows in, the stored form out and in again, the values out
        return {"bytes": 2 * r * c * es + 2 * _stored(r, c), "flops": 3 * r * c}
    n, hi, ho = case["n"], case["h_in"], case["h_out"]
    base = _stored(ho, hi) + n * ho * es
    if case["op"] == "matmul":
        return {"bytes": base + _stored(n, hi), "flops": 2 * n * hi * ho}
    # the adapters a batch is expected to name, at their ranks
    ranks = _ranks(case)
    p = np.arange(1, case["slots"] + 1, dtype=np.float64) ** -1.1
    p = p / p.sum() * (1.0 - case["p_base"])
    draws = (n + case["run"] - 1) // case["run"]
    named = float(np.sum((1.0 - (1.0 - p) ** draws) * np.array(ranks)))
    mean_rank = float(np.sum(p * np.array(ranks)))
    return {"bytes": int(base + n * hi * es + named * (hi + ho) * es),
            "flops": int(2 * n * hi * ho + 2 * n * mean_rank * (hi + ho))}


# ---- inputs ---------------------------------------------------------------------------------

def _gen(seed, *key):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + sum((i + 1) * 7919 * int(k) for i, k in enumerate(key))) % (2 ** 62))
    return g


def _activations(g, rows, cols, dtype):
    """Normal activations with a few loud channels and a few silent stretches."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    x *= torch.where(loud, 12.0, 1.0)
    silent = torch.rand(cols // 32 + 1, generator=g, device="cuda") < 0.01
    x.masked_fill_(silent.repeat_interleave(32)[:cols], 0.0)
    return x.to(DT[dtype])


def _weight(g, rows, cols, dtype):
    return (torch.randn(rows, cols, generator=g, device="cuda") * 0.02).to(DT[dtype])


def _ranks(case):
    full = [case["r_max"]] * case["slots"]
    if not case["mixed"]:
        return full
    steps = [max(1, case["r_max"] // 8), max(1, case["r_max"] // 4), case["r_max"]]
    return [steps[s % 3] for s in range(case["slots"])]


def _adapters(case, g):
    """Stacked adapters [slots, r_max, .] (rows past an adapter's rank are zero) and alpha / r."""
    S, R, hi, ho, dt = case["slots"], case["r_max"], case["h_in"], case["h_out"], DT[case["dtype"]]
    ranks = _ranks(case)
    A = ((torch.rand(S, R, hi, generator=g, device="cuda") * 2 - 1) / math.sqrt(hi)).to(dt)
    B = (torch.randn(S, ho, R, generator=g, device="cuda") * 0.01).to(dt)
    live = torch.arange(R, device="cuda")[None, :] < torch.tensor(ranks, device="cuda")[:, None]
    A *= live[:, :, None]
    B *= live[:, None, :]
    return A, B, ranks, [2.0 * r for r in ranks]


def _slots_of(case, seed):
    """The adapter slot of every token: Zipf(1.1) per run of tokens, -1 for none."""
    rng = np.random.default_rng([int(seed), case["n"], case["slots"]])
    p = np.arange(1, case["slots"] + 1, dtype=np.float64) ** -1.1
    runs = (case["n"] + case["run"] - 1) // case["run"]
    slot = rng.choice(case["slots"], size=runs, p=p / p.sum())
    slot[rng.random(runs) < case["p_base"]] = -1
    idx = np.repeat(slot, case["run"])[:case["n"]].astype(np.int32)
    return torch.from_numpy(idx).cuda()


def _inputs(case, seed):
    op = case["op"]
    if op in ("roundtrip", "readback"):
        g = _gen(seed, case["rows"], case["cols"])
        if op == "readback":
            return {"src": _weight(g, case["rows"], case["cols"], case["dtype"])}
        wide = _activations(g, case["rows"], case["ld"], case["dtype"])
        return {"x": wide[:, :case["cols"]]}
    g = _gen(seed, case["n"], case["h_in"], case["h_out"])
    d = {"x": _activations(g, case["n"], case["h_in"], case["dtype"]),
         "w": _weight(g, case["h_out"], case["h_in"], case["dtype"])}
    if op == "linear":
        d["A"], d["B"], d["ranks"], d["alphas"] = _adapters(case, g)
        d["idx"] = _slots_of(case, seed)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    st = {"case": case}
    if not own:
        if op == "roundtrip":
            st["x"] = d["x"]
        elif op == "readback":
            st["q"] = _pack(d["src"])
        else:
            st["w"] = _pack(d["w"])
            if op == "matmul":
                st["x"] = _pack(d["x"])
            else:
                st["x"], st["idx"] = d["x"], d["idx"]
                st["A"], st["B"] = d["A"], d["B"]
                st["scale"] = torch.tensor([a / r for a, r in zip(d["alphas"], d["ranks"])], device="cuda")
        return st

    import adapter_gemm_segment_gb300 as ags

    st["ags"] = ags
    dt = DT[case["dtype"]]
    if op == "roundtrip":
        st["x"] = d["x"]
        st["q"] = ags.Fp4Matrix(case["rows"], case["cols"], "cuda")
        st["out"] = torch.empty(case["rows"], case["cols"], dtype=dt, device="cuda")
    elif op == "readback":
        st["q"] = ags.lora_fp4_quantize(d["src"], ags.Fp4Matrix(case["rows"], case["cols"], "cuda"))
        st["out"] = torch.empty(case["rows"], case["cols"], dtype=dt, device="cuda")
    else:
        n, hi, ho = case["n"], case["h_in"], case["h_out"]
        st["w"] = ags.lora_fp4_quantize(d["w"], ags.Fp4Matrix(ho, hi, "cuda"))
        st["y"] = torch.empty(n, ho, dtype=dt, device="cuda")
        if op == "matmul":
            st["x"] = ags.lora_fp4_quantize(d["x"], ags.Fp4Matrix(n, hi, "cuda"))
        else:
            st["x"] = d["x"]
            pool = ags.LoraPool(hi, ho, case["r_max"], case["slots"], dt, "cuda")
            pool.load_slots(range(case["slots"]), [d["A"][s, :r].contiguous() for s, r in enumerate(d["ranks"])],
                            [d["B"][s, :, :r].contiguous() for s, r in enumerate(d["ranks"])], d["alphas"])
            st["pool"] = pool
            # the segments of a batch: built once, shared by every linear the batch runs through
            st["seg"] = pool.segment(d["idx"])
            st["ws"] = pool.fp4_linear_workspace(n)
    return st


def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    ags, op = st["ags"], st["case"]["op"]
    if op == "roundtrip":
        ags.lora_fp4_quantize(st["x"], st["q"])
        return ags.lora_fp4_dequantize(st["q"], st["out"])
    if op == "readback":
        return ags.lora_fp4_dequantize(st["q"], st["out"])
    if op == "matmul":
        return ags.lora_fp4_matmul(st["x"], st["w"], st["y"])
    return ags.lora_fp4_linear_fwd(st["pool"].handle, st["w"], st["x"], st["y"], st["seg"], st["ws"])


# ---- the plain form -------------------------------------------------------------------------

def _quantise(x):
    """float32 rows -> (signed element values, scale exponents) of blocks of 32; a block with an
    infinity or a NaN has a NaN scale."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    f = torch.zeros(rows, nb * 32, device=x.device)
    f[:, :cols] = x
    f = f.view(rows, nb, 32)
    amax = f.abs().amax(-1)
    e = torch.frexp(amax).exponent - 3  # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    v = f * torch.exp2(-e.float())[..., None]
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step  # ties to even, which is the even code
    bad = ~torch.isfinite(f).all(-1)
    a = torch.where(bad[..., None], torch.zeros_like(a), a)
    return torch.copysign(a, f), e, bad


def _pack(x):
    """A stored matrix: two codes a byte (low half first), one scale byte a block."""
    rows, cols = x.shape
    v, e, bad = _quantise(x.float())
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    code = torch.searchsorted(grid, v.abs().contiguous()).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = code.view(rows, -1)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return {"codes": packed, "scales": scale, "cols": cols}


def _unpack(q):
    """float32 values of a stored matrix."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=q["codes"].device)
    rows, half = q["codes"].shape
    v = torch.empty(rows, half, 2, device=q["codes"].device)
    v[..., 0] = table[(q["codes"] & 15).int()]
    v[..., 1] = table[(q["codes"] >> 4).int()]
    s = torch.exp2(q["scales"].float() - 127)
    s = torch.where(q["scales"] == 255, torch.full_like(s, float("nan")), s)
    return (v.view(rows, -1, 32) * s[..., None]).view(rows, -1)[:, :q["cols"]]


def _plain(st):
    case = st["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op == "roundtrip":
        return _unpack(_pack(st["x"])).to(dt)
    if op == "readback":
        return _unpack(st["q"]).to(dt)
    w = _unpack(st["w"])
    if op == "matmul":
        return (_unpack(st["x"]) @ w.T).to(dt)
    x = st["x"].float()
    v, e, bad = _quantise(x)
    s = torch.where(bad, torch.full_like(e, 0).float() + float("nan"), torch.exp2(e.float()))
    y = (v * s[..., None]).view(x.shape[0], -1)[:, :x.shape[1]] @ w.T
    # every adapter's term for every token, the token's own kept
    S, R = case["slots"], case["r_max"]
    t = (x @ st["A"].float().view(S * R, -1).T).view(-1, S, R) * st["scale"][None, :, None]
    mine = st["idx"][:, None] == torch.arange(S, device=x.device)[None, :]
    t = torch.where(mine[..., None], t, torch.zeros_like(t)).view(-1, S * R)
    y += t @ st["B"].float().permute(0, 2, 1).reshape(S * R, -1)
    return y.to(dt)


# ---- the definition in 64 bits ----------------------------------------------------------------

def _values64(x):
    """What the stored form of x stands for, by the definition: in each block of 32 the scale is
    2 to the power floor(log2 max|x|) - 2 (no less than 2^-127), and every element becomes the
    nearest of the sixteen values times the scale; of two equally near the one with the even code."""
    rows, cols = x.shape
    x = x.double()
    out = torch.empty_like(x)
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    for c0 in range(0, cols, 4096):
        part = x[:, c0:c0 + 4096]
        pad = (-part.shape[1]) % 32
        b = torch.nn.functional.pad(part, (0, pad)).reshape(rows, -1, 32)
        top = b.abs().amax(-1, keepdim=True)
        # floor(log2 top), put right where log2 rounds across a whole number
        ex = torch.floor(torch.log2(top))
        ex = torch.where(torch.exp2(ex) > top, ex - 1, ex)
        ex = torch.where(torch.exp2(ex + 1) <= top, ex + 1, ex)
        scale = torch.exp2(torch.clamp(ex - 2, min=-127.0))
        ratio = b.abs() / scale
        near = torch.zeros_like(ratio)
        for k in range(1, 8):
            mid = (mags[k - 1] + mags[k]) / 2
            up = ratio >= mid if k % 2 == 0 else ratio > mid
            near = torch.where(up, torch.full_like(near, mags[k]), near)
        val = torch.sign(b) * near * scale
        val = torch.where(torch.isfinite(b).all(-1, keepdim=True), val, torch.full_like(val, float("nan")))
        out[:, c0:c0 + 4096] = val.reshape(rows, -1)[:, :part.shape[1]]
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "roundtrip":
        return _values64(d["x"])
    if op == "readback":
        return _values64(d["src"])
    x64 = d["x"].double()
    y = _values64(d["x"]) @ _values64(d["w"]).T
    if op == "linear":
        for s, r in enumerate(d["ranks"]):
            mine = torch.nonzero(d["idx"] == s).flatten()
            if mine.numel():
                low = x64[mine] @ d["A"][s, :r].double().T
                y[mine] += (d["alphas"][s] / r) * (low @ d["B"][s, :, :r].double().T)
    return y
