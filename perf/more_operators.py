"""Cases of the 8-bit integer operators: what is timed and against which plain form.

A frozen base weight held in 8-bit integers with one scale a row (an output channel), under
activations held the same way (one scale a token), takes half the bytes of a 16-bit one and keeps
every product and sum exact.  A row x is stored as codes c and a float32 scale s: s = max|x| / 127
rounded to float32, c the whole number nearest x / s (ties to the even one), at most 127 either way.

  roundtrip   quantise rows, then read them back (both calls of one pass)
  norm        residual addition, root-mean-square norm and its output in 8 bits, read back:
              h = x + residual; y = h / sqrt(mean h^2 + eps) * weight; y stored as above
  matmul      y = sx sw (Cx Cw^T) of two stored 8-bit matrices
  linear      y = Q(x) Wq^T + (alpha/r) (x A_s^T) B_s^T: the LoRA-augmented linear over an 8-bit
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
EPS = 1e-5


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # a column window of a wider float32 buffer: odd width, odd row count
        dict(name="roundtrip_window", op="roundtrip", rows=257, cols=1009, ld=1040, dtype="f32"),
        # the up projection's weight: quantised once when a model is loaded, read back to merge an adapter
        dict(name="roundtrip_weight", op="roundtrip", rows=11008, cols=4096, ld=4096, dtype="bf16"),
        # one decode token ahead of a layer's projections: latency is all that counts
        dict(name="norm_token", op="norm", rows=1, cols=4096, residual=True, dtype="f16"),
        # the first norm of a model (no residual yet) at an odd width in float32
        dict(name="norm_odd", op="norm", rows=333, cols=2731, residual=False, dtype="f32"),
        # the tokens of a prefill batch (32 requests of 512)
        dict(name="norm_prefill", op="norm", rows=16384, cols=4096, residual=True, dtype="bf16"),
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
    op = rng.choice(["roundtrip", "norm", "norm", "matmul", "matmul", "linear", "linear", "linear"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("roundtrip", "norm"):
        cols = _log(rng, 1, 11008)
        rows = _log(rng, 1, max(1, min(16384, 16384 * 4096 // cols)))
        if op == "norm":
            return dict(op=op, rows=rows, cols=cols, residual=rng.choice([True, False]), dtype=dtype)
        return dict(op=op, rows=rows, cols=cols, ld=cols + rng.choice([0, 0, 1, 8, 24, 100]), dtype=dtype)
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
    """Bytes of a stored matrix: one an element and a float32 scale a row."""
    return rows * (cols + 4)


def work(case):
    es = ES[case["dtype"]]
    if case["op"] in ("roundtrip", "norm"):
        r, c = case["rows"], case["cols"]
        # the stored form out and in again, the values out
        back = 2 * _stored(r, c) + r * c * es
        if case["op"] == "roundtrip":
            return {"bytes": r * c * es + back, "flops": 4 * r * c}
        # x in and y out, the residual in and out, the weight
        streams = 4 if case["residual"] else 2
        return {"bytes": streams * r * c * es + c * es + back, "flops": 9 * r * c}
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
    """Normal activations with a few loud channels and a few silent tokens."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    x *= torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.002, 0.0, 1.0)
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
    """Stacked adapters [slots, r_max, .] (rows past an adapter's rank are zero) and their alphas."""
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
    if op in ("roundtrip", "norm"):
        g = _gen(seed, case["rows"], case["cols"])
        if op == "roundtrip":
            return {"x": _activations(g, case["rows"], case["ld"], case["dtype"])[:, :case["cols"]]}
        d = {"x": _activations(g, case["rows"], case["cols"], case["dtype"]), "residual": None}
        if case["residual"]:
            d["residual"] = (torch.randn(case["rows"], case["cols"], generator=g, device="cuda") * 3).to(DT[case["dtype"]])
        d["weight"] = (1 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(DT[case["dtype"]])
        return d
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
    if op in ("roundtrip", "norm"):
        st.update(d)
    elif op == "linear":
        st["x"], st["idx"] = d["x"], d["idx"]
    if not own:
        if op in ("matmul", "linear"):
            st["w"] = _pack(d["w"].float())
        if op == "matmul":
            st["x"] = _pack(d["x"].float())
        if op == "linear":
            st["A"], st["B"] = d["A"], d["B"]
            st["scale"] = torch.tensor([a / r for a, r in zip(d["alphas"], d["ranks"])], device="cuda")
        return st

    import adapter_gemm_segment_gb300 as ags

    st["ags"] = ags
    dt = DT[case["dtype"]]
    if op in ("roundtrip", "norm"):
        st["q"] = ags.I8Matrix(case["rows"], case["cols"], "cuda")
        st["out"] = torch.empty(case["rows"], case["cols"], dtype=dt, device="cuda")
        if op == "norm":
            st["y"] = torch.empty_like(st["out"])
            st["sum"] = torch.empty_like(st["out"]) if case["residual"] else None
    else:
        n, hi, ho = case["n"], case["h_in"], case["h_out"]
        st["w"] = ags.lora_i8_quantize(d["w"], ags.I8Matrix(ho, hi, "cuda"))
        st["y"] = torch.empty(n, ho, dtype=dt, device="cuda")
        if op == "matmul":
            st["x"] = ags.lora_i8_quantize(d["x"], ags.I8Matrix(n, hi, "cuda"))
            st["ws"] = torch.empty(max(256, ags.lora_i8_matmul_workspace_bytes(n, ho, hi)), dtype=torch.uint8, device="cuda")
        else:
            pool = ags.LoraPool(hi, ho, case["r_max"], case["slots"], dt, "cuda")
            pool.load_slots(range(case["slots"]), [d["A"][s, :r].contiguous() for s, r in enumerate(d["ranks"])],
                            [d["B"][s, :, :r].contiguous() for s, r in enumerate(d["ranks"])], d["alphas"])
            st["pool"] = pool
            # the segments of a batch: built once, shared by every linear the batch runs through
            st["seg"] = pool.segment(d["idx"])
            st["ws"] = pool.i8_linear_workspace(n)
    return st


def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    ags, op = st["ags"], st["case"]["op"]
    if op == "roundtrip":
        ags.lora_i8_quantize(st["x"], st["q"])
        return ags.lora_i8_dequantize(st["q"], st["out"])
    if op == "norm":
        ags.lora_i8_rmsnorm(st["x"], st["weight"], EPS, out=st["q"], y=st["y"], residual=st["residual"],
                            residual_out=st["sum"])
        values = ags.lora_i8_dequantize(st["q"], st["out"])
        return (st["y"], values) if st["sum"] is None else (st["y"], values, st["sum"])
    if op == "matmul":
        return ags.lora_i8_matmul(st["x"], st["w"], st["y"], st["ws"])
    return ags.lora_i8_linear_fwd(st["pool"].handle, st["w"], st["x"], st["y"], st["seg"], st["ws"])


# ---- the plain form -------------------------------------------------------------------------

def _codes(v):
    """float64 rows -> (codes int8, scales float32).  In 64 bits: a value next to the border of two
    codes has to fall on its own side."""
    scale = (v.abs().amax(1, keepdim=True) / 127).float()
    bad = ~torch.isfinite(scale)
    c = torch.round(v / scale.double()).clamp(-127, 127)
    c = torch.where(bad | (scale == 0), torch.zeros_like(c), c)
    return c.to(torch.int8), torch.where(bad, torch.full_like(scale, float("nan")), scale)


def _pack(x):
    codes, scales = _codes(x.double())
    return {"codes": codes, "scales": scales}


def _unpack(q):
    return q["codes"].float() * q["scales"]


def _sums(x, w):
    """Cx Cw^T: whole numbers that float32 holds (these inputs' stay far below 2^24)."""
    return x["codes"].float() @ w["codes"].float().T


def _plain(st):
    case = st["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op == "roundtrip":
        return _unpack(_pack(st["x"])).to(dt)
    if op == "norm":
        h = st["x"]
        if st["residual"] is not None:
            h = (h.float() + st["residual"].float()).to(dt)
        d = h.double()
        d = d * torch.rsqrt(torch.mean(d * d, dim=1, keepdim=True) + EPS) * st["weight"].double()
        codes, scales = _codes(d)
        values = (codes.float() * scales).to(dt)
        return (d.to(dt), values) if st["residual"] is None else (d.to(dt), values, h)
    if op == "matmul":
        return (_sums(st["x"], st["w"]) * st["x"]["scales"] * st["w"]["scales"].T).to(dt)
    x = st["x"].float()
    q = _pack(x)
    y = _sums(q, st["w"]) * q["scales"] * st["w"]["scales"].T
    # every adapter's term for every token, the token's own kept
    S, R = case["slots"], case["r_max"]
    t = (x @ st["A"].float().view(S * R, -1).T).view(-1, S, R) * st["scale"][None, :, None]
    mine = st["idx"][:, None] == torch.arange(S, device=x.device)[None, :]
    t = torch.where(mine[..., None], t, torch.zeros_like(t)).view(-1, S * R)
    y += t @ st["B"].float().permute(0, 2, 1).reshape(S * R, -1)
    return y.to(dt)


# ---- the definition in 64 bits ----------------------------------------------------------------

def _values64(v):
    """What the stored form of the rows v (float64) stands for: the scale s is the float32 nearest
    max|v| / 127, and every element becomes the nearest of -127 s, .., 127 s, of two equally near
    ones the even multiple."""
    out = torch.empty_like(v)
    step = max(1, (1 << 25) // max(1, v.shape[1]))
    for r0 in range(0, v.shape[0], step):
        part = v[r0:r0 + step]
        s = (torch.maximum(part.amax(1), -part.amin(1)) / 127.0).to(torch.float32).to(torch.float64)[:, None]
        q = torch.where(s > 0, part.abs() / s, torch.zeros_like(part))
        low = torch.floor(q)
        over = q - low
        up = (over > 0.5) | ((over == 0.5) & (torch.remainder(low, 2) == 1))
        m = torch.clamp(low + up.to(low.dtype), max=127.0)
        val = torch.sign(part) * m * s
        ok = torch.isfinite(part).all(1, keepdim=True)
        out[r0:r0 + step] = torch.where(ok, val, torch.full_like(val, float("nan")))
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "roundtrip":
        return _values64(d["x"].double())
    if op == "norm":
        total = d["x"].double()
        if d["residual"] is not None:
            total = total + d["residual"].double()
        # the norm is of the sum as it is stored
        h = total.to(DT[case["dtype"]]).double()
        size = torch.sqrt(torch.sum(h.square(), dim=1, keepdim=True) / case["cols"] + EPS)
        y = h * d["weight"].double() / size
        return (y, _values64(y)) if d["residual"] is None else (y, _values64(y), total)
    x64 = d["x"].double()
    y = _values64(x64) @ _values64(d["w"].double()).T
    if op == "linear":
        for s, r in enumerate(d["ranks"]):
            mine = torch.nonzero(d["idx"] == s).flatten()
            if mine.numel():
                low = x64[mine] @ d["A"][s, :r].double().T
                y[mine] += (d["alphas"][s] / r) * (low @ d["B"][s, :, :r].double().T)
    return y
