"""The front half of a decoder layer over 8-bit base weights, with 16-bit adapters.

Quantises the base weights of a 7B-shaped layer once, mounts rank-8 adapters, and runs the residual addition and
norm before the q, k and v projections and before the gate and up projections: the norm stores its output in 8
bits beside the 16-bit one, the projections that read it share it, and one segment table serves the batch.
Prints each projection's distance from the 16-bit base's output, the bytes of the weights, and the time of the
run either way.

    python examples/i8_layer.py [--tokens 64] [--prefill 4096] [--adapters 100] [--hidden 4096] [--ff 11008]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import adapter_gemm_segment_gb300 as ags  # noqa: E402

EPS = 1e-5
NORMS = (("attn", ("q_proj", "k_proj", "v_proj")), ("mlp", ("gate_proj", "up_proj")))


class Projection:
    """One linear: the 16-bit base (kept for comparison), its 8-bit form and its adapter pool."""

    def __init__(self, h_in, h_out, n_adapters, rank, gen, dtype):
        self.W = (torch.randn(h_out, h_in, generator=gen, device="cuda") * 0.02).to(dtype)
        self.w8 = ags.lora_i8_quantize(self.W, ags.I8Matrix(h_out, h_in))
        self.pool = ags.LoraPool(h_in, h_out, rank, n_adapters, dtype)
        bound = h_in ** -0.5
        A = [((torch.rand(rank, h_in, generator=gen, device="cuda") * 2 - 1) * bound).to(dtype) for _ in range(n_adapters)]
        B = [(torch.randn(h_out, rank, generator=gen, device="cuda") * 0.01).to(dtype) for _ in range(n_adapters)]
        self.pool.load_slots(range(n_adapters), A, B, [2.0 * rank] * n_adapters)
        torch.cuda.synchronize()  # the mount has read A and B


def run(layer, gains, xs, seg, out, eight_bit, hidden, normed, stored):
    """The norms and projections into out[name]; hidden, normed, stored: room for the norms' outputs."""
    for feed, names in NORMS:
        ags.lora_i8_rmsnorm(xs[feed], gains[feed], EPS, out=stored if eight_bit else None, y=normed,
                            residual=xs["residual"], residual_out=hidden)
        for name in names:
            p = layer[name]
            if eight_bit:
                p.pool.i8_linear(p.w8, normed, seg, xq=stored, y=out[name])
            else:
                p.pool.linear(p.W, normed, seg, y=out[name])


def timed(fn, n=20):
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--prefill", type=int, default=4096)
    ap.add_argument("--adapters", type=int, default=100)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ff", type=int, default=11008)
    args = ap.parse_args()
    dtype, H = torch.bfloat16, args.hidden
    gen = torch.Generator(device="cuda").manual_seed(0)
    widths = {"attn": H, "mlp": args.ff}
    layer = {name: Projection(H, widths[feed], args.adapters, 8, gen, dtype) for feed, names in NORMS for name in names}
    gains = {feed: (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype) for feed, _ in NORMS}
    full = sum(p.W.numel() * 2 for p in layer.values())
    small = sum(p.w8.nbytes for p in layer.values())
    print(f"base weights: {full / 1e6:.1f} MB in bf16, {small / 1e6:.1f} MB in 8 bits")

    for label, n, length in (("decode", args.tokens, 1), ("prefill", args.prefill, 512)):
        idx = torch.randint(-1, args.adapters, ((n + length - 1) // length,), generator=gen, device="cuda")
        idx = idx.repeat_interleave(length)[:n].to(torch.int32)
        xs = {f: torch.randn(n, H, generator=gen, device="cuda").to(dtype) for f in ("attn", "mlp", "residual")}
        hidden, normed, stored = torch.empty_like(xs["attn"]), torch.empty_like(xs["attn"]), ags.I8Matrix(n, H)
        seg = layer["q_proj"].pool.segment(idx)  # once a batch, for every projection
        out = {b: {name: torch.empty(n, p.W.shape[0], dtype=dtype, device="cuda") for name, p in layer.items()}
               for b in (False, True)}
        times = {b: timed(lambda b=b: run(layer, gains, xs, seg, out[b], b, hidden, normed, stored)) for b in (False, True)}
        if ags.lora_segment_status(seg) != ags.LORA_OK:
            raise RuntimeError("the batch was refused")
        print(f"{label}, {n} tokens: {times[False]:.0f} us over bf16 bases, {times[True]:.0f} us over 8 bits")
        # one serves every projection: the calls of a stream run one after the other
        room = max(ags.lora_i8_linear_workspace_bytes(p.pool.handle, n) for p in layer.values())
        print(f"  workspace of the 8-bit projections together: {room / 1e6:.1f} MB")
        for name in layer:
            a, b = out[False][name].float(), out[True][name].float()
            print(f"  {name:10s} relative difference {((a - b).norm() / a.norm()).item():.4f}")


if __name__ == "__main__":
    main()
