"""A decoder layer's projections over 4-bit base weights, with 16-bit adapters.

Quantises the base weights of a 7B-shaped layer once, mounts rank-8 adapters, and runs the layer's
seven LoRA-augmented linears for a decode batch and a prefill batch: one segment table a batch, and x
stored in 4 bits once for the projections that read it (q, k and v; gate and up).  Prints each
projection's distance from the 16-bit base's output, the bytes of the weights, and the time of a layer
either way.

    python examples/fp4_layer.py [--tokens 64] [--prefill 4096] [--adapters 100]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import adapter_gemm_segment_gb300 as ags  # noqa: E402

H, FF = 4096, 11008
PROJS = (("q_proj", H, H, "attn"), ("k_proj", H, H, "attn"), ("v_proj", H, H, "attn"), ("o_proj", H, H, "o"),
         ("gate_proj", H, FF, "mlp"), ("up_proj", H, FF, "mlp"), ("down_proj", FF, H, "down"))


class Projection:
    """One linear: the 16-bit base (kept for comparison), its 4-bit form and its adapter pool."""

    def __init__(self, h_in, h_out, n_adapters, rank, gen, dtype):
        self.W = (torch.randn(h_out, h_in, generator=gen, device="cuda") * 0.02).to(dtype)
        self.w4 = ags.lora_fp4_quantize(self.W, ags.Fp4Matrix(h_out, h_in))
        self.pool = ags.LoraPool(h_in, h_out, rank, n_adapters, dtype)
        bound = h_in ** -0.5
        A = [((torch.rand(rank, h_in, generator=gen, device="cuda") * 2 - 1) * bound).to(dtype) for _ in range(n_adapters)]
        B = [(torch.randn(h_out, rank, generator=gen, device="cuda") * 0.01).to(dtype) for _ in range(n_adapters)]
        self.pool.load_slots(range(n_adapters), A, B, [2.0 * rank] * n_adapters)
        torch.cuda.synchronize()  # the mount has read A and B


def run_layer(layer, xs, seg, out, four_bit, stored):
    """Every projection of the layer into out[name]; stored[feed]: room for x's 4-bit form."""
    made = set()
    for name, _, _, feed in PROJS:
        p = layer[name]
        if not four_bit:
            p.pool.linear(p.W, xs[feed], seg, y=out[name])
            continue
        if feed not in made:
            ags.lora_fp4_quantize(xs[feed], stored[feed])
            made.add(feed)
        p.pool.fp4_linear(p.w4, xs[feed], seg, xq=stored[feed], y=out[name])


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
    args = ap.parse_args()
    dtype = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer = {name: Projection(h_in, h_out, args.adapters, 8, gen, dtype) for name, h_in, h_out, _ in PROJS}
    full = sum(p.W.numel() * 2 for p in layer.values())
    small = sum(p.w4.nbytes for p in layer.values())
    print(f"base weights: {full / 1e6:.0f} MB in bf16, {small / 1e6:.0f} MB in 4 bits")

    # a stored weight reads back as what the products use: the nearest values, 4.25 bits each
    W = layer["q_proj"].W
    back = ags.lora_fp4_dequantize(layer["q_proj"].w4, torch.empty_like(W))
    print(f"q_proj read back: relative error {((back - W).float().norm() / W.float().norm()).item():.3f}")

    for label, n, run in (("decode", args.tokens, 1), ("prefill", args.prefill, 512)):
        idx = torch.randint(-1, args.adapters, ((n + run - 1) // run,), generator=gen, device="cuda")
        idx = idx.repeat_interleave(run)[:n].to(torch.int32)
        xs = {f: torch.randn(n, h_in, generator=gen, device="cuda").to(dtype) for _, h_in, _, f in PROJS}
        stored = {f: ags.Fp4Matrix(n, x.shape[1]) for f, x in xs.items()}
        seg = layer["q_proj"].pool.segment(idx)  # once a batch, for every projection
        out = {four: {name: torch.empty(n, h_out, dtype=dtype, device="cuda") for name, _, h_out, _ in PROJS}
               for four in (False, True)}
        times = {four: timed(lambda f=four: run_layer(layer, xs, seg, out[f], f, stored)) for four in (False, True)}
        if ags.lora_segment_status(seg) != ags.LORA_OK:
            raise RuntimeError("the batch was refused")
        print(f"{label}, {n} tokens: {times[False]:.0f} us a layer over bf16 bases, {times[True]:.0f} us over 4 bits")
        for name in layer:
            a, b = out[False][name].float(), out[True][name].float()
            print(f"  {name:10s} relative difference {((a - b).norm() / a.norm()).item():.3f}")


if __name__ == "__main__":
    main()
