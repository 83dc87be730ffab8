"""What the Python entry point of the linear over a 4-bit base refuses before the library, which sees bare
pointers, could read or write past a tensor."""
import ctypes

import pytest
import torch

import adapter_gemm_segment_gb300 as ags


class Weight:
    rows, cols = 64, 256
    struct = ags.lora_fp4_matrix()


@pytest.fixture
def call(monkeypatch):
    """lora_fp4_linear_fwd of 20 tokens on host tensors; returns whether the library was called."""
    reached = []

    class Library:
        def lora_fp4_linear_fwd(self, *args):
            reached.append(args)
            return ags.LORA_OK

    monkeypatch.setattr(ags, "_lib", Library())
    monkeypatch.setattr(ags, "_dev", lambda t, name: t)
    monkeypatch.setattr(ags, "_stream", lambda stream: ctypes.c_void_p(0))
    handle = ctypes.c_void_p(1)
    handle.dtype = torch.float16
    seg = ags.lora_segments()
    seg.n_tokens = 20

    def run(x, y):
        ags.lora_fp4_linear_fwd(handle, Weight, x, y, seg, torch.zeros(1024, dtype=torch.uint8))
        return len(reached) == 1

    run.reached = reached
    return run


def half(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def test_matching_tensors_reach_the_library(call):
    assert call(half(20, 256), half(20, 64))


def test_leading_dimensions_are_rows(call):
    assert call(half(4, 5, 256), half(20, 1, 64))


@pytest.mark.parametrize("x,y", [
    (half(19, 256), half(20, 64)), (half(21, 256), half(20, 64)), (half(20, 248), half(20, 64)), (half(20 * 256), half(20, 64)),
    (half(20, 256), half(19, 64)), (half(20, 256), half(20, 56)), (half(20, 256), half(40, 32)),
    (half(20, 256).bfloat16(), half(20, 64)), (half(20, 256), half(20, 64).float()), (half(20, 256).float(), half(20, 64).float()),
    (half(20, 256).bfloat16(), half(20, 64).bfloat16())])
def test_other_shapes_and_types_are_refused(call, x, y):
    with pytest.raises(ags.LoraError) as e:
        call(x, y)
    assert e.value.code == ags.LORA_EINVAL and not call.reached


@pytest.mark.parametrize("device", ["cpu", "meta", torch.device("cpu")])
def test_a_matrix_off_the_gpu_is_refused(device):
    with pytest.raises(ValueError):
        ags.Fp4Matrix(64, 256, device)


@pytest.mark.gpu
def test_refusals_through_a_pool(lib):
    pool = lib.LoraPool(256, 64, 8, 1, torch.float16, "cuda")
    w = lib.lora_fp4_quantize(torch.zeros(64, 256, device="cuda"), lib.Fp4Matrix(64, 256))
    seg = pool.segment(torch.full((20,), -1, dtype=torch.int32, device="cuda"))
    x = half(20, 256).cuda()
    assert pool.fp4_linear(w, x, seg).shape == (20, 64)
    for bad in (x[:19], x.float(), x.bfloat16(), x.view(-1), x[:, :128].contiguous()):
        with pytest.raises(lib.LoraError) as e:
            pool.fp4_linear(w, bad, seg)
        assert e.value.code == lib.LORA_EINVAL
    for bad in (half(20, 56).cuda(), half(19, 64).cuda(), half(20, 64).cuda().float()):
        with pytest.raises(lib.LoraError) as e:
            pool.fp4_linear(w, x, seg, y=bad)
        assert e.value.code == lib.LORA_EINVAL
    pool.close()


@pytest.mark.gpu
def test_pools_past_32_bit_box_coordinates(lib):
    """2048 slots x 2^20 features are 2^31 rows of B (34 GB): small batches, whose kernel addresses them in
    boxes with 32-bit coordinates, are refused; larger ones read the last slot."""
    h_out = 1 << 20
    pool = lib.LoraPool(64, h_out, 8, 2048, torch.float16, "cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randn(8, 64, generator=gen, device="cuda").half()
    B = torch.randn(h_out, 8, generator=gen, device="cuda").half()
    pool.load_slot(2047, A, B, 8.0)
    w = lib.lora_fp4_quantize(torch.zeros(h_out, 64, device="cuda"), lib.Fp4Matrix(h_out, 64))
    x = torch.randn(300, 64, generator=gen, device="cuda").half()
    idx = torch.full((300,), 2047, dtype=torch.int32, device="cuda")
    with pytest.raises(lib.LoraError) as e:
        pool.fp4_linear(w, x[:20], pool.segment(idx[:20]))
    assert e.value.code == lib.LORA_EUNSUP
    y = pool.fp4_linear(w, x, pool.segment(idx))
    ref = (x[-2:].double() @ A.double().T) @ B.double().T
    assert (y[-2:].double() - ref).abs().max() <= 2e-3 * ref.abs().max()
    pool.close()
