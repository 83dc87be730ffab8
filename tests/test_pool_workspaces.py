"""The workspaces that LoraPool keeps for calls that are given none: one for each stream."""
import contextlib

import numpy as np
import pytest
import torch

import adapter_gemm_segment_gb300 as ags
from adapter_gemm_segment_gb300 import workloads as wl


class Seg:
    def __init__(self, n):
        self.n_tokens = n


@pytest.fixture
def pool(monkeypatch):
    """A pool whose device calls are replaced: every linear records the workspace it was given."""
    monkeypatch.setattr(ags, "_on_stream", lambda stream: contextlib.nullcontext(), raising=False)
    monkeypatch.setattr(ags, "_capturing", lambda: False, raising=False)
    monkeypatch.setattr(ags, "_device_bytes", lambda nbytes, device: torch.zeros(nbytes, dtype=torch.uint8))
    monkeypatch.setattr(ags, "lora_fp4_linear_workspace_bytes", lambda handle, n: 1000 * n)
    monkeypatch.setattr(ags, "lora_linear_workspace_bytes", lambda handle, n: 3000 if n < 10 else 200 * n)
    monkeypatch.setattr(ags, "lora_fp4_linear_fwd", lambda handle, w, x, y, seg, ws, xq=None, stream=None: ws)
    monkeypatch.setattr(ags, "lora_linear_fwd", lambda handle, W, x, y, seg, ws, variant=0, stream=None: ws)
    p = ags.LoraPool.__new__(ags.LoraPool)
    p.h_in, p.h_out, p.dtype, p.handle, p._ws = 32, 32, torch.float32, None, {}
    return p


def calls(pool):
    def fp4(n, stream):
        return pool.fp4_linear(None, torch.zeros(n, 32), Seg(n), y=torch.zeros(n, 32), stream=stream)

    def linear(n, stream):
        return pool.linear(None, torch.zeros(n, 32), Seg(n), y=torch.zeros(n, 32), stream=stream)

    return fp4, linear


def test_streams_do_not_share_a_workspace(pool):
    for call in calls(pool):
        a, b = call(16, 64), call(16, 128)
        assert a.data_ptr() != b.data_ptr()
        assert call(16, 64).data_ptr() == a.data_ptr() and call(16, 128).data_ptr() == b.data_ptr()


def test_the_four_bit_linear_keeps_the_largest_alone(pool):
    fp4, _ = calls(pool)
    for n in (5, 100, 7, 100, 60):
        assert fp4(n, 64).numel() >= 1000 * n
    assert len(pool._ws) == 1
    assert fp4(3, 64).numel() == 100000


def test_the_linear_has_enough_for_fewer_tokens(pool):
    _, linear = calls(pool)
    assert linear(12, 64).numel() >= 2400 and linear(3, 64).numel() >= 3000


def test_a_captured_call_keeps_its_own(pool, monkeypatch):
    fp4, _ = calls(pool)
    eager = fp4(8, 64)
    monkeypatch.setattr(ags, "_capturing", lambda: True, raising=False)
    assert fp4(8, 64).data_ptr() != eager.data_ptr()


def test_memory_is_allocated_on_the_stream_of_the_call(pool, monkeypatch):
    """Both y and the workspace: memory of another stream may still be in use there."""
    on = []

    @contextlib.contextmanager
    def on_stream(stream):
        on.append(stream)
        yield

    monkeypatch.setattr(ags, "_on_stream", on_stream, raising=False)
    pool.fp4_linear(None, torch.zeros(4, 32), Seg(4), stream=64)
    pool.linear(None, torch.zeros(4, 32), Seg(4), stream=64)
    assert on == [64] * 4


@pytest.mark.gpu
@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("four_bit", [True, False])
def test_two_streams_at_once(lib, n, four_bit):
    """The same n on two streams with different x, and a captured call replayed beside them."""
    case = wl.random_case(91, n, 4096, 4096, [16] * 4, r_max=16, dtype=torch.bfloat16, p_base=0.1)
    pool = lib.LoraPool(4096, 4096, 16, 4, torch.bfloat16, "cuda")
    for s in range(4):
        pool.load_slot(s, case.adapters.A[s].cuda(), case.adapters.B[s].cuda(), case.adapters.alphas[s])
    W = case.W.cuda()
    w = lib.lora_fp4_quantize(W, lib.Fp4Matrix(4096, 4096))
    xs = [case.x.cuda(), -case.x.flip(0).cuda(), 2 * case.x.roll(1, 0).cuda()]
    idx = case.idx.cuda()

    def call(x, seg, y=None, stream=None):
        if four_bit:
            return pool.fp4_linear(w, x, seg, y=y, stream=stream)
        return pool.linear(W, x, seg, y=y, stream=stream)

    segs = [pool.segment(idx) for _ in xs]  # a table each: the calls of one table run on one stream
    want = []
    for x, seg in zip(xs, segs):
        want.append(call(x, seg).clone())
        torch.cuda.synchronize()
    graph, captured = torch.cuda.CUDAGraph(), torch.empty_like(want[2])
    with torch.cuda.graph(graph):
        call(xs[2], segs[2], captured)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[torch.empty_like(want[0]) for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for j in range(2):
            if i % 2:
                call(xs[j], segs[j], got[j][i], stream=streams[j])
            else:
                with torch.cuda.stream(streams[j]):
                    call(xs[j], segs[j], got[j][i])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for j in range(2):
        for y in got[j]:
            assert torch.equal(y, want[j])
    assert torch.equal(captured, want[2])
    assert np.isfinite(captured.float().cpu().numpy()).all()
    pool.close()
