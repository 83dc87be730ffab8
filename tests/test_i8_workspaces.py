"""The workspaces of 8-bit linears that are given none: one for each stream, shared by every pool, as calls on a stream run
one after the other.  Above 512 tokens it holds the weight in float16, several times what 8 bits save of one weight."""
import contextlib
import gc
import threading
import time
import weakref

import pytest
import torch

import adapter_gemm_segment_gb300 as ags
from adapter_gemm_segment_gb300 import workloads as wl


class Seg:
    def __init__(self, n):
        self.n_tokens = n


@pytest.fixture
def pools(monkeypatch):
    """Three pools whose device calls are replaced: every linear returns the workspace it was given."""
    monkeypatch.setattr(ags, "_on_stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(ags, "_capturing", lambda: False)
    monkeypatch.setattr(ags, "lora_i8_linear_workspace_bytes", lambda handle, n: 1000 * n * handle)
    monkeypatch.setattr(ags, "lora_i8_linear_fwd", lambda handle, w, x, y, seg, ws, xq=None, stream=None: ws)
    monkeypatch.setattr(ags.LoraPool, "close", lambda self: None)
    made = []
    for size in (1, 2, 3):
        p = ags.LoraPool.__new__(ags.LoraPool)
        p.h_in, p.h_out, p.dtype, p.handle, p._ws = 32, 32, torch.float32, size, {}
        made.append(p)
    del p
    yield made
    made.clear()
    gc.collect()


def call(pool, n, stream=64):
    return pool.i8_linear(None, torch.zeros(n, 32), Seg(n), y=torch.zeros(n, 32), stream=stream)


def test_pools_share_one_on_a_stream(pools):
    a, b, c = pools
    first = call(c, 100)
    assert first.numel() >= 300000
    for pool, n in ((a, 100), (b, 100), (b, 150), (c, 7), (c, 100), (a, 300)):
        assert call(pool, n).data_ptr() == first.data_ptr()
    # the largest need is everyone's from then on
    second = call(b, 151)
    assert second.numel() >= 302000
    for pool, n in ((a, 1), (b, 151), (c, 100)):
        assert call(pool, n).data_ptr() == second.data_ptr()


def test_streams_have_their_own(pools):
    a, b, _ = pools
    assert call(a, 10, 64).data_ptr() != call(a, 10, 128).data_ptr()
    assert call(a, 10, 128).data_ptr() == call(b, 5, 128).data_ptr()


def test_a_captured_call_has_its_own(pools, monkeypatch):
    eager = call(pools[0], 8)
    monkeypatch.setattr(ags, "_capturing", lambda: True)
    one, two = call(pools[0], 8), call(pools[1], 8)
    assert len({eager.data_ptr(), one.data_ptr(), two.data_ptr()}) == 3
    assert one.numel() >= 8000 and two.numel() >= 16000


def test_the_memory_goes_with_the_last_pool(pools, monkeypatch):
    made = []
    empty = torch.empty

    def counted(*args, **kw):
        t = empty(*args, **kw)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", counted)
    for p in pools:
        call(p, 10)
    assert made and made[-1]() is not None
    del p
    while pools:
        assert made[-1]() is not None
        pools.pop()
        gc.collect()
    assert all(ref() is None for ref in made)


def test_a_need_that_could_not_be_met_is_asked_for_again(pools, monkeypatch):
    """Out of memory while it grows: the call fails, and the next one starts over."""
    small = call(pools[0], 10)
    empty = torch.empty
    del small

    def full(*args, **kw):
        raise RuntimeError("out of memory")

    monkeypatch.setattr(torch, "empty", full)
    with pytest.raises(RuntimeError):
        call(pools[1], 1000)
    monkeypatch.setattr(torch, "empty", empty)
    assert call(pools[0], 10).numel() >= 10000
    assert call(pools[1], 1000).numel() >= 2000000


def test_memory_is_allocated_on_the_stream_of_the_call(pools, monkeypatch):
    on = []

    @contextlib.contextmanager
    def on_stream(stream):
        on.append(stream)
        yield

    monkeypatch.setattr(ags, "_on_stream", on_stream)
    pools[0].i8_linear(None, torch.zeros(4, 32), Seg(4), stream=64)
    assert on and set(on) == {64}


def test_threads_take_turns_on_a_stream(pools, monkeypatch):
    """A linear is several launches: those of two threads may not mix where they share a workspace."""
    inside, worst = {}, {}
    guard = threading.Lock()

    def slow(handle, w, x, y, seg, ws, xq=None, stream=None):
        with guard:
            inside[stream] = inside.get(stream, 0) + 1
            worst[stream] = max(worst.get(stream, 0), inside[stream])
        time.sleep(0.01)
        with guard:
            inside[stream] -= 1
        return ws

    monkeypatch.setattr(ags, "lora_i8_linear_fwd", slow)
    threads = [threading.Thread(target=lambda p=p, s=s: [call(p, 10, s) for _ in range(5)]) for p in pools for s in (64, 128)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert worst == {64: 1, 128: 1}


# ---- on the GPU -------------------------------------------------------------------------------------

def layer(lib, shapes, slots, n, seed):
    """Pools, stored weights, x and references (each call by itself, with a workspace of its own)."""
    made = []
    for i, (h_in, h_out) in enumerate(shapes):
        case = wl.random_case(seed + i, n, h_in, h_out, [8] * slots, r_max=8, dtype=torch.bfloat16, p_base=0.1)
        pool = lib.LoraPool(h_in, h_out, 8, slots, torch.bfloat16, "cuda")
        for s in range(slots):
            pool.load_slot(s, case.adapters.A[s].cuda(), case.adapters.B[s].cuda(), case.adapters.alphas[s])
        w, x = lib.lora_i8_quantize(case.W.cuda(), lib.I8Matrix(h_out, h_in)), case.x.cuda()
        seg = pool.segment(case.idx.cuda())
        torch.cuda.synchronize()
        want = pool.i8_linear(w, x, seg, ws=pool.i8_linear_workspace(n))
        torch.cuda.synchronize()
        made.append((pool, w, x, seg, want))
    return made


SHAPES = [(512, 512), (512, 264), (1096, 520), (512, 1096), (264, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,slots", [(3, 4), (8, 4), (40, 60), (300, 4), (700, 4), (700, 100), (2100, 4)])
def test_pools_back_to_back(lib, n, slots):
    """Calls of other shapes follow at once in the same workspace, where kernels start before those ahead have ended."""
    made = layer(lib, SHAPES, slots, n, 5)
    for _ in range(5):
        got = [pool.i8_linear(w, x, seg) for pool, w, x, seg, _ in made for _ in range(2)]
        torch.cuda.synchronize()
        for y, want in zip(got, [m[4] for m in made for _ in range(2)]):
            assert torch.equal(y, want)
    for pool, *_ in made:
        pool.close()


@pytest.mark.gpu
def test_two_threads_on_one_stream(lib):
    made = layer(lib, SHAPES, 4, 700, 9)
    bad = []

    def work(part):
        for _ in range(30):
            for pool, w, x, seg, want in part:
                y = pool.i8_linear(w, x, seg)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want):
                    bad.append(pool)

    threads = [threading.Thread(target=work, args=(made[i::2],)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    for pool, *_ in made:
        pool.close()


@pytest.mark.gpu
def test_a_prefill_leaves_less_than_the_16_bit_weights_would(lib):
    """Seven pools, as a layer's projections: what the calls keep is one workspace, the largest, and with the stored
    weights it is less than the weights in 16 bits."""
    n, shapes = 700, [(2048, 2048)] * 4 + [(2048, 5504)] * 2 + [(5504, 2048)]
    made = layer(lib, shapes, 4, n, 3)
    most = max(lib.lora_i8_linear_workspace_bytes(pool.handle, n) for pool, *_ in made)
    ys = [torch.empty_like(m[4]) for m in made]
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()
    for (pool, w, x, seg, _), y in zip(made, ys):
        pool.i8_linear(w, x, seg, y=y)
    torch.cuda.synchronize()
    kept = torch.cuda.memory_allocated() - before
    assert kept <= most + 512
    stored, full = sum(m[1].nbytes for m in made), sum(2 * h_in * h_out for h_in, h_out in shapes)
    assert stored + kept < full
    for (pool, *_, want), y in zip(made, ys):
        assert torch.equal(y, want)
        pool.close()
    made.clear()
    del pool
    gc.collect()
    assert torch.cuda.memory_allocated() < before
