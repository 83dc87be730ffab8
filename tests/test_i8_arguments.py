"""What the 8-bit entry points refuse, on the host, before anything is enqueued.  Addresses here are made up:
a call that is not refused would be a failure of the test."""
import ctypes

import pytest
import torch

import adapter_gemm_segment_gb300 as ags

P = 0x10000  # an aligned address no call may use


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def mat(rows, cols, codes=P, scales=P):
    return ags.lora_i8_matrix(codes, scales, rows, cols)


def refused(rc, code):
    assert rc == code, (rc, ags.lora_last_error())
    assert ags.lora_last_error()


def test_bytes():
    assert ags.lora_i8_bytes(3, 17) == (96, 12)
    assert ags.lora_i8_bytes(0, 1) == (0, 0)
    assert ags.lora_i8_bytes(2, 131071) == (2 * 131072, 8)
    assert ags.lora_i8_bytes(2 ** 31 - 256, 1) == (16 * (2 ** 31 - 256), 4 * (2 ** 31 - 256))
    for shape, code in (((-1, 4), ags.LORA_EINVAL), ((4, 0), ags.LORA_EINVAL), ((4, 131072), ags.LORA_EUNSUP),
                        ((2 ** 31 - 255, 1), ags.LORA_EUNSUP)):
        with pytest.raises(ags.LoraError) as e:
            ags.lora_i8_bytes(*shape)
        assert e.value.code == code


def test_quantize_and_read_back_refusals():
    lib = ags.load_library()
    for f in (lambda m, p, dt, ld: lib.lora_i8_quantize(p, dt, ld, ctypes.byref(m), None),
              lambda m, p, dt, ld: lib.lora_i8_dequantize(ctypes.byref(m), p, dt, ld, None)):
        refused(f(mat(4, 8), None, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8), P, 3, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8), P, 0, 7), ags.LORA_EINVAL)
        refused(f(mat(4, 8), P + 2, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8), P + 1, 1, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8, codes=0), P, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8, scales=0), P, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 8, codes=P + 16), P, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(-1, 8), P, 0, 8), ags.LORA_EINVAL)
        refused(f(mat(4, 131072), P, 0, 131072), ags.LORA_EUNSUP)
        assert f(mat(0, 8), P, 0, 8) == ags.LORA_OK
    refused(lib.lora_i8_quantize(P, 0, 8, None, None), ags.LORA_EINVAL)


def norm_args(**kw):
    out = mat(4, 8)
    a = ags.lora_i8_norm()
    a.x_dev = a.weight_dev = a.residual_dev = a.residual_out_dev = P
    a.y_dev = 2 * P
    a.ldx = a.ldr = a.ldro = a.ldy = 8
    a.rows, a.cols, a.dtype, a.eps = 4, 8, 0, 1e-5
    a.out = ctypes.pointer(out)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(x_dev=None), ags.LORA_EINVAL), (dict(weight_dev=None), ags.LORA_EINVAL), (dict(residual_out_dev=None), ags.LORA_EINVAL),
    (dict(y_dev=None, out=None), ags.LORA_EINVAL), (dict(ldx=7), ags.LORA_EINVAL), (dict(ldr=7), ags.LORA_EINVAL),
    (dict(ldro=7), ags.LORA_EINVAL), (dict(ldy=7), ags.LORA_EINVAL), (dict(dtype=5), ags.LORA_EINVAL),
    (dict(eps=0.0), ags.LORA_EINVAL), (dict(eps=float("nan")), ags.LORA_EINVAL), (dict(eps=2.0), ags.LORA_EINVAL),
    (dict(eps=-1e-5), ags.LORA_EINVAL), (dict(rows=-1), ags.LORA_EINVAL), (dict(cols=0), ags.LORA_EINVAL),
    (dict(rows=5), ags.LORA_EINVAL), (dict(cols=131072, ldx=131072), ags.LORA_EUNSUP), (dict(x_dev=P + 2), ags.LORA_EINVAL),
    (dict(weight_dev=P + 2), ags.LORA_EINVAL), (dict(y_dev=P + 1), ags.LORA_EINVAL), (dict(y_dev=P), ags.LORA_EINVAL)])
def test_norm_refusals(change, code):
    refused(ags.load_library().lora_i8_rmsnorm(ctypes.byref(norm_args(**change)), None), code)


def test_norm_null_arguments():
    refused(ags.load_library().lora_i8_rmsnorm(None, None), ags.LORA_EINVAL)


def test_matmul_refusals():
    lib = ags.load_library()

    def call(x, w, y=P, dt=0, ld=16, ws=P, nbytes=1 << 40):
        return lib.lora_i8_matmul(ctypes.byref(x), ctypes.byref(w), y, dt, ld, ws, nbytes, None)

    refused(call(mat(300, 8), mat(16, 9)), ags.LORA_EINVAL)
    refused(call(mat(300, 8), mat(16, 8), y=None), ags.LORA_EINVAL)
    refused(call(mat(300, 8), mat(16, 8), ld=15), ags.LORA_EINVAL)
    refused(call(mat(300, 8), mat(16, 8), dt=-1), ags.LORA_EINVAL)
    refused(call(mat(300, 8, codes=0), mat(16, 8)), ags.LORA_EINVAL)
    refused(call(mat(300, 8), mat(16, 8), ws=P + 16), ags.LORA_EINVAL)
    assert call(mat(0, 8), mat(16, 8)) == ags.LORA_OK and call(mat(3, 8), mat(0, 8)) == ags.LORA_OK
    for n in (9, 100, 300, 5000):
        need = ags.lora_i8_matmul_workspace_bytes(n, 16, 8)
        if need:
            refused(call(mat(n, 8), mat(16, 8), ws=None), ags.LORA_EINVAL)
            refused(call(mat(n, 8), mat(16, 8), nbytes=need - 1), ags.LORA_ENOSPACE)


def test_matmul_workspace_sizes():
    last = 0
    for n in (0, 1, 8, 9, 64, 256, 257, 16384):
        need = ags.lora_i8_matmul_workspace_bytes(n, 4096, 4096)
        assert need >= last
        last = need
    with pytest.raises(ags.LoraError):
        ags.lora_i8_matmul_workspace_bytes(-1, 16, 8)


class Weight:
    rows, cols = 64, 256
    struct = ags.lora_i8_matrix()


@pytest.fixture
def call(monkeypatch):
    """lora_i8_linear_fwd of 20 tokens on host tensors; returns whether the library was called."""
    reached = []

    class Library:
        def lora_i8_linear_fwd(self, *args):
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
        ags.lora_i8_linear_fwd(handle, Weight, x, y, seg, torch.zeros(1024, dtype=torch.uint8))
        return len(reached) == 1

    run.reached = reached
    return run


def half(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def test_linear_tensors_that_match_reach_the_library(call):
    assert call(half(20, 256), half(20, 64))


@pytest.mark.parametrize("x,y", [
    (half(19, 256), half(20, 64)), (half(20, 248), half(20, 64)), (half(20 * 256), half(20, 64)), (half(20, 256), half(19, 64)),
    (half(20, 256), half(40, 32)), (half(20, 256).bfloat16(), half(20, 64)), (half(20, 256), half(20, 64).float())])
def test_linear_other_shapes_and_types_are_refused(call, x, y):
    with pytest.raises(ags.LoraError) as e:
        call(x, y)
    assert e.value.code == ags.LORA_EINVAL and not call.reached


def test_tensors_off_the_gpu_are_refused():
    with pytest.raises(ValueError):
        ags.I8Matrix(64, 256, "cpu")
    with pytest.raises(ValueError):
        ags.lora_i8_rmsnorm(torch.zeros(4, 8), torch.zeros(8), 1e-5, y=torch.zeros(4, 8))
    with pytest.raises(ValueError):
        ags.lora_i8_rmsnorm(torch.zeros(8), torch.zeros(8), 1e-5)
