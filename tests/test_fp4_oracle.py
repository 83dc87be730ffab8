"""The 4-bit oracle against hand-worked values, and the entry points' refusals (host checks only:
every call here is refused before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

from oracle import fp4_oracle as Q


def test_hand_worked_block():
    # largest 6 -> floor(log2 6) - 2 = 0: scale 1, byte 127
    x = np.zeros((1, 32))
    x[0, :14] = [6, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, -0.25, -0.75, -2.5, -7.0 / 8]
    codes, scales = Q.quantise(x)
    assert scales.tolist() == [[127]]
    got = Q.values(codes, scales, 32)[0, :14]
    assert got.tolist() == [6, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 0, -1, -2, -1]
    assert codes[0, 10] == 8  # a negative value that rounds to nothing keeps its sign


def test_saturation_and_scale_range():
    x = np.zeros((6, 32))
    x[0, 0] = 7.9  # scale 1, 7.9 saturates at 6
    x[1, 0] = 8.0  # next binade: scale 2, value 4 * 2
    x[2, 0] = 2.0 ** -149  # far below the smallest scale: byte 0, rounds to nothing
    x[3, 0] = 2.0 ** -125  # scale 2^-127, value 4 * 2^-127
    x[4, 0] = 3.4e38
    x[5, 3] = np.inf
    codes, scales = Q.quantise(x)
    assert scales[:, 0].tolist() == [127, 128, 0, 0, 127 + 125, 255]
    v = Q.values(codes, scales, 32)
    assert v[0, 0] == 6 and v[1, 0] == 8 and v[2, 0] == 0 and v[3, 0] == 2.0 ** -125
    assert v[4, 0] == 6 * 2.0 ** 125 and np.isnan(v[5]).all() and (codes[5] == 0).all()


def test_nearest_by_brute_force():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 96)) * np.exp(rng.standard_normal((40, 1)) * 3)
    codes, scales = Q.quantise(x)
    v = Q.values(codes, scales, 96)
    for r in range(40):
        for c in range(96):
            s = 2.0 ** (int(scales[r, c // 32]) - 127)
            near = min(abs(x[r, c] - q * s) for q in Q.VALUES)
            clipped = abs(x[r, c]) > 6 * s
            assert clipped or abs(x[r, c] - v[r, c]) == near


def test_scale_offsets_are_a_permutation():
    rows, cols = 300, 500
    r, b = np.meshgrid(np.arange(384), np.arange(16), indexing="ij")
    off = Q.scale_offset(r, b, cols)
    assert sorted(off.ravel().tolist()) == list(range(3 * 4 * 512))
    assert Q.pack_scales(np.zeros((rows, 16), np.uint8), cols).size == 3 * 4 * 512


# ---- refusals ---------------------------------------------------------------------------------

FAKE = 1 << 20  # an aligned address that no accepted call here dereferences


def _lib():
    import adapter_gemm_segment_gb300 as ags

    return ags, ags.load_library()


def _matrix(ags, rows=64, cols=256, codes=FAKE, scales=FAKE):
    return ags.lora_fp4_matrix(codes, scales, rows, cols)


def test_sizes():
    ags, _ = _lib()
    assert ags.lora_fp4_bytes(1, 1) == (16, 1024)
    assert ags.lora_fp4_bytes(129, 257) == (129 * 144, 2 * 4 * 512)
    assert ags.lora_fp4_bytes(0, 64) == (0, 0)
    assert ags.lora_fp4_bytes(11008, 4096) == (11008 * 2048, 86 * 32 * 512)
    for rows, cols in ((-1, 4), (4, 0), (4, -3)):
        with pytest.raises(ags.LoraError) as e:
            ags.lora_fp4_bytes(rows, cols)
        assert e.value.code == ags.LORA_EINVAL


@pytest.mark.parametrize("kw,ptr,dtype,ld", [
    (dict(), 0, 0, 256),                    # no input
    (dict(), FAKE, 7, 256),                 # unknown dtype
    (dict(), FAKE, 0, 255),                 # rows overlap
    (dict(), FAKE + 2, 0, 256),             # float32 off its alignment
    (dict(codes=0), FAKE, 0, 256),
    (dict(scales=FAKE + 16), FAKE, 0, 256),
    (dict(rows=-1), FAKE, 0, 256),
    (dict(cols=0), FAKE, 0, 256),
])
def test_quantize_and_dequantize_refusals(kw, ptr, dtype, ld):
    ags, lib = _lib()
    m = _matrix(ags, **kw)
    assert lib.lora_fp4_quantize(ptr, dtype, ld, ctypes.byref(m), None) == ags.LORA_EINVAL
    assert lib.lora_fp4_dequantize(ctypes.byref(m), ptr, dtype, ld, None) == ags.LORA_EINVAL
    assert ags.lora_last_error()


def test_matmul_refusals():
    ags, lib = _lib()
    x, w = _matrix(ags, 8, 256), _matrix(ags, 32, 256)
    call = lambda x, w, y=FAKE, dt=1, ld=32: lib.lora_fp4_matmul(  # noqa: E731
        ctypes.byref(x) if x else None, ctypes.byref(w) if w else None, y, dt, ld, None)
    assert call(None, w) == ags.LORA_EINVAL
    assert call(x, None) == ags.LORA_EINVAL
    assert call(x, _matrix(ags, 32, 255)) == ags.LORA_EINVAL
    assert call(x, w, y=0) == ags.LORA_EINVAL
    assert call(x, w, y=FAKE + 1) == ags.LORA_EINVAL
    assert call(x, w, dt=9) == ags.LORA_EINVAL
    assert call(x, w, ld=31) == ags.LORA_EINVAL
    # nothing to do is not an error
    assert call(_matrix(ags, 0, 256, 0, 0), w, y=0) == ags.LORA_OK
    assert call(x, _matrix(ags, 0, 256, 0, 0), y=0) == ags.LORA_OK
