"""The norm's outputs over its inputs: an output may lie exactly on an input, or share nothing with it.  Anything else
(another row stride, a shift) is written by one row while another still reads it, and refused on the host.  Addresses here
are made up; no call gets past the host."""
import ctypes
import itertools

import numpy as np
import pytest

import adapter_gemm_segment_gb300 as ags

BASE = 0x1000000
ARRAYS = ("x", "residual", "residual_out", "y")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def call(rows, cols, **where):
    """rc of the norm of float32 arrays at (element offset, row stride).  out has a row too many, which is checked last:
    no call gets past the host."""
    a = ags.lora_i8_norm()
    a.weight_dev = BASE >> 1
    a.rows, a.cols, a.dtype, a.eps = rows, cols, 0, 1e-5
    out = ags.lora_i8_matrix(BASE, BASE, rows + 1, cols)
    a.out = ctypes.pointer(out)
    for name, ld in zip(ARRAYS, ("ldx", "ldr", "ldro", "ldy")):
        if where.get(name) is not None:
            at, stride = where[name]
            setattr(a, name + "_dev", BASE + 4 * at)
            setattr(a, ld, stride)
    return ags.load_library().lora_i8_rmsnorm(ctypes.byref(a), None)


def cells(rows, cols, at, ld):
    return (at + np.arange(rows)[:, None] * ld + np.arange(cols)).ravel()


def sound(rows, cols, out, other):
    """Whether every element that the two share is the same one of both."""
    _, i, j = np.intersect1d(cells(rows, cols, *out), cells(rows, cols, *other), return_indices=True)
    return np.array_equal(i, j)


FAR = 1 << 20


@pytest.mark.parametrize("output", ["residual_out", "y"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (2, 8), (4, 5), (7, 3)])
def test_overlaps_that_race_are_refused(output, rows, cols):
    """Every small shift and stride, against the elements that the two share."""
    refused = 0
    for ld_in, ld_out, shift in itertools.product(range(cols, 4 * cols), range(cols, 4 * cols), range(-3 * cols, 3 * cols + 1)):
        for over in ("x", "residual"):
            where = {"x": (FAR, cols), "residual": (2 * FAR, cols), "residual_out": (3 * FAR, cols), "y": (4 * FAR, cols)}
            where[over], where[output] = (100, ld_in), (100 + shift, ld_out)
            assert call(rows, cols, **where) == ags.LORA_EINVAL
            raced = "overlaps" in ags.lora_last_error()
            assert raced != sound(rows, cols, where[output], where[over]), (over, ld_in, ld_out, shift)
            refused += raced
    assert refused > 100


def test_y_over_residual_out_is_refused():
    for shift, ld in ((0, 8), (3, 8), (8, 8), (0, 9), (-8, 16)):
        where = {"x": (FAR, 8), "residual": (2 * FAR, 8), "residual_out": (100, 8), "y": (100 + shift, ld)}
        assert call(4, 8, **where) == ags.LORA_EINVAL and "y overlaps residual_out" in ags.lora_last_error()
    # without a residual too: residual_out is x's copy then
    assert call(4, 8, x=(FAR, 8), residual_out=(100, 8), y=(104, 8)) == ags.LORA_EINVAL
    assert "y overlaps residual_out" in ags.lora_last_error()


@pytest.mark.parametrize("where", [
    {"x": (100, 8), "residual": (FAR, 8), "residual_out": (FAR, 8), "y": (100, 8)},         # both in place
    {"x": (100, 16), "residual": (108, 16), "residual_out": (108, 16), "y": (FAR, 8)},      # windows of one buffer
    {"x": (100, 24), "residual": (108, 24), "residual_out": (116, 24), "y": (100, 24)},
    {"x": (100, 16), "residual": (FAR, 8), "residual_out": (2 * FAR, 8), "y": (108, 16)},
    {"x": (100, 8), "residual": (132, 8), "residual_out": (164, 9), "y": (132, 8)},         # one behind the other
    {"x": (100, 16), "residual": (FAR, 8), "residual_out": (2 * FAR, 8), "y": (108, 48)}])  # strides that never meet
def test_sound_overlaps_are_taken(where):
    assert call(4, 8, **where) == ags.LORA_EINVAL
    assert "out is 5 x 8" in ags.lora_last_error()
