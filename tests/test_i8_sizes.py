"""Sizes past 32 bits, which the C entry points take as int32: refused by the binding, not cut off."""
import pytest
import torch

import adapter_gemm_segment_gb300 as ags


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("rows,cols", [(2 ** 32, 16), (2 ** 32 + 4, 16), (2 ** 31, 16), (4, 2 ** 32 + 16), (-2 ** 32 + 4, 16)])
def test_stored_matrices(rows, cols):
    with pytest.raises(ags.LoraError) as e:
        ags.lora_i8_bytes(rows, cols)
    assert e.value.code in (ags.LORA_EUNSUP, ags.LORA_EINVAL)
    with pytest.raises(ags.LoraError):
        ags.I8Matrix(rows, cols)


@pytest.mark.parametrize("sizes", [(2 ** 32 + 9, 16, 16), (9, 2 ** 32 + 16, 16), (9, 16, 2 ** 32 + 16)])
def test_product_workspaces(sizes):
    with pytest.raises(ags.LoraError):
        ags.lora_i8_matmul_workspace_bytes(*sizes)


def test_linear_workspaces():
    with pytest.raises(ags.LoraError) as e:
        ags.lora_i8_linear_workspace_bytes(None, 2 ** 32 + 9)
    assert e.value.code == ags.LORA_EUNSUP


@pytest.mark.parametrize("shape", [(2 ** 32 + 4, 8), (2 ** 31, 8), (4, 2 ** 32 + 8)])
def test_norms(shape):
    x = torch.empty(shape, dtype=torch.float16, device="meta")
    with pytest.raises(ags.LoraError) as e:
        ags.lora_i8_rmsnorm(x, torch.empty(shape[1], dtype=torch.float16, device="meta"), 1e-5, y=x)
    assert e.value.code == ags.LORA_EUNSUP
