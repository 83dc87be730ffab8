"""Prefill batches (more than 256 tokens) over pools whose r_max is an odd multiple of 8: the
tensor-core shrink's MMA is then 8 rows wider than the adapter rows it loads."""
import numpy as np
import pytest
import torch

from adapter_gemm_segment_gb300 import workloads as wl
from oracle import lora_oracle as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r_max,slots", [(8, 3), (24, 1), (24, 3), (40, 5), (72, 3), (136, 2)])
def test_prefill_odd_rank_blocks(lib, r_max, slots):
    case = wl.random_case(31, 300, 512, 256, [r_max] * slots, r_max=r_max, dtype=torch.bfloat16, p_base=0.2)
    pool = lib.LoraPool(case.h_in, case.h_out, r_max, slots, case.dtype, "cuda")
    for s in range(slots):
        pool.load_slot(s, case.adapters.A[s].cuda(), case.adapters.B[s].cuda(), case.adapters.alphas[s])
    seg = pool.segment(case.idx.cuda())
    for variant in (lib.LORA_VARIANT_FUSED, lib.LORA_VARIANT_SEPARATE):
        y = pool.linear(torch.zeros_like(case.W).cuda(), case.x.cuda(), seg, variant=variant)
        got = y.cpu().double().numpy()
        W0 = wl.LinearCase(case.name, case.x, torch.zeros_like(case.W), case.adapters, case.idx)
        ref = np.asarray(O.lora_linear_case(W0), dtype=np.float64)
        assert np.isfinite(got).all()
        # s rounded to bf16 (2^-9), y rounded to bf16 (2^-9), against the largest output
        assert np.abs(got - ref).max() <= 1e-2 * np.abs(ref).max()
        assert lib.lora_segment_status(seg) == lib.LORA_OK
    pool.close()
