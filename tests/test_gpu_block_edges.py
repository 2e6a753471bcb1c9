"""Values and sizes at the edge of the calls in include/moe_int4_block.h: no rows
beside weights that are not finite."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from test_gpu_block import BF16, F32, poison

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_gradients_of_no_rows_are_zero_beside_nonfinite_weights(gpu_lib, dt, bad):
    d = 136
    e = torch.empty((0, d), dtype=dt, device="cuda")
    w, gate = torch.full((d,), bad, device="cuda"), torch.full((1, d), bad, dtype=dt, device="cuda")
    dw, dg = [poison((d,), F32) for _ in range(2)], poison((1, d), dt)
    moe.moe_block_norm_grad(e, e, e, e, e.clone(), e.clone(), dw[0], dw[1], dg, w, w, gate)
    assert (dw[0] == 0).all() and (dw[1] == 0).all() and (dg == 0).all()
