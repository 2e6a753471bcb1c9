"""What the AdamW step's Python side sees to, on tensors of the CPU (no GPU needed:
every step below is refused)."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import layer as L

BF16 = torch.bfloat16
NAMES = ("params", "masters", "grads", "m", "v", "m_scales", "v_scales")


def z(n, dt=torch.float32):
    return torch.zeros(n, dtype=dt)


def lists(n=300):
    """Two bf16 tensors with masters and 8-bit moments, by argument name."""
    types = dict(params=BF16, grads=BF16, m=torch.float8_e4m3fn, v=torch.uint8)
    return {k: [z(2 if "scales" in k else n, types.get(k, torch.float32)) for _ in range(2)] for k in NAMES}


@pytest.mark.parametrize("how", ["replaced", "moved away and back"])
@pytest.mark.parametrize("name", NAMES)
def test_a_step_refuses_memory_that_was_replaced(name, how):
    """Of any of its arrays: it would write to the old memory, and the tensor not see it."""
    a = lists()
    q = moe.AdamWTensors(**a)
    t = a[name][1]
    if how == "replaced":
        t.data = torch.zeros_like(t)
    else:
        t.data = t.data.to(torch.float64)
        t.data = t.data.to(a[name][0].dtype)
    with pytest.raises(ValueError, match="lies elsewhere"):
        moe.moe_adamw(q, torch.ones(1, dtype=torch.int64), 1e-3)


def test_a_step_takes_lists_that_stayed():
    q = moe.AdamWTensors(**lists())
    with pytest.raises(ValueError, match="not on the GPU"):  # past the look at the memory
        moe.moe_adamw(q, torch.ones(1, dtype=torch.int64), 1e-3)


@pytest.mark.parametrize("bits", [32, 8])
def test_state_that_is_put_in_place_of_the_steps_is_refused(bits):
    opt = L.AdamW([z(300, BF16)], [z(300)], bits)
    state = [opt.params, opt.grads, opt.masters, opt.m, opt.v]
    for q in state + ([opt.m_scales, opt.v_scales] if bits == 8 else []):
        with pytest.raises(TypeError):
            q[0] = torch.zeros_like(q[0])
    opt.m[0].data = torch.zeros_like(opt.m[0])
    with pytest.raises(ValueError, match="lies elsewhere"):
        opt.step(1e-3)
    assert int(opt.count) == 0
