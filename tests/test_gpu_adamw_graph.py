"""The AdamW step beside torch's autograd."""
import pytest
import torch

from int4_routed_expert_logits_amd import layer as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.bfloat16, 8)])
def test_a_backward_pass_over_weights_of_before_the_step_is_refused(gpu_lib, dtype, bits):
    print(dtype, bits, flush=True)
    p = torch.nn.Parameter(torch.ones(64, dtype=dtype, device="cuda"))
    grad = torch.ones(64, device="cuda")
    opt = L.AdamW([p], [grad], bits)
    x = torch.ones(64, dtype=dtype, device="cuda", requires_grad=True)
    loss = (p * x).sum()
    before = p._version
    opt.step(1e-2)
    assert p._version > before and not torch.equal(p, torch.ones_like(p))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    (p * x).sum().backward()  # over the new ones
    assert torch.equal(x.grad, p.detach())


def test_parameters_made_in_inference_mode_are_stepped(gpu_lib):
    with torch.inference_mode():
        p = torch.ones(64, device="cuda")
    opt = L.AdamW([p], [torch.ones(64, device="cuda")])
    opt.step(1e-2)
    assert (p < 1).all()
