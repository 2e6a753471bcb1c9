"""The norms of include/moe_int4_block.h at their edges: no rows beside weights that
are not finite, operands that are absent, blocks in a chain."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import layer as L
from test_gpu_block import BF16, F32, gen, poison, rand

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


def kernels_of(call):
    """Names of the kernels that a call launches."""
    call()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.key for e in p.key_averages()]


@pytest.mark.parametrize("y,res,pre,ahead", [
    (BF16, BF16, None, True), (BF16, BF16, BF16, True), (None, BF16, BF16, True),
    (BF16, None, BF16, True), (BF16, BF16, F32, False), (F32, F32, None, False),
    (None, F32, BF16, False), (BF16, F32, None, False)])
def test_norm_gradient_of_bf16_rows_fetches_ahead(gpu_lib, y, res, pre, ahead):
    """The kernel that reads the next row early (its second argument) is for rows
    of bf16, whatever type is given for a row that is not there."""
    T, d = 8, 520
    row = lambda dt: None if dt is None else torch.ones((T, d), dtype=dt, device="cuda")  # noqa: E731
    w = torch.ones(d, device="cuda")
    rdt = res or y
    dy, dres = row(y), row(rdt)
    names = kernels_of(lambda: moe.moe_block_norm_grad(
        row(y), row(res), row(rdt), row(pre), dy, dres, None, None, None,
        w if y and not res else None, w if pre else None))
    [name] = [n for n in names if "norm_grad_rows" in n]
    assert name.split("<")[1].split(",")[1].strip() == ("true" if ahead else "false"), name


def test_chained_blocks_are_the_blocks_one_by_one(gpu_lib):
    """The second block on the first's next_normed, against its norm done alone: the
    same bits where the residual is float32, so that nothing is rounded in between."""
    T, d, eps = 5, 136, 1e-5
    g = gen(5)
    res, w = rand(g, T, d, dt=F32), [1 + rand(g, d, dt=F32, scale=0.1) for _ in range(4)]
    norms = [L.BlockNorms(w[0], w[1], eps=eps), L.BlockNorms(w[2], w[3], eps=eps)]
    layer = lambda n: n * 0.5  # noqa: E731
    new = lambda: torch.empty((T, d), device="cuda")  # noqa: E731
    n, r = [new(), new()], [new(), new(), new()]
    L.run_block(res, norms[0], layer, n[0], r[0], norms[1], n[1])
    L.run_block(r[0], norms[1], layer, n[1], r[1], normed_ready=True)
    L.run_block(r[0], norms[1], layer, new(), r[2])
    assert torch.equal(r[1], r[2])
