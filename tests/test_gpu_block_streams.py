"""layer.py's helpers on another stream than the current one."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import layer as L
from test_gpu_block import BF16, gen, rand, say

pytestmark = pytest.mark.gpu

BUSY = 40_000_000  # cycles, about 20 ms


def same_codes(a, b):
    return all(torch.equal(getattr(a, n).view(torch.uint8), getattr(b, n).view(torch.uint8))
               for n in ("gate_up", "down")) and all(map(torch.equal, a.scales, b.scales))


@pytest.mark.parametrize("handle", [False, True])
def test_quantize_on_a_side_stream_leaves_queued_work_its_memory(gpu_lib, handle):
    """Memory freed with work still queued on it may come back as the codes': that
    work reads what it was queued to read, and the codes are the quantiser's."""
    say(f"quantize on a side stream, raw handle {handle}")
    g = gen(1)
    ex = L.FloatExperts(rand(g, 8, 512, 1024), rand(g, 8, 1024, 512))
    want = L.FloatExperts.quantize(ex)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(3):
        torch.cuda.empty_cache()
        old = torch.full((8 * 512 * 1024,), 7, dtype=torch.uint8, device="cuda")
        copy = torch.empty_like(old)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        copy.copy_(old)
        at = old.data_ptr()
        del old
        got = L.FloatExperts.quantize(ex, side.cuda_stream if handle else side)
        say(f"  the codes took the freed memory: {got.gate_up.data_ptr() == at}")
        torch.cuda.current_stream().wait_stream(side)
        assert (copy == 7).all() and same_codes(got, want)
        assert torch.equal(got.gate_up.view(torch.uint8), want.gate_up.view(torch.uint8))


def test_quantize_may_be_followed_by_freeing_the_weights(gpu_lib):
    """The bf16 weights, dropped while the side stream still reads them."""
    side = torch.cuda.Stream()
    shape = (8, 512, 1024)
    w = [rand(gen(i), *shape) for i in range(2)]
    want = L.FloatExperts.quantize(L.FloatExperts(w[0], w[1]))
    torch.cuda.synchronize()
    ex = L.FloatExperts(w[0].clone(), w[1].clone())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = L.FloatExperts.quantize(ex, side)
    del ex
    junk = [torch.full(shape, 3.0, dtype=BF16, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert same_codes(got, want) and len(junk) == 4


@pytest.mark.parametrize("handle", [False, True])
def test_block_on_a_side_stream(gpu_lib, handle):
    """run_block's norms, and a layer that names no stream, in order on `stream`,
    behind work that is queued there: the same as on the current one."""
    sh, T = moe.Shape(320, 192, 8, 2, 64, 192), 40
    g, d, f, E = gen(3), 320, 192, 8
    ex = L.FloatExperts(rand(g, E, 2 * f, d, scale=0.05), rand(g, E, d, f, scale=0.07),
                        rand(g, 1, 2 * f, d, scale=0.05), rand(g, 1, d, f, scale=0.07))
    wr, res = rand(g, E, d, dt=torch.float32, scale=0.05), rand(g, T, d)
    norms = L.BlockNorms(torch.rand(d, generator=g).cuda(), torch.rand(d, generator=g).cuda())

    def block(stream):
        buf = L.FloatLayerBuffers.allocate(sh, T)
        normed, out = (torch.zeros((T, d), dtype=BF16, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        s = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        L.run_block(res, norms, lambda n: L.run_layer_float(n, wr, None, ex, buf), normed, out,
                    stream=stream and (stream.cuda_stream if handle else stream))
        torch.cuda.synchronize()
        return out

    want = block(None)
    assert torch.equal(block(torch.cuda.Stream()), want) and (want != 0).any()
