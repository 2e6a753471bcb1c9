"""GPU parity of the layer for a few tokens with its float64 form
(tests/more_ref.py, which also derives the allowances)."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
import more_ref as ref
from block_ref import d64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def weights(g, kind, n, d, f):
    """(gate_up, down, scales ...) on the GPU."""
    shapes = ((n, 2 * f, d), (n, d, f))
    up = lambda v, m: -(-v // m)  # noqa: E731
    if kind == "bf16":
        return tuple((torch.randn(s, generator=g) * s[2] ** -0.5).to(BF16).cuda() for s in shapes)
    if kind == "int8":
        return (*(torch.randint(-128, 128, s, generator=g).to(torch.int8).cuda() for s in shapes),
                *(((torch.rand(s[:2], generator=g) + 0.5) / 74 * s[2] ** -0.5).cuda() for s in shapes))
    return (*((torch.randn(s, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
              for s in shapes),
            *(((torch.rand((n, up(s[1], 128), up(s[2], 128)), generator=g) + 0.5) / 100 *
               s[2] ** -0.5).cuda() for s in shapes))


def make(kind, T, d, f, E, k, shared, seed, idx=None):
    g = gen(seed)
    c = dict(shape=(d, f, E, k, 64, f if shared else 0), T=T,
             x=torch.randn((T, d), generator=g).to(BF16).cuda(), experts=weights(g, kind, E, d, f),
             shared=weights(g, kind, 1, d, f) if shared else None)
    if idx is None:
        idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]) if T else \
            torch.zeros((0, k))
    c["idx"] = idx.int().cuda()
    c["w"] = torch.softmax(torch.randn((T, k), generator=g), 1).cuda()
    return c


def run(c, out=F32, w_router=None, bias=None, stream=None):
    o = torch.full((c["T"], c["shape"][0]), 768.0, dtype=out, device="cuda")
    ws = torch.full((max(256, moe.moe_layer_few_workspace_bytes(c["shape"], c["T"])),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_layer_few(c["shape"], c["x"], w_router, bias, c["experts"], c["shared"], c["idx"],
                      c["w"], o, ws, stream)
    return o


def check(c, got, out, what=""):
    want, allow = ref.layer_few(c["x"], c["idx"], c["w"], c["experts"], c["shared"], out)
    got = d64(got)
    assert torch.isfinite(got).all()
    ratio = float(((got - want).abs() / allow.clamp(min=1e-300)).max()) if got.numel() else 0.0
    say(f"  {what} worst error / allowance {ratio:.3f}")
    assert ratio <= 1.0


LAYERS = {"least": (64, 64, 4, 2), "one_expert": (128, 64, 1, 1), "odd": (320, 192, 8, 3),
          "wide": (192, 1088, 16, 4), "long": (1472, 320, 12, 8), "many": (128, 128, 1024, 8)}
TOKENS = [1, 2, 3, 8, 15, 17, 32]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("layer,T", [("least", t) for t in TOKENS] + [("odd", t) for t in TOKENS] + [
    ("one_expert", 1), ("one_expert", 31), ("wide", 1), ("wide", 16), ("long", 2), ("long", 29),
    ("many", 1), ("many", 32)])
def test_layer(gpu_lib, layer, T, kind, shared):
    say(f"layer_few {layer} {LAYERS[layer]} T={T} {kind} shared={shared}")
    c = make(kind, T, *LAYERS[layer], shared, 3 * T + shared)
    for out in (F32, BF16):
        check(c, run(c, out), out, str(out))
    assert torch.equal(run(c), run(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_largest_sizes(gpu_lib, kind):
    c = make(kind, 2, 8192, 8192, 2, 1, False, 5)
    check(c, run(c), F32, kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_top_32_of_few_tokens(gpu_lib, kind):
    c = make(kind, 8, 192, 128, 64, 32, True, 6)
    check(c, run(c), F32, kind)


@pytest.mark.parametrize("T,k", [(32, 8), (7, 3), (17, 2), (1, 4)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_one_expert_takes_every_pair(gpu_lib, kind, T, k):
    """The same expert in every slot of every token: up to 256 rows of one group."""
    c = make(kind, T, 192, 128, 8, k, True, T, idx=torch.full((T, k), 5))
    check(c, run(c), F32, kind)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_ids_out_of_range_contribute_nothing(gpu_lib, kind):
    idx = torch.tensor([[0, -1, 3], [8, 9, -7], [2 ** 31 - 1, 1, 1], [-2 ** 31, 8, 7]])
    for shared in (False, True):
        c = make(kind, 4, 320, 192, 8, 3, shared, 8, idx=idx)
        check(c, run(c), F32, f"shared={shared}")
    c = make(kind, 4, 320, 192, 8, 3, False, 8, idx=torch.full((4, 3), -1))
    assert (run(c) == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (9, 256, 8), (32, 64, 8), (5, 1024, 32)])
def test_routing_is_the_routers(gpu_lib, kind, T, E, k):
    """With a router the call routes as moe_route does, and gives the bits that it
    gives for that routing."""
    c = make(kind, T, 256, 64, E, k, True, 100 + T)
    g = gen(T)
    w_router = torch.randn((E, 256), generator=g).mul_(0.05).cuda()
    for bias in (None, torch.randn(E, generator=g).cuda()):
        idx, w = torch.empty_like(c["idx"]), torch.empty_like(c["w"])
        ws = torch.empty(max(256, moe.moe_route_workspace_bytes(c["shape"], T)), dtype=torch.uint8,
                         device="cuda")
        moe.moe_route(c["shape"], c["x"], w_router, bias, idx, w, ws)
        c["idx"].fill_(-3)
        c["w"].fill_(9)
        got = run(c, F32, w_router, bias)
        assert torch.equal(c["idx"], idx) and torch.equal(c["w"], w)
        assert torch.equal(got, run(c, F32))
    check(c, got, F32, kind)


def test_a_token_that_is_not_finite_stays_alone(gpu_lib):
    for kind in ("bf16", "e4m3", "int8"):
        c = make(kind, 9, 320, 192, 8, 3, True, 4)
        clean = run(c)
        c["x"][4, 7] = float("nan")
        c["x"][6, 0] = float("inf")
        got = run(c)
        rest = [0, 1, 2, 3, 5, 7, 8]
        assert torch.equal(got[rest], clean[rest])
        assert not torch.isfinite(got[4]).any() and not torch.isfinite(got[6]).all()


def test_weights_that_no_token_chose_are_not_looked_at(gpu_lib):
    c = make("bf16", 3, 320, 192, 8, 2, False, 4, idx=torch.tensor([[0, 2], [2, 5], [5, 0]]))
    clean = run(c)
    for e in (1, 3, 4, 6, 7):
        c["experts"][0][e] = float("nan")
        c["experts"][1][e] = float("inf")
    assert torch.equal(run(c), clean)


def test_infinite_h_is_no_nan(gpu_lib):
    """h past float32's largest is an infinity, whose rest is not inf - inf."""
    c = make("bf16", 1, 64, 64, 1, 1, False, 1, idx=torch.zeros((1, 1)))
    c["x"].fill_(3e38)
    c["experts"][0].fill_(1.0)
    c["experts"][1].fill_(1.0)
    assert (run(c) == float("inf")).all()


@pytest.mark.parametrize("out", [F32, BF16])
def test_h_past_bfloat16s_largest(gpu_lib, out):
    """h = 2^64 (2^63 255/128 + 2^55 3/2) = (2 - 2^-9) 2^127, which float32 holds and
    bf16 would round to infinity.  out = 64 h 2^-20: h's parts hold it exactly in
    float32, and within 2^-17 for an out of bf16, whose own rounding is 2^-9."""
    c = make("bf16", 1, 64, 64, 1, 1, False, 1, idx=torch.zeros((1, 1)))
    c["w"].fill_(1.0)
    c["x"].zero_()
    c["x"][0, :2] = 1.0
    gu = c["experts"][0]
    gu.zero_()
    gu[0, :64, 0] = 2.0 ** 64
    gu[0, 64:, 0] = 2.0 ** 63 * 255 / 128
    gu[0, 64:, 1] = 2.0 ** 55 * 1.5
    c["experts"][1].fill_(2.0 ** -20)
    h = 2.0 ** 64 * (2.0 ** 63 * 255 / 128 + 2.0 ** 55 * 1.5)
    got = d64(run(c, out))
    allow = 0.0 if out == F32 else 2.0 ** -17 + 2.0 ** -9
    assert ((got - 64 * h * 2.0 ** -20).abs() <= allow * 64 * h * 2.0 ** -20).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_an_infinite_weight_where_workgroups_share_the_steps(gpu_lib, kind):
    """Two experts of 64 columns over a long f: several workgroups share a tile's
    steps, and the ones without any of the second expert leave its weight alone."""
    c = make(kind, 1, 64, 8192, 2, 2, False, 3, idx=torch.tensor([[0, 1]]))
    c["x"].abs_()
    for w in c["experts"][:2]:
        w.copy_(w.float().abs().clamp(max=100).to(w.dtype))
    for weights in ((1.0, float("inf")), (float("inf"), 1.0)):
        c["w"].copy_(torch.tensor([weights]))
        assert (run(c) == float("inf")).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("T,d,f,E,k,shared", [
    (1, 64, 8192, 2, 2, True), (28, 128, 3584, 5, 3, False), (8, 2176, 1088, 16, 8, True),
    (32, 4160, 64, 100, 8, False), (32, 4608, 192, 40, 8, True), (16, 8128, 320, 4, 2, False)])
def test_layouts_of_the_down_product(gpu_lib, T, d, f, E, k, shared, kind):
    """Split steps, one to four fragments a wavefront, and columns that fill the last
    workgroup's in part."""
    c = make(kind, T, d, f, E, k, shared, T + d)
    for out in (F32, BF16):
        check(c, run(c, out), out, f"{kind} {out}")
    assert torch.equal(run(c), run(c))


def test_256_experts_of_one_pair_each(gpu_lib):
    """As many experts hit as the grouping holds."""
    idx = torch.randperm(1024, generator=gen(9))[:256].view(32, 8)
    for kind in ("bf16", "e4m3", "int8"):
        c = make(kind, 32, 128, 64, 1024, 8, True, 10, idx=idx)
        check(c, run(c), F32, kind)


def test_one_workspace_in_two_graphs(gpu_lib):
    """Graphs that are replayed one after the other may share a workspace."""
    cases = [make(kind, T, 320, 192, 8, 3, True, T) for kind, T in (("bf16", 5), ("int8", 20))]
    ws = torch.empty(max(moe.moe_layer_few_workspace_bytes(c["shape"], c["T"]) for c in cases),
                     dtype=torch.uint8, device="cuda")
    want = [run(c) for c in cases]
    graphs, outs = [], [torch.empty_like(w) for w in want]
    for c, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_layer_few(c["shape"], c["x"], None, None, c["experts"], c["shared"], c["idx"],
                              c["w"], o, ws)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].fill_(3)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


def test_batch_does_not_change_a_token_much(gpu_lib):
    """A token alone and among others: both within their allowances of each other's
    reference."""
    c = make("e4m3", 12, 320, 192, 8, 3, True, 21)
    whole = run(c)
    for t in (0, 11):
        one = dict(c, T=1, x=c["x"][t:t + 1].clone(), idx=c["idx"][t:t + 1].clone(),
                   w=c["w"][t:t + 1].clone())
        check(one, run(one), F32)
        check(one, whole[t:t + 1], F32)


def test_two_at_once_on_two_streams(gpu_lib):
    cases = [make("bf16", 8, 320, 192, 8, 3, True, s) for s in (31, 32)]
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(run(c))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_captured_and_replayed(gpu_lib, kind):
    c = make(kind, 5, 320, 192, 8, 3, True, 41)
    g = gen(1)
    w_router = torch.randn((8, 320), generator=g).mul_(0.05).cuda()
    out = torch.empty((5, 320), device="cuda")
    ws = torch.empty(moe.moe_layer_few_workspace_bytes(c["shape"], 5), dtype=torch.uint8,
                     device="cuda")

    def call():
        moe.moe_layer_few(c["shape"], c["x"], w_router, None, c["experts"], c["shared"], c["idx"],
                          c["w"], out, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        c["x"].copy_(torch.randn((5, 320), generator=g).to(BF16))
        call()
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(3)
        c["idx"].fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_empty_batch(gpu_lib):
    c = make("bf16", 0, 64, 64, 4, 2, False, 1)
    assert run(c).shape == (0, 64)
