"""What layer.py's calls on float and 8-bit experts see to before anything is
enqueued (no GPU needed: no call here gets as far as the library)."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import _binding as B
from int4_routed_expert_logits_amd import layer as L

BF16 = torch.bfloat16
E, D, F, T = 4, 128, 64, 3


@pytest.fixture
def no_library(monkeypatch):
    """Any call of the library's binding ends the test."""
    def enqueued(*a, **k):
        raise AssertionError("the library was called")
    for name in B.EXPORTS:
        if callable(getattr(B, name, None)) and not name.endswith("_bytes"):
            monkeypatch.setattr(B, name, enqueued)


def bf(*shape, device="cpu"):
    return torch.zeros(shape, dtype=BF16, device=device)


def layer(codes=False):
    sh = moe.Shape(D, F, E, 2, 64, 0)
    buf = L.FloatLayerBuffers.allocate(sh, T, codes=codes, device="cpu")
    if codes:
        q = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)  # noqa: E731
        return L.FloatExperts(q(E, 2 * F, D), q(E, D, F),
                              scales=(torch.zeros(E, 1, 1), torch.zeros(E, 1, 1))), buf
    return L.FloatExperts(bf(E, 2 * F, D), bf(E, D, F)), buf


X_BAD = [
    ("float32", lambda: bf(T, D).float(), TypeError, "x is torch.float32"),
    ("expanded", lambda: bf(D).expand(T, D), ValueError, "x is not contiguous"),
    ("strided", lambda: bf(T, 2 * D)[:, :D], ValueError, "x is not contiguous"),
    ("transposed", lambda: bf(D, T).t(), ValueError, "x is not contiguous"),
    ("elsewhere", lambda: bf(T, D, device="meta"), ValueError, "x is on meta"),
]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("what,x,error,match", X_BAD, ids=[b[0] for b in X_BAD])
def test_layer_refuses_an_x_it_would_read_past(no_library, what, x, error, match, codes):
    ex, buf = layer(codes)
    with pytest.raises(error, match=match):
        L.run_layer_float(x(), torch.zeros(E, D), None, ex, buf)
    if not codes:
        with pytest.raises(error, match=match):
            L.run_layer_float_grad(bf(T, D), x(), ex, buf, L.FloatLayerGrads.allocate(buf, ex))


ROUTER_BAD = [
    ("few experts", lambda: torch.zeros(E - 1, D), None, ValueError, "w_router has shape"),
    ("few columns", lambda: torch.zeros(E, D // 2), None, ValueError, "w_router has shape"),
    ("bf16", lambda: bf(E, D), None, TypeError, "w_router is torch.bfloat16"),
    ("transposed", lambda: torch.zeros(D, E).t(), None, ValueError, "w_router is not contiguous"),
    ("short bias", lambda: torch.zeros(E, D), lambda: torch.zeros(E - 1), ValueError, "bias has shape"),
    ("float64 bias", lambda: torch.zeros(E, D), lambda: torch.zeros(E).double(), TypeError,
     "bias is torch.float64"),
    ("strided bias", lambda: torch.zeros(E, D), lambda: torch.zeros(2 * E)[::2], ValueError,
     "bias is not contiguous"),
    ("no router", lambda: None, None, ValueError, "w_router is missing"),
]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("what,wr,bias,error,match", ROUTER_BAD, ids=[b[0] for b in ROUTER_BAD])
def test_layer_refuses_a_router_it_would_read_past(no_library, what, wr, bias, error, match, codes):
    ex, buf = layer(codes)
    with pytest.raises(error, match=match):
        L.run_layer_float(bf(T, D), wr(), bias and bias(), ex, buf)


# ----------------------------------------------------------------------------
# streams, by what is asked of them
# ----------------------------------------------------------------------------

class Stream:
    """Records what is asked of it."""
    cuda_stream = 77

    def __init__(self, log, name):
        self.log, self.name = log, name

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


@pytest.fixture
def streams(monkeypatch):
    """(log, a side stream): the log of waits, calls and recorded tensors."""
    log = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(log, "current"))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.append(("record", s.name, t.data_ptr())))
    return log, Stream(log, "side")


def test_quantize_on_a_stream_waits_and_keeps_its_memory(streams, monkeypatch):
    """The memory it allocates belongs to the current stream: the side stream
    waits for the work queued there before it writes, and no tensor that it
    touches is handed out again before it is done."""
    log, side = streams
    monkeypatch.setattr(B, "moe_blockscale_quantize",
                        lambda w, rows, codes, scales, stream: log.append(
                            ("write", w.data_ptr(), codes.data_ptr(), scales.data_ptr(), stream)))
    ex = L.FloatExperts(bf(E, 2 * F, D), bf(E, D, F), bf(1, 2 * F, D), bf(1, D, F))
    q = L.FloatExperts.quantize(ex, side)
    assert log[0] == ("wait", "side", "current")
    writes = [e for e in log if e[0] == "write"]
    assert len(writes) == 4 and all(e[-1] is side for e in writes)
    recorded = {e[2] for e in log if e[0] == "record" and e[1] == "side"}
    assert recorded == {p for e in writes for p in e[1:-1]}
    assert q.gate_up.shape == ex.gate_up.shape and q.shared_scales[1].shape == (1, 1, 1)
    log.clear()
    L.FloatExperts.quantize(ex)
    assert [e[0] for e in log] == ["write"] * 4  # on the current stream: nothing to wait for


def test_block_runs_its_layer_on_its_stream(streams, monkeypatch):
    """A layer that names no stream reads `normed` behind the norm that writes it."""
    log, side = streams
    now = ["current"]

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            now.append("current" if self.s is None else self.s.name)

        def __exit__(self, *a):
            now.pop()

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(B, "moe_block_norm", lambda *a, **k: log.append(
        ("norm", (k.get("stream") or a[-1]).name)))

    def inner(n):
        log.append(("layer", now[-1]))
        return n

    t = bf(T, D)
    L.run_block(t, L.BlockNorms(torch.ones(D)), inner, bf(T, D), bf(T, D), stream=side)
    assert log == [("norm", "side"), ("layer", "side"), ("norm", "side")] and now == ["current"]


# ----------------------------------------------------------------------------
# another GPU than the current one
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("current", [0, 1])
def test_layer_runs_on_its_buffers_gpu(monkeypatch, current):
    """moe_route_union and moe_combine launch on the current GPU: the layer and
    its gradient make their buffers' GPU current, and leave the other one so."""
    at = [current]

    class On:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            at.append(self.d)

        def __exit__(self, *a):
            at.pop()

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(B, "_current_device", lambda: at[-1])
    monkeypatch.setattr(B, "_T", B._T or B._types())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    calls = []
    for name in B.EXPORTS:
        if callable(getattr(B, name, None)) and not name.endswith("_bytes"):
            monkeypatch.setattr(B, name, lambda *a, name=name, **k: calls.append((name, at[-1])))
    for codes in (False, True):
        ex, buf = layer(codes)
        L.run_layer_float(bf(T, D), torch.zeros(E, D), None, ex, buf)
        if not codes:
            L.run_layer_float_grad(bf(T, D), bf(T, D), ex, buf, L.FloatLayerGrads.allocate(buf, ex))
    by_address = [(n, d) for n, d in calls if n in ("moe_route_union", "moe_combine")]
    assert len(by_address) == 5 and all(d == 1 for _, d in by_address), by_address
    assert at == [current]


def test_chained_blocks_do_each_norm_once(monkeypatch):
    """Two blocks: the first's pre norm, its layer, one pass for its post norm with
    the second's pre norm, the second's layer, its post norm."""
    log = []
    monkeypatch.setattr(B, "moe_block_norm", lambda y, res, out, normed, *a, **k: log.append(
        ("norm", y is not None, normed is not None)))
    t, n = bf(T, D), [bf(T, D), bf(T, D)]
    norms = [L.BlockNorms(torch.ones(D), torch.ones(D)) for _ in range(2)]
    inner = lambda v: (log.append(("layer", [v is x for x in n].index(True))), v)[1]  # noqa: E731
    L.run_block(t, norms[0], inner, n[0], t, norms[1], n[1])
    L.run_block(t, norms[1], inner, n[1], t, normed_ready=True)
    assert log == [("norm", False, True), ("layer", 0), ("norm", True, True), ("layer", 1),
                   ("norm", True, False)]
