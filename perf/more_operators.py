"""Timed cases of the operators on 8-bit integer experts, of the layer for a few
tokens and of the optimiser's step.

  rowscale_mm  y[p] = W_e x[row(p)] over rows grouped by expert, in 8-bit
               integers with a float32 scale per token and per output channel;
               the tokens are quantised within the pass, or come from SwiGLU
  layer_few    the whole layer for a few tokens (routing where asked for, gate,
               up, SwiGLU, down, combine, shared expert) on bfloat16, e4m3 or
               8-bit integer experts
  adamw        one AdamW step over many tensors, states in 32 or in 8 bits

`run` computes a case in its plain form (elementary torch operations in float32,
rounded once at the end), or through the library where `own` is set.  Sizes
are the layers of synth.WORKLOADS (d, f, experts, top-k, tokens); `draw` spreads
over the ranges those stand for.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BLOCK = 128        # e4m3 weights: rows and columns per scale
STATE_BLOCK = 256  # 8-bit optimiser states: elements per scale
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
STEP = 100
LAYER_64 = "268435456,134217728,131072"  # gate and up, down, router: d 2048, f 1024, 64 experts


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # an 8-token step's gate and up products over integer experts of the
        # ~19 MB-expert layer: the activations are quantised, then about 57
        # experts' codes are read
        dict(name="rowscale_step_8", op="rowscale_mm", T=8, k=8, E=256, N=4096, K=6144,
             zipf=False, gather=True, swiglu=False, out="f32"),
        # the same layer over a 2048-token prompt with skewed routing
        dict(name="rowscale_prompt_2048", op="rowscale_mm", T=2048, k=8, E=256, N=4096, K=6144,
             zipf=True, gather=True, swiglu=False, out="bf16"),
        # ... and its down products: SwiGLU of the 16,384 rows, quantised, first
        dict(name="rowscale_down_2048", op="rowscale_mm", T=2048, k=8, E=256, N=6144, K=2048,
             zipf=True, gather=False, swiglu=True, out="bf16"),
        # a 4096-token prompt over the 64-expert layer, where the products bound
        # the call
        dict(name="rowscale_prompt_4096", op="rowscale_mm", T=4096, k=8, E=64, N=2048, K=2048,
             zipf=False, gather=True, swiglu=False, out="bf16"),
        # one token through the ~19 MB-expert layer on its bfloat16 checkpoint
        dict(name="few_1_bf16", op="layer_few", T=1, k=8, E=256, d=6144, f=2048, kind="bf16",
             shared=True, route=True, out="f32"),
        # a step of 8 tokens on the same layer's integer experts
        dict(name="few_8_int8", op="layer_few", T=8, k=8, E=256, d=6144, f=2048, kind="int8",
             shared=True, route=True, out="bf16"),
        # three tokens of a draft to verify, routed already, small experts
        dict(name="few_3_e4m3", op="layer_few", T=3, k=8, E=256, d=2048, f=512, kind="e4m3",
             shared=True, route=False, out="f32"),
        # 32 users' tokens on the 64-expert layer: about four rows an expert
        dict(name="few_32_bf16", op="layer_few", T=32, k=8, E=64, d=2048, f=1024, kind="bf16",
             shared=False, route=True, out="bf16"),
        # the norm weights of eight blocks: 16 vectors, where launches count
        dict(name="adamw_norms_16", op="adamw", sizes=",".join(["6144"] * 16), p="f32", g="f32",
             bits=32, scaled=False),
        # the 64-expert layer's bfloat16 weights with float32 masters and states
        dict(name="adamw_layer_64", op="adamw", sizes=LAYER_64, p="master", g="f32", bits=32,
             scaled=True),
        # ... with 8-bit states
        dict(name="adamw_layer_64_8bit", op="adamw", sizes=LAYER_64, p="master", g="f32", bits=8,
             scaled=True),
        # many odd tensors, bfloat16 without masters
        dict(name="adamw_ragged_90", op="adamw", p="bf16", g="bf16", bits=8, scaled=False,
             sizes=",".join(str(1 + (7919 * i * i) % (200003 if i % 5 == 0 else 8191))
                            for i in range(90))),
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(high, max(low, step * round(v / step))))


def draw(rng):
    op = rng.choice(["rowscale_mm", "layer_few", "layer_few", "adamw"])
    while op == "rowscale_mm":
        E = _log(rng, 1, 256)
        c = dict(op=op, T=_log(rng, 1, 4096), k=min(E, rng.randint(1, 8)), E=E,
                 N=_log(rng, 64, 6144, 8), K=_log(rng, 64, 6144, 16), zipf=rng.random() < 0.5,
                 swiglu=rng.random() < 0.3)
        c["gather"] = not c["swiglu"] and rng.random() < 0.5
        c["out"] = "bf16" if c["swiglu"] else rng.choice(["bf16", "f32"])
        # no dearer than the largest listed case: weights and products
        if E * c["N"] * c["K"] <= 6.4e9 and c["T"] * c["k"] * c["N"] * c["K"] <= 4e11:
            return c
    while op == "layer_few":
        E = _log(rng, 1, 256)
        c = dict(op=op, T=_log(rng, 1, 32), k=min(E, rng.randint(1, 8)), E=E,
                 d=_log(rng, 64, 6144, 64), f=_log(rng, 64, 4096, 64),
                 kind=rng.choice(["bf16", "e4m3", "int8"]), shared=rng.random() < 0.5,
                 route=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
        if E * c["d"] * c["f"] <= 3.3e9 and (c["T"] * c["k"] + 1) * c["d"] * c["f"] <= 8.2e8:
            return c
    n, sizes = _log(rng, 1, 200), []
    top = _log(rng, 1, 10 ** 8 // n)
    for _ in range(n):
        sizes.append(str(_log(rng, 1, top)))
    return dict(op=op, sizes=",".join(sizes), p=rng.choice(["f32", "bf16", "master"]),
                g=rng.choice(["bf16", "f32"]), bits=rng.choice([8, 32]), scaled=rng.random() < 0.5)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _choose(g, T, k, E, zipf):
    """[T, k] distinct experts of every token, popular ones more often where `zipf`."""
    logp = torch.zeros(E, device="cuda")
    if zipf:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logp = -1.1 * torch.log(rank.float())
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dt=torch.bfloat16, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(scale)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def integers(*shape):
        """int8 codes as a quantised bell of weights has them."""
        return normal(*shape, scale=40.0).round_().clamp_(-127, 127).to(torch.int8)

    s = dict(case=c)
    if c["op"] == "rowscale_mm":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        P, X = T * k, T if c["gather"] else T * k
        flat = _choose(g, T, k, E, c["zipf"]).reshape(-1)
        perm = torch.argsort(flat, stable=True)
        offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
        ends = offsets.tolist()  # the plain form's plan: the groups that hold rows
        s["groups"] = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
        s |= dict(offsets=offsets.int(), rows=perm.int() if c["gather"] else None,
                  div=k if c["gather"] else 1)
        s["x"] = normal(X, 2 * K, scale=1.5) if c["swiglu"] else normal(X, K)
        s |= dict(wq=integers(E, N, K), ws=2e-4 + 6e-4 * uniform(E, N),
                  xq=torch.empty((X, K), dtype=torch.int8, device="cuda"),
                  xs=torch.empty(X, device="cuda"),
                  y=torch.empty((P, N), dtype=DTYPES[c["out"]], device="cuda"))
    elif c["op"] == "layer_few":
        T, k, E, d, f = c["T"], c["k"], c["E"], c["d"], c["f"]

        def matrices(n, rows, cols):
            if c["kind"] == "bf16":
                return normal(n, rows, cols, scale=0.02), None
            if c["kind"] == "int8":
                return integers(n, rows, cols), 2e-4 + 6e-4 * uniform(n, rows)
            codes = normal(n, rows, cols, scale=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            return codes, 1e-4 + 3e-4 * uniform(n, -(-rows // BLOCK), -(-cols // BLOCK))

        def expert(n):
            (gu, gus), (dn, dns) = matrices(n, 2 * f, d), matrices(n, d, f)
            return gu, dn, gus, dns

        s |= dict(shape=(d, f, E, k, 64, f if c["shared"] else 0), x=normal(T, d),
                  experts=expert(E), shared=expert(1) if c["shared"] else None,
                  w_router=None, bias=None, out=torch.empty((T, d), dtype=DTYPES[c["out"]],
                                                            device="cuda"))
        if c["route"]:
            rank = torch.randperm(E, generator=g, device="cuda") + 1
            s |= dict(w_router=normal(E, d, dt=torch.float32, scale=0.02),
                      bias=-0.3 * torch.log(rank.float()),
                      idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                      w=torch.empty((T, k), device="cuda"))
        else:
            s |= dict(idx=_choose(g, T, k, E, False).int(),
                      w=torch.softmax(normal(T, k, dt=torch.float32), 1))
    else:
        # every kind in one buffer, a tensor from a multiple of 256 elements on, with
        # zeros between them
        sizes = [int(v) for v in c["sizes"].split(",")]
        blocks = [-(-n // STATE_BLOCK) for n in sizes]
        total, f32 = sum(blocks) * STATE_BLOCK, torch.float32
        first = [STATE_BLOCK * sum(blocks[:i]) for i in range(len(sizes))]
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        for i, n in zip(first, sizes):
            used[i:i + n] = True

        def values(scale):
            return normal(total, dt=f32, scale=scale).mul_(used)

        full, m = values(0.02), values(1e-3)
        root, grad = values(3e-3).abs_(), values(2e-3)  # of the second moment
        flat = dict(p=full if c["p"] == "f32" else full.to(torch.bfloat16),
                    master=full if c["p"] == "master" else None, m=m, ms=None, vs=None)
        if c["bits"] == 32:
            flat["v"] = root.square_()
        else:
            flat["m"], flat["ms"] = _m_codes(m.view(-1, STATE_BLOCK))
            flat["v"], flat["vs"] = _v_codes(root.view(-1, STATE_BLOCK))
        s |= dict(flat=flat, grad=grad.to(DTYPES[c["g"]]),
                  step=torch.tensor([STEP], dtype=torch.int64, device="cuda"),
                  scale=torch.tensor([0.5], device="cuda") if c["scaled"] else None)
        # the tensors themselves
        cut = lambda t: [t.view(-1)[i:i + n] for i, n in zip(first, sizes)]  # noqa: E731
        s["lists"] = {k: None if t is None else cut(t) for k, t in (flat | dict(g=s["grad"])).items()
                      if k not in ("ms", "vs")}
        s["lists"] |= {k: None if flat[k] is None else list(flat[k].split(blocks))
                       for k in ("ms", "vs")}
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"rowscale_mm": _rowscale_mm, "layer_few": _layer_few, "adamw": _adamw}[c["op"]](s, c)


def _run_own(s, c):
    import int4_routed_expert_logits_amd as moe
    if c["op"] == "rowscale_mm":
        if c["swiglu"]:
            moe.moe_swiglu_rowscale(s["x"], s["xq"], s["xs"])
        else:
            moe.moe_rowscale_quantize(s["x"], s["xq"], s["xs"])
        moe.moe_rowscale_mm(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], s["y"], s["rows"],
                            s["div"])
        return s["y"]
    if c["op"] == "layer_few":
        n = moe.moe_layer_few_workspace_bytes(s["shape"], c["T"])
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        moe.moe_layer_few(s["shape"], s["x"], s["w_router"], s["bias"], s["experts"], s["shared"],
                          s["idx"], s["w"], s["out"], ws)
        return _few_out(s, c, s["out"], s["idx"], s["w"])
    if "tensors" not in s:  # the list that a training loop makes once
        q = s["lists"]
        s["tensors"] = moe.AdamWTensors(q["p"], q["g"], q["m"], q["v"], q["master"], q["ms"],
                                        q["vs"])
    moe.moe_adamw(s["tensors"], s["step"], LR, BETA1, BETA2, EPS, DECAY, s["scale"])
    return s["flat"]


def _few_out(s, c, out, idx, w):
    return dict(out=out, idx=idx, w=w) if c["route"] else out


def _row_codes(v):
    """(codes, scales) of float32 rows: scale = absmax times float32's 1 / 127, the
    code the integer nearest to v / scale, decided in 64 bits."""
    top = v.abs().amax(1, keepdim=True)
    scale = torch.where(top == 0, 1.0, (top * (1 / 127)).clamp(min=2.0 ** -126))
    return (v.double() / scale.double()).round().float(), scale


def _rowscale_mm(s, c):
    x = s["x"].float()
    if c["swiglu"]:
        gate, up = x.split(c["K"], 1)
        x = gate * torch.sigmoid(gate) * up
    q, scale = _row_codes(x)
    if s["rows"] is not None:
        at = (s["rows"] // s["div"]).long()
        q, scale = q[at], scale[at]
    return torch.cat([(q[a:b] @ s["wq"][e].float().t() * scale[a:b] * s["ws"][e]).to(s["y"].dtype)
                      for e, a, b in s["groups"]])


def _weights(kind, w, scales, e):
    """Experts e's matrices as float32."""
    v = w[e].float()
    if kind == "bf16":
        return v
    if kind == "int8":
        return v * scales[e].unsqueeze(2)
    _, r, k = v.shape
    full = scales[e].repeat_interleave(BLOCK, 1)[:, :r].repeat_interleave(BLOCK, 2)[:, :, :k]
    return v * full


def _ffn(kind, weights, e, x):
    """Rows x [P, d] each through its expert e [P]."""
    gu, dn, gus, dns = weights
    gate, up = torch.bmm(_weights(kind, gu, gus, e), x.unsqueeze(2)).squeeze(2).chunk(2, 1)
    h = gate * torch.sigmoid(gate) * up
    return torch.bmm(_weights(kind, dn, dns, e), h.unsqueeze(2)).squeeze(2)


def _layer_few(s, c):
    T, k, x = c["T"], c["k"], s["x"].float()
    idx, w = s["idx"], s["w"]
    if c["route"]:
        logits = s["x"].double() @ s["w_router"].double().t() + s["bias"].double()
        best, order = torch.sort(logits, dim=1, descending=True, stable=True)
        idx, w = order[:, :k].int(), torch.softmax(best[:, :k], 1).float()
    y = _ffn(c["kind"], s["experts"], idx.reshape(-1).long(), x.repeat_interleave(k, 0))
    out = (w.unsqueeze(2) * y.view(T, k, -1)).sum(1)
    if c["shared"]:
        gu, dn, gus, dns = s["shared"]
        one = torch.zeros(1, dtype=torch.long, device="cuda")
        gate, up = (x @ _weights(c["kind"], gu, gus, one)[0].t()).chunk(2, 1)
        out = out + (gate * torch.sigmoid(gate) * up) @ _weights(c["kind"], dn, dns, one)[0].t()
    return _few_out(s, c, out.to(s["out"].dtype), idx, w)


def _two_to(n):
    return ((n.int() + 127) << 23).view(torch.float32)


def _m_codes(v):
    """e4m3 codes with the smallest power of two that keeps a block within 448."""
    m, e = torch.frexp(v.abs().amax(1, keepdim=True))  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, 0, torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    return (v / _two_to(e)).to(torch.float8_e4m3fn), _two_to(e).view(-1)


def _v_codes(r):
    """8-bit codes of a second moment's root: c = 32 e + t stands for t 2^e (t up
    to 63, 32 and more where e > 0) times the smallest power of two that keeps a
    block within 4032; the nearest, ties to even, and not 0 for what is not 0."""
    m, e = torch.frexp(r.amax(1, keepdim=True))  # 4032 = 0.984375 * 2^12
    e = torch.where(m == 0, 0, torch.where(m <= 0.984375, e - 12, e - 11).clamp(min=-126))
    q = r / _two_to(e)
    top = (torch.frexp(q)[1] - 6).clamp(min=0)  # q / 2^top < 64
    code = 32 * top + torch.round(q / _two_to(top))
    return torch.where(r > 0, code.clamp(min=1), code).to(torch.uint8), _two_to(e).view(-1)


def _v_root(codes, scales):
    c = codes.int()
    e = ((c >> 5) - 1).clamp(min=0)
    return (c - 32 * e).float() * _two_to(e) * scales


def _adamw(s, c):
    q = s["flat"]
    t = s["step"].double()
    size = (LR / (1 - BETA1 ** t)).float()           # learning rate, bias of m taken out
    root = (1 / torch.sqrt(1 - BETA2 ** t)).float()  # ... of the second moment's root
    store = q["p"] if q["master"] is None else q["master"]
    g, p = s["grad"].float(), store.float()
    if s["scale"] is not None:
        g = g * s["scale"]
    m, v = q["m"], q["v"]
    if c["bits"] == 8:
        m = (m.float() * q["ms"].unsqueeze(1)).view(-1)
        v = _v_root(v, q["vs"].unsqueeze(1)).square().view(-1)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    r = torch.sqrt(v)
    p = p * (1 - LR * DECAY) - m / (r * root + EPS) * size
    store.copy_(p)
    if q["master"] is not None:
        q["p"].copy_(p)
    if c["bits"] == 32:
        q["m"].copy_(m)
        q["v"].copy_(v)
    else:
        for codes, scales, new in ((q["m"], q["ms"], _m_codes(m.view(-1, STATE_BLOCK))),
                                   (q["v"], q["vs"], _v_codes(r.view(-1, STATE_BLOCK)))):
            codes.copy_(new[0])
            scales.copy_(new[1])
    return q


# ----------------------------------------------------------------------------
# the work of a pass, and its values in 64 bits
# ----------------------------------------------------------------------------

def _hit(T, k, E, zipf):
    """Experts expected to hold rows."""
    p = [r ** -1.1 if zipf else 1.0 for r in range(1, E + 1)]
    share = [min(1.0, k * v / sum(p)) for v in p]
    return sum(1 - (1 - q) ** T for q in share)


def work(case):
    c, op = case, case["op"]
    if op == "rowscale_mm":
        P, N, K = c["T"] * c["k"], c["N"], c["K"]
        X = c["T"] if c["gather"] else P
        return dict(bytes=_hit(c["T"], c["k"], c["E"], c["zipf"]) * N * (K + 4) +
                    X * K * 2 * (2 if c["swiglu"] else 1) + P * N * SIZE[c["out"]],
                    flops=2.0 * P * N * K)
    if op == "layer_few":
        T, k, E, d, f = c["T"], c["k"], c["E"], c["d"], c["f"]
        hit = _hit(T, k, E, False) + c["shared"]
        return dict(bytes=hit * 3 * d * f * (2 if c["kind"] == "bf16" else 1) +
                    (4 * E * d if c["route"] else 0) + T * d * (2 + SIZE[c["out"]]),
                    flops=6.0 * T * (k + c["shared"]) * d * f)
    n = sum(int(v) for v in c["sizes"].split(","))
    p = {"f32": 8, "bf16": 4, "master": 10}[c["p"]]
    states = 16 if c["bits"] == 32 else 4 + 16 / STATE_BLOCK
    return dict(bytes=n * (p + SIZE[c["g"]] + states), flops=15.0 * n)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    silu = lambda z: z / (1 + torch.exp(-z))  # noqa: E731
    if c["op"] == "rowscale_mm":
        x, K = s["x"].to(f64), c["K"]
        if c["swiglu"]:
            x = silu(x[:, :K]) * x[:, K:]
        scale = torch.empty(x.shape[0], dtype=f64, device="cuda")
        codes = torch.empty_like(x)
        for i in range(0, x.shape[0], 1024):
            v = x[i:i + 1024]
            top = v.abs().max(1).values
            sc = (top.float() * (1 / 127)).to(f64)  # the scale is a float32
            sc[top == 0] = 1.0
            scale[i:i + 1024] = sc
            codes[i:i + 1024] = torch.round(v / sc[:, None])
        at = torch.arange(c["T"] * c["k"], device="cuda") if s["rows"] is None else (
            torch.div(s["rows"].long(), s["div"], rounding_mode="floor"))
        y = torch.zeros((c["T"] * c["k"], c["N"]), dtype=f64, device="cuda")
        for e, a, b in s["groups"]:
            sums = torch.matmul(codes[at[a:b]], s["wq"][e].to(f64).T)
            y[a:b] = sums * scale[at[a:b], None] * s["ws"][e].to(f64)[None, :]
        return y
    if c["op"] == "layer_few":
        x, k = s["x"].to(f64), c["k"]
        idx, w = s["idx"].long(), s["w"].to(f64)
        if c["route"]:
            logits = torch.matmul(x, s["w_router"].to(f64).T) + s["bias"].to(f64)
            w, idx = torch.topk(logits, k, dim=1)
            w = torch.exp(w - w[:, :1])
            w = w / w.sum(1, keepdim=True)

        def mat(weights, which, e):
            m, sc = weights[which][e].float().to(f64), weights[2 + which]
            if c["kind"] == "int8":
                return m * sc[e].to(f64)[:, None]
            if c["kind"] == "e4m3":
                r = torch.arange(m.shape[0], device="cuda") // BLOCK
                q = torch.arange(m.shape[1], device="cuda") // BLOCK
                return m * sc[e].to(f64)[r][:, q]
            return m

        def through(weights, e, rows):
            both = torch.matmul(rows, mat(weights, 0, e).T)
            return torch.matmul(silu(both[:, :c["f"]]) * both[:, c["f"]:], mat(weights, 1, e).T)

        out = torch.zeros_like(x)
        for e in torch.unique(idx).tolist():
            t, j = torch.nonzero(idx == e, as_tuple=True)
            out.index_add_(0, t, through(s["experts"], e, x[t]) * w[t, j][:, None])
        if c["shared"]:
            out += through(s["shared"], 0, x)
        return _few_out(s, c, out, None, w)
    q, gs = s["flat"], 1.0 if s["scale"] is None else float(s["scale"])
    b1, b2 = 1 - BETA1 ** STEP, 1 - BETA2 ** STEP
    m, v = q["m"].float().to(f64), q["v"]
    if c["bits"] == 32:
        v = v.to(f64)
    else:
        m = (m * q["ms"].to(f64)[:, None]).reshape(-1)
        high = torch.clamp(v.to(torch.int64) // 32 - 1, min=0)
        v = (((v.to(torch.int64) - 32 * high) * 2 ** high * q["vs"].to(f64)[:, None]) ** 2).reshape(-1)
    g = s["grad"].to(f64) * gs
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = (q["p"] if q["master"] is None else q["master"]).to(f64)
    p = p * (1 - LR * DECAY) - LR / b1 * m / (torch.sqrt(v / b2) + EPS)
    new = dict(p=p, master=None if q["master"] is None else p, m=m, v=v, ms=None, vs=None)
    if c["bits"] == 8:  # codes at a border may fall on either side of it
        new |= dict(m=None, v=None)
    return new
