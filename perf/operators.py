"""Timed cases of the operators on float (bfloat16) and 8-bit expert weights.

  grouped_mm      y[p] = W_e x[row(p)] over rows grouped by expert, its input
                  gradient and its weight gradient
  blockscale_mm   the same product over e4m3 codes: one float32 scale per 128
                  columns of an activation row (quantised within the pass) and
                  per 128 x 128 weights
  swiglu          h = silu(gate) * up over grouped rows, and its gradient
  block_norm      r = res + scale * gate * norm(y), n = norm(r), and the gradient
  combine_grad    gradient of the gate-weighted combine of a token's experts

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
EPS = 1e-6
BLOCK = 128


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one token's gate and up products in the ~19 MB-expert layer: 8 experts
        # of 256, one row each; the weights of those 8 are all there is to read
        dict(name="mm_step_1", op="grouped_mm", way="forward", T=1, k=8, E=256, N=4096, K=6144,
             zipf=False, gather=True, out="f32"),
        # the same layer over a 2048-token prompt with skewed routing: some experts
        # take over a thousand rows, the median about ten
        dict(name="mm_prompt_2048", op="grouped_mm", way="forward", T=2048, k=8, E=256, N=4096,
             K=6144, zipf=True, gather=True, out="bf16"),
        # training the 64-expert layer on 4096 tokens: gradient of the gate and up
        # products' input
        dict(name="mm_input_grad_4096", op="grouped_mm", way="input_grad", T=4096, k=8, E=64,
             N=2048, K=2048, zipf=False, gather=False, out="bf16"),
        # ... and of the down product's weights, uneven groups
        dict(name="mm_weight_grad_4096", op="grouped_mm", way="weight_grad", T=4096, k=8, E=64,
             N=2048, K=1024, zipf=True, gather=False, out="f32"),
        # an 8-token step over 8-bit experts: the activations are quantised, then
        # about 57 experts' codes are read
        dict(name="blockscale_step_8", op="blockscale_mm", T=8, k=8, E=256, N=4096, K=6144,
             zipf=False, gather=True, out="f32"),
        dict(name="blockscale_prompt_2048", op="blockscale_mm", T=2048, k=8, E=256, N=4096, K=6144,
             zipf=True, gather=True, out="bf16"),
        # activation of the 2048-token prompt's 16,384 rows
        dict(name="swiglu_prompt_2048", op="swiglu", way="forward", P=16384, f=2048, dt="bf16"),
        # its gradient in the 64-expert layer's training step, a ragged batch
        dict(name="swiglu_grad_4093", op="swiglu", way="grad", P=8 * 4093, f=1024, dt="bf16"),
        # one token between two layers: post norm, residual, the next pre norm
        dict(name="norm_step_1", op="block_norm", way="forward", T=1, d=6144, y="f32", res="bf16",
             out="bf16", post=True, pre=True, gate="channel"),
        # the same pair's gradient over a 2048-token batch
        dict(name="norm_grad_2048", op="block_norm", way="grad", T=2048, d=6144, y="bf16",
             res="bf16", out="bf16", post=True, pre=True, gate="channel"),
        # combine's gradient: a few tokens, and a 2048-token batch
        dict(name="combine_grad_33", op="combine_grad", T=33, k=8, d=2048, y="f32", out="f32"),
        dict(name="combine_grad_2048", op="combine_grad", T=2048, k=8, d=6144, y="bf16",
             out="bf16"),
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(high, max(low, step * round(v / step))))


def draw(rng):
    op = rng.choice(["grouped_mm", "grouped_mm", "grouped_mm", "blockscale_mm", "blockscale_mm",
                     "swiglu", "block_norm", "block_norm", "combine_grad"])
    if op in ("grouped_mm", "blockscale_mm"):
        while True:
            E = _log(rng, 1, 256)
            c = dict(op=op, T=_log(rng, 1, 4096), k=min(E, rng.randint(1, 8)), E=E,
                     N=_log(rng, 64, 6144, 8), K=_log(rng, 64, 6144, 16),
                     zipf=rng.random() < 0.5, gather=rng.random() < 0.5,
                     out=rng.choice(["bf16", "f32"]))
            if op == "grouped_mm":
                c["way"] = rng.choice(["forward", "input_grad", "weight_grad"])
                c["gather"] = c["gather"] and c["way"] != "input_grad"
            # no dearer than the largest listed case: weights and products
            if E * c["N"] * c["K"] <= 1.6e9 and c["T"] * c["k"] * c["N"] * c["K"] <= 2e11:
                return c
    if op == "swiglu":
        while True:
            c = dict(op=op, way=rng.choice(["forward", "grad"]), P=_log(rng, 1, 32768),
                     f=_log(rng, 64, 8192, 8), dt=rng.choice(["bf16", "f32"]))
            if c["P"] * c["f"] <= 3.3e7:
                return c
    if op == "block_norm":
        c = dict(op=op, way=rng.choice(["forward", "grad"]), T=_log(rng, 1, 2048),
                 d=_log(rng, 64, 6144, 8), y=rng.choice(["bf16", "f32"]),
                 res=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                 post=rng.random() < 0.7, pre=rng.random() < 0.7,
                 gate=rng.choice(["none", "channel", "token"]))
        return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 8), d=_log(rng, 64, 8192, 64),
                 y=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
        if c["T"] * c["k"] * c["d"] <= 1e8:
            return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _route(g, T, k, E, zipf):
    """Distinct experts of every token, popular ones first drawn where `zipf`:
    the grouping (offsets, slot at each grouped position and its inverse)."""
    logp = torch.zeros(E, device="cuda")
    if zipf:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logp = -1.1 * torch.log(rank.float())
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    idx = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    return offsets.int(), perm.int(), inv.int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dt=torch.bfloat16, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(scale)

    s = dict(case=c)
    if c["op"] in ("grouped_mm", "blockscale_mm"):
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        P = T * k
        offsets, perm, _ = _route(g, T, k, E, c["zipf"])
        s |= dict(offsets=offsets, rows=perm if c["gather"] else None, div=k if c["gather"] else 1)
        ends = offsets.tolist()  # the plain form's plan: the groups that hold rows
        s["groups"] = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
        out, X = DTYPES[c["out"]], T if c["gather"] else P
        if c["op"] == "blockscale_mm":
            s["x"] = normal(X, K)
            s["wq"] = normal(E, N, K, scale=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s["ws"] = 1e-4 + 3e-4 * torch.rand((E, -(-N // BLOCK), -(-K // BLOCK)), generator=g,
                                               device="cuda")
            s["xq"] = torch.empty((X, K), dtype=torch.float8_e4m3fn, device="cuda")
            s["xs"] = torch.empty((X, -(-K // BLOCK)), device="cuda")
            s["y"] = torch.empty((P, N), dtype=out, device="cuda")
        elif c["way"] == "forward":
            s |= dict(x=normal(X, K), w=normal(E, N, K, scale=0.02),
                      y=torch.empty((P, N), dtype=out, device="cuda"))
        elif c["way"] == "input_grad":
            s |= dict(dy=normal(P, N, scale=1e-2), w=normal(E, N, K, scale=0.02),
                      dx=torch.empty((P, K), dtype=out, device="cuda"))
        else:
            s |= dict(dy=normal(P, N, scale=1e-2), x=normal(X, K),
                      dw=torch.empty((E, N, K), dtype=out, device="cuda"))
    elif c["op"] == "swiglu":
        dt = DTYPES[c["dt"]]
        s["gu"] = normal(c["P"], 2 * c["f"], dt=dt, scale=1.5)
        if c["way"] == "forward":
            s["h"] = torch.empty((c["P"], c["f"]), dtype=dt, device="cuda")
        else:
            s["dh"] = normal(c["P"], c["f"], dt=dt, scale=1e-2)
            s["dgu"] = torch.empty_like(s["gu"])
    elif c["op"] == "block_norm":
        T, d = c["T"], c["d"]
        ydt, rdt, ndt = DTYPES[c["y"]], DTYPES[c["res"]], DTYPES[c["out"]]
        f32 = torch.float32
        s |= dict(y=normal(T, d, dt=ydt, scale=0.7), res=normal(T, d, dt=rdt),
                  w_post=1 + normal(d, dt=f32, scale=0.1) if c["post"] else None,
                  w_pre=1 + normal(d, dt=f32, scale=0.1) if c["pre"] else None,
                  gate=None if c["gate"] == "none" else
                  normal(1 if c["gate"] == "channel" else T, d, dt=ydt), scale=0.5)
        new = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
        if c["way"] == "forward":
            s |= dict(r=new(s["res"]),
                      n=torch.empty((T, d), dtype=ndt, device="cuda") if c["pre"] else None)
        else:
            s |= dict(dr=normal(T, d, dt=rdt, scale=1e-2),
                      dn=normal(T, d, dt=ndt, scale=1e-2) if c["pre"] else None,
                      dy=new(s["y"]), dres=new(s["res"]), dw_post=new(s["w_post"]),
                      dw_pre=new(s["w_pre"]), dgate=new(s["gate"]))
    else:
        T, k, d = c["T"], c["k"], c["d"]
        _, _, inv = _route(g, T, k, 64, True)
        s |= dict(shape=(d, 64, 64, k, 64, 0), inv=inv, w=torch.softmax(normal(T, k, dt=torch.float32), 1),
                  dout=normal(T, d, dt=DTYPES[c["out"]], scale=1e-2),
                  y=normal(T * k, d, dt=DTYPES[c["y"]]))
        s |= dict(dy=torch.empty_like(s["y"]), dw=torch.empty_like(s["w"]))
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"grouped_mm": _mm, "blockscale_mm": _blockscale_mm, "swiglu": _swiglu,
            "block_norm": _block_norm, "combine_grad": _combine_grad}[c["op"]](s, c)


def _run_own(s, c):
    import int4_routed_expert_logits_amd as moe
    op, way = c["op"], c.get("way")
    if op == "grouped_mm":
        if way == "forward":
            moe.moe_grouped_mm(s["x"], s["w"], s["offsets"], s["y"], s["rows"], s["div"])
            return s["y"]
        if way == "input_grad":
            moe.moe_grouped_mm_dx(s["dy"], s["w"], s["offsets"], s["dx"])
            return s["dx"]
        ws = _scratch(moe.moe_grouped_mm_dw_workspace_bytes(c["E"], c["T"] * c["k"], c["N"],
                                                            c["K"]))
        moe.moe_grouped_mm_dw(s["dy"], s["x"], s["offsets"], s["dw"], ws, s["rows"], s["div"])
        return s["dw"]
    if op == "blockscale_mm":
        moe.moe_blockscale_quantize(s["x"], 1, s["xq"], s["xs"])
        moe.moe_blockscale_mm(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], s["y"], s["rows"],
                              s["div"])
        return s["y"]
    if op == "swiglu":
        if way == "forward":
            moe.moe_swiglu(s["gu"], s["h"])
            return s["h"]
        moe.moe_swiglu_grad(s["gu"], s["dh"], s["dgu"])
        return s["dgu"]
    if op == "block_norm":
        if way == "forward":
            moe.moe_block_norm(s["y"], s["res"], s["r"], s["n"], s["w_post"], s["w_pre"], s["gate"],
                               s["scale"], EPS)
            return dict(r=s["r"], n=s["n"])
        ws = _scratch(moe.moe_block_norm_grad_workspace_bytes(c["T"], c["d"]))
        moe.moe_block_norm_grad(s["y"], s["res"], s["dr"], s["dn"], s["dy"], s["dres"],
                                s["dw_post"], s["dw_pre"], s["dgate"], s["w_post"], s["w_pre"],
                                s["gate"], s["scale"], EPS, ws)
        return dict(dy=s["dy"], dres=s["dres"], dw_post=s["dw_post"], dw_pre=s["dw_pre"],
                    dgate=s["dgate"])
    moe.moe_combine_grad(s["shape"], s["dout"], s["y"], s["inv"], s["w"], s["dy"], s["dw"])
    return dict(dy=s["dy"], dw=s["dw"])


def _scratch(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


def _rows(s, a, b):
    """Input rows of grouped positions a .. b."""
    x = s["x"]
    return (x[a:b] if s["rows"] is None else x[(s["rows"][a:b] // s["div"]).long()]).float()


def _mm(s, c):
    """One float32 product per group that holds rows."""
    if c["way"] == "forward":
        y = torch.empty_like(s["y"])
        for e, a, b in s["groups"]:
            y[a:b] = _rows(s, a, b) @ s["w"][e].float().t()
        return y
    if c["way"] == "input_grad":
        dx = torch.empty_like(s["dx"])
        for e, a, b in s["groups"]:
            dx[a:b] = s["dy"][a:b].float() @ s["w"][e].float()
        return dx
    dw = torch.zeros_like(s["dw"])
    for e, a, b in s["groups"]:
        dw[e] = s["dy"][a:b].float().t() @ _rows(s, a, b)
    return dw


def _quantised(x):
    """x's e4m3 values with a power-of-two scale per 128 columns, the smallest
    that keeps the largest magnitude within 448, as float32."""
    R, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(R, -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(2, keepdim=True))  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, 0, torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    scale = ((e.int() + 127) << 23).view(torch.float32)  # 2^e
    return ((v / scale).to(torch.float8_e4m3fn).float() * scale).view(R, -1)[:, :K]


def _blockscale_mm(s, c):
    x = _quantised(s["x"])
    if s["rows"] is not None:
        x = x[(s["rows"] // s["div"]).long()]
    y = torch.empty_like(s["y"])
    N, K = c["N"], c["K"]
    for e, a, b in s["groups"]:
        w = torch.nn.functional.pad(s["wq"][e].float(), (0, -K % BLOCK, 0, -N % BLOCK))
        w.view(-(-N // BLOCK), BLOCK, -1, BLOCK).mul_(s["ws"][e][:, None, :, None])
        y[a:b] = x[a:b] @ w[:N, :K].t()
    return y


def _swiglu(s, c):
    g, u = s["gu"].float().split(c["f"], 1)
    sig = torch.sigmoid(g)
    if c["way"] == "forward":
        return (g * sig * u).to(s["h"].dtype)
    dh = s["dh"].float()
    return torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1).to(s["dgu"].dtype)


def _block_norm(s, c):
    y, gate = s["y"].float(), 1.0 if s["gate"] is None else s["gate"].float()
    one = torch.ones(c["d"], device=y.device)
    w1, w2 = one if s["w_post"] is None else s["w_post"], one if s["w_pre"] is None else s["w_pre"]
    a = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) if c["post"] else torch.ones_like(y[:, :1])
    yh = y * a
    r = s["res"].float() + s["scale"] * gate * (w1 * yh)
    b = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    if c["way"] == "forward":
        return dict(r=r.to(s["r"].dtype), n=(w2 * (r * b)).to(s["n"].dtype) if c["pre"] else None)
    dr, dw2 = s["dr"].float(), None
    if c["pre"]:
        dn, rh = s["dn"].float(), r * b
        v = w2 * dn
        dr = dr + b * (v - rh * (v * rh).mean(1, keepdim=True))
        dw2 = (dn * rh).sum(0)
    dp = s["scale"] * gate * dr
    v = w1 * dp
    dy = a * (v - yh * (v * yh).mean(1, keepdim=True)) if c["post"] else dp
    dgate = None
    if s["gate"] is not None:
        dgate = s["scale"] * dr * (w1 * yh)
        dgate = (dgate.sum(0, keepdim=True) if c["gate"] == "channel" else dgate).to(s["gate"].dtype)
    return dict(dy=dy.to(s["y"].dtype), dres=dr.to(s["res"].dtype),
                dw_post=(dp * yh).sum(0) if c["post"] else None, dw_pre=dw2, dgate=dgate)


def _combine_grad(s, c):
    T, k = c["T"], c["k"]
    dout, inv = s["dout"].float(), s["inv"].long()
    dy = torch.empty_like(s["y"])
    dy[inv] = (s["w"].unsqueeze(2) * dout.unsqueeze(1)).view(T * k, -1).to(dy.dtype)
    dw = (s["y"][inv].float().view(T, k, -1) * dout.unsqueeze(1)).sum(2)
    return dict(dy=dy, dw=dw)


# ----------------------------------------------------------------------------
# the work of a pass, and its values in 64 bits
# ----------------------------------------------------------------------------

def _groups_hit(c):
    """Experts expected to hold rows."""
    p = [r ** -1.1 if c["zipf"] else 1.0 for r in range(1, c["E"] + 1)]
    share = [min(1.0, c["k"] * v / sum(p)) for v in p]
    return sum(1 - (1 - q) ** c["T"] for q in share)


def work(case):
    c, op = case, case["op"]
    if op in ("grouped_mm", "blockscale_mm"):
        P, N, K = c["T"] * c["k"], c["N"], c["K"]
        X = c["T"] if c["gather"] else P
        hit, flops = _groups_hit(c), 2.0 * P * N * K
        if op == "blockscale_mm":
            return dict(bytes=hit * N * K + X * K * 2 + P * N * SIZE[c["out"]], flops=flops)
        if c["way"] == "forward":
            return dict(bytes=hit * N * K * 2 + X * K * 2 + P * N * SIZE[c["out"]], flops=flops)
        if c["way"] == "input_grad":
            return dict(bytes=hit * N * K * 2 + P * N * 2 + P * K * SIZE[c["out"]], flops=flops)
        return dict(bytes=P * N * 2 + X * K * 2 + c["E"] * N * K * SIZE[c["out"]], flops=flops)
    if op == "swiglu":
        n = c["P"] * c["f"]
        return dict(bytes=n * SIZE[c["dt"]] * (3 if c["way"] == "forward" else 5), flops=8.0 * n)
    if op == "block_norm":
        n, sy, sr, sn = c["T"] * c["d"], SIZE[c["y"]], SIZE[c["res"]], SIZE[c["out"]] * c["pre"]
        gate = {"none": 0, "channel": c["d"], "token": n}[c["gate"]] * sy
        vectors = 4 * c["d"] * (c["post"] + c["pre"])
        if c["way"] == "forward":
            return dict(bytes=n * (sy + 2 * sr + sn) + gate + vectors, flops=10.0 * n)
        return dict(bytes=n * (2 * sy + 3 * sr + sn) + 2 * gate + 2 * vectors, flops=30.0 * n)
    n = c["T"] * c["d"]
    return dict(bytes=n * SIZE[c["out"]] + 2 * n * c["k"] * SIZE[c["y"]], flops=3.0 * n * c["k"])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    two_to = lambda n: ((n + 1023) << 52).view(f64)  # noqa: E731
    if c["op"] in ("grouped_mm", "blockscale_mm"):
        ends = [(a, b) for _, a, b in s["groups"]]
        ids = [e for e, _, _ in s["groups"]]
        at = torch.arange(c["T"] * c["k"], device="cuda") if s["rows"] is None else (
            torch.div(s["rows"].long(), s["div"], rounding_mode="floor"))
        if c["op"] == "blockscale_mm":
            x = s["x"].to(f64)
            xq = torch.empty_like(x)
            for k0 in range(0, c["K"], BLOCK):
                v = x[:, k0:k0 + BLOCK]
                top = v.abs().max(1, keepdim=True).values
                # the smallest 2^n with top <= 448 * 2^n (1 for a block of zeros)
                n = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).long()
                n = torch.where(top > 448 * two_to(n), n + 1, n)
                n = torch.where(top <= 448 * two_to(n - 1), n - 1, n).clamp(min=-126)
                n = torch.where(top == 0, torch.zeros_like(n), n)
                q = v / two_to(n)
                # e4m3: steps of 2^(exponent - 3), exponents from -6; half steps to even
                _, up = torch.frexp(q.abs().clamp(min=2.0 ** -6))  # exponent + 1
                step = two_to(up.long() - 4)
                xq[:, k0:k0 + BLOCK] = torch.round(q / step) * step * two_to(n)
            y = torch.zeros((c["T"] * c["k"], c["N"]), dtype=f64, device="cuda")
            rows = torch.arange(c["N"], device="cuda") // BLOCK
            cols = torch.arange(c["K"], device="cuda") // BLOCK
            for e, (a, b) in zip(ids, ends):
                w = s["wq"][e].to(torch.float32).to(f64) * s["ws"][e].to(f64)[rows][:, cols]
                y[a:b] = torch.matmul(xq[at[a:b]], w.T)
            return y
        if c["way"] == "weight_grad":
            dw = torch.zeros((c["E"], c["N"], c["K"]), dtype=f64, device="cuda")
            for e, (a, b) in zip(ids, ends):
                torch.matmul(s["dy"][a:b].to(f64).T, s["x"][at[a:b]].to(f64), out=dw[e])
            return dw
        src, back = (s["x"], False) if c["way"] == "forward" else (s["dy"], True)
        y = torch.zeros((c["T"] * c["k"], c["K"] if back else c["N"]), dtype=f64, device="cuda")
        for e, (a, b) in zip(ids, ends):
            w = s["w"][e].to(f64)
            y[a:b] = torch.matmul(src[at[a:b]].to(f64), w if back else w.T)
        return y
    if c["op"] == "swiglu":
        g, u = s["gu"][:, :c["f"]].to(f64), s["gu"][:, c["f"]:].to(f64)
        den = 1 + torch.exp(-g)
        if c["way"] == "forward":
            return g / den * u
        dh = s["dh"].to(f64)
        slope = (den + g * torch.exp(-g)) / den ** 2  # d/dg of g / (1 + e^-g)
        return torch.cat([dh * u * slope, dh * g / den], 1)
    if c["op"] == "block_norm":
        d = c["d"]
        up = lambda v, n: (torch.ones((1, n), dtype=f64, device="cuda")  # noqa: E731
                           if v is None else v.to(f64).reshape(-1, n))
        y, res, w1, w2, gate = s["y"].to(f64), s["res"].to(f64), up(s["w_post"], d), up(
            s["w_pre"], d), up(s["gate"], d)
        ay = 1 / torch.sqrt(y.square().sum(1, keepdim=True) / d + EPS)
        if not c["post"]:
            ay = torch.ones_like(ay)
        p = y * ay * w1
        r = res + gate * p * s["scale"]
        ar = 1 / torch.sqrt(r.square().sum(1, keepdim=True) / d + EPS)
        if c["way"] == "forward":
            return dict(r=r, n=r * ar * w2 if c["pre"] else None)
        t = s["dr"].to(f64)  # the whole gradient of r
        if c["pre"]:
            dn = s["dn"].to(f64)
            t = t + ar * w2 * dn - r * ar ** 3 * (w2 * dn * r).sum(1, keepdim=True) / d
        dp = t * gate * s["scale"]
        dy = dp
        if c["post"]:
            dy = ay * w1 * dp - y * ay ** 3 * (w1 * dp * y).sum(1, keepdim=True) / d
        dgate = t * p * s["scale"]
        return dict(dy=dy, dres=t, dw_post=(dp * y * ay).sum(0) if c["post"] else None,
                    dw_pre=(s["dn"].to(f64) * r * ar).sum(0) if c["pre"] else None,
                    dgate=None if c["gate"] == "none" else
                    dgate.sum(0, keepdim=True) if c["gate"] == "channel" else dgate)
    T, k = c["T"], c["k"]
    at = s["inv"].long().view(T, k)
    dout, y = s["dout"].to(f64), s["y"].to(f64)
    dy, dw = torch.zeros_like(y), torch.zeros((T, k), dtype=f64, device="cuda")
    for j in range(k):
        dy[at[:, j]] = s["w"][:, j:j + 1].to(f64) * dout
        dw[:, j] = (y[at[:, j]] * dout).sum(1)
    return dict(dy=dy, dw=dw)
