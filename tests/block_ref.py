"""Plain float64 forms, on the CPU, of the calls in include/moe_int4_block.h,
and the rounding allowances their tests use."""
import torch

F64 = torch.float64
BLOCK = 128


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def d64(t):
    return t.detach().cpu().to(F64)


def groups(offsets):
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def source(x, rows, div):
    """x by grouped position; rows out of range are zero."""
    if rows is None:
        return x
    rows = rows.cpu().long()
    ok = (rows >= 0) & (rows < x.shape[0] * div)
    src = torch.where(ok, rows, 0) // div
    return x[src] * ok[:, None].to(x.dtype)


def grouped_mm(x, w, offsets, P, rows=None, div=1):
    """(y, sum of the products' magnitudes) [P, N]; positions of no group are 0."""
    x, w = source(d64(x), rows, div), d64(w)
    y = torch.zeros((P, w.shape[1]), dtype=F64)
    mag = torch.zeros_like(y)
    for e, a, b in groups(offsets):
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = x[a:b].abs() @ w[e].abs().T
    return y, mag


def grouped_mm_dx(dy, w, offsets):
    return grouped_mm(dy, d64(w).transpose(1, 2), offsets, dy.shape[0])


def grouped_mm_dw(dy, x, offsets, E, rows=None, div=1):
    dy, x = d64(dy), source(d64(x), rows, div)
    dw = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=F64)
    mag = torch.zeros_like(dw)
    for e, a, b in groups(offsets):
        dw[e] = dy[a:b].T @ x[a:b]
        mag[e] = dy[a:b].abs().T @ x[a:b].abs()
    return dw, mag


def e4m3_values():
    """The finite non-negative e4m3 values: (1 + m / 8) 2^(e - 7), m / 8 2^-6."""
    return torch.tensor([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=F64)


def e4m3_round(v):
    """Nearest e4m3 value, ties to the even code, by search over all values."""
    t = e4m3_values()
    a = v.abs().reshape(-1)
    hi = torch.searchsorted(t, a).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - t[lo], t[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (t[pick].reshape(v.shape)) * torch.where(v < 0, -1.0, 1.0).to(F64)


def quantize(x, block_rows):
    """(values of the codes, scales) of [n, R, K] or [R, K]."""
    x = d64(x)
    flat = x.reshape(-1, x.shape[-2], x.shape[-1])
    n, R, K = flat.shape
    br = 1 if block_rows == 1 else BLOCK
    sr, sk = -(-R // br), -(-K // BLOCK)
    values, scales = torch.zeros_like(flat), torch.ones((n, sr, sk), dtype=F64)
    for i in range(n):
        for r in range(sr):
            for k in range(sk):
                v = flat[i, r * br:(r + 1) * br, k * BLOCK:(k + 1) * BLOCK]
                ok = torch.isfinite(v)
                top = float(torch.where(ok, v.abs(), 0.0).max())
                e = -126 if top else 0
                while top > 448 * 2.0 ** e:
                    e += 1
                q = e4m3_round(torch.where(ok, v, 0.0) / 2.0 ** e)
                values[i, r * br:(r + 1) * br, k * BLOCK:(k + 1) * BLOCK] = torch.where(
                    ok, q, float("nan"))
                scales[i, r, k] = 2.0 ** e
    lead = x.shape[:-2]
    return values.reshape(x.shape), scales.reshape(*lead, sr, sk)


def dequantize(codes, scales, block_rows):
    """float64 values of e4m3 codes and their block scales."""
    v = codes.cpu().view(torch.float8_e4m3fn).float().to(F64)
    s = d64(scales).repeat_interleave(BLOCK, -1)[..., :v.shape[-1]]
    if block_rows != 1:
        s = s.repeat_interleave(BLOCK, -2)[..., :v.shape[-2], :]
    return v * s


def swiglu(gu):
    g, u = d64(gu).chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def swiglu_grad(gu, dh):
    g, u = d64(gu).chunk(2, 1)
    dh = d64(dh)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)


def block_norm(y, res, w_post, w_pre, gate, scale, eps):
    """Any tensor may be None: (r, n)."""
    p = 0.0
    if y is not None:
        p = y if w_post is None else y * w_post / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        p = scale * (p if gate is None else gate * p)
    r = p if res is None else res + p
    n = None if w_pre is None else r * w_pre / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    return r, n


def block_norm_grad(y, res, w_post, w_pre, gate, scale, eps, dr, dn):
    """The gradient by its formula: dict of dy, dres, dgate, dw_post, dw_pre."""
    r, _ = block_norm(y, res, w_post, w_pre, gate, scale, eps)
    d = r.shape[1]
    t = torch.zeros_like(r) if dr is None else dr.clone()
    out = dict(dy=None, dgate=None, dw_post=None, dw_pre=None)
    if w_pre is not None:
        b = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
        v = w_pre * dn
        t = t + b * v - r * b ** 3 * (v * r).sum(1, keepdim=True) / d
        out["dw_pre"] = (dn * r * b).sum(0)
    out["dres"] = t
    if y is not None:
        g = torch.ones((1, d), dtype=F64) if gate is None else gate
        w = torch.ones(d, dtype=F64) if w_post is None else w_post
        a = torch.ones((y.shape[0], 1), dtype=F64)
        if w_post is not None:
            a = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        dp = scale * g * t
        out["dw_post"] = None if w_post is None else (dp * y * a).sum(0)
        dg = scale * t * w * y * a
        out["dgate"] = None if gate is None else (dg if g.shape[0] == y.shape[0] else
                                                  dg.sum(0, keepdim=True))
        v = w * dp
        out["dy"] = v if w_post is None else a * v - y * a ** 3 * (v * y).sum(1, keepdim=True) / d
    return out


def combine_grad(dout, y, inv, w):
    """(dy, dw, sum of the dot products' magnitudes); rows of dy no slot has are NaN."""
    dout, y, w = d64(dout), d64(y), d64(w)
    T, k = w.shape
    dy, dw = torch.full_like(y, float("nan")), torch.zeros_like(w)
    mag = torch.zeros_like(w)
    for s, p in enumerate(inv.cpu().tolist()):
        if 0 <= p < T * k:
            t, j = divmod(s, k)
            dy[p] = w[t, j] * dout[t]
            dw[t, j] = (y[p] * dout[t]).sum()
            mag[t, j] = (y[p] * dout[t]).abs().sum()
    return dy, dw, mag
