"""Plain forms, on the CPU, of the calls on 8-bit integers, of the layer for a few
tokens and of the AdamW step: in float64, or where a call's every rounding is
documented in exactly those roundings."""
import numpy as np
import torch

from block_ref import BLOCK, d64

F64 = torch.float64
U = 2.0 ** -24  # half a step of float32


# ----------------------------------------------------------------------------
# 8-bit integers with a scale per row
# ----------------------------------------------------------------------------

def row_quantize(x):
    """(codes int64, scales float32) of [..., K], decided by exact fractions' worth
    of float64: a quotient of two float32 numbers nearer than 2^-53 to a half-way
    point is that point."""
    x = x.detach().cpu().float()
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    scale = torch.from_numpy(np.maximum(top.numpy() * np.float32(1 / 127), np.float32(2.0 ** -126)))
    scale = torch.where(top == 0, torch.ones(()), scale)
    scale[bad] = float("nan")
    q = torch.round(x.to(F64) / scale.to(F64)[..., None])  # ties to even
    return torch.where(bad[..., None], torch.zeros((), dtype=F64), q).long(), scale


def rowscale_mm(xq, xs, wq, ws, offsets, P, out, rows=None, div=1):
    """Every rounding as documented: the exact sum to float32, times each scale in
    float32, to out; positions of no group are 0."""
    xq, wq, xs, ws = (t.detach().cpu() for t in (xq, wq, xs, ws))
    src = torch.arange(P) if rows is None else rows.cpu().long()
    ok = (src >= 0) & (src < xq.shape[0] * div)
    src = torch.where(ok, src, 0) // div
    y = torch.zeros((P, wq.shape[1]), dtype=torch.float32)
    o = offsets.cpu().tolist()
    for e, (a, b) in enumerate(zip(o, o[1:])):
        if b > a:
            rows_e = xq[src[a:b]].to(F64) * ok[a:b, None]
            sums = (rows_e @ wq[e].to(F64).T).to(torch.float32)  # below 2^53: exact, then once
            s = torch.where(ok[a:b], xs[src[a:b]], torch.zeros(()))
            y[a:b] = sums * s[:, None] * ws[e][None, :]
    return y.to(out)


# ----------------------------------------------------------------------------
# the layer for a few tokens
# ----------------------------------------------------------------------------

def matrix(w, scales):
    """Float64 values [n, R, K] of an expert matrix in any of its forms."""
    w = w.detach().cpu()
    if w.dtype == torch.bfloat16:
        return w.to(F64)
    if w.dtype == torch.int8:
        return w.to(F64) * d64(scales)[:, :, None]
    v = w.view(torch.float8_e4m3fn).float().to(F64)
    s = d64(scales).repeat_interleave(BLOCK, 1)[:, :v.shape[1]]
    return v * s.repeat_interleave(BLOCK, 2)[:, :, :v.shape[2]]


def layer_few(x, idx, w, experts, shared, out):
    """(out, allowance): the layer in float64, and how far sums in float32, scales
    applied in float32, h with 16 significant bits and the last rounding may take
    the call from it."""
    x, idx, w = d64(x), idx.cpu().long(), d64(w)
    T, d = x.shape

    def ffn(weights, e, rows):
        gu, dn, gus, dns = weights if len(weights) == 4 else (*weights, None, None)
        both = matrix(gu[e:e + 1], None if gus is None else gus[e:e + 1])[0]
        down = matrix(dn[e:e + 1], None if dns is None else dns[e:e + 1])[0]
        f = both.shape[0] // 2
        v, mag = rows @ both.T, rows.abs() @ both.abs().T
        # d products added up (2^-23 each, an adder that truncates included), and
        # the scales: one or two float32 products, of a pair first for e4m3
        err = (d + 4) * 2 * U * mag
        g, u, eg, eu = v[:, :f], v[:, f:], err[:, :f], err[:, f:]
        s = 1 / (1 + torch.exp(-g))
        h = g * s * u
        # |silu'| < 1.1; exp, sum, quotient and product a few roundings; 2^-17 the split
        eh = 1.1 * u.abs() * eg + (g * s).abs() * eu + 1.1 * eg * eu + h.abs() * (8 * U + 2.0 ** -17)
        y, ymag = h @ down.T, (h.abs() + eh) @ down.abs().T
        return y, eh @ down.abs().T + (2 * f + 4) * 2 * U * ymag

    y, err, mag = torch.zeros((T, d), dtype=F64), torch.zeros((T, d), dtype=F64), 0.0
    for t in range(T):
        for j, e in enumerate(idx[t].tolist()):
            if 0 <= e < experts[0].shape[0]:
                v, ev = ffn(experts, e, x[t:t + 1])
                y[t] += w[t, j] * v[0]
                err[t] += w[t, j].abs() * (ev[0] + 2 * (idx.shape[1] + 2) * U * v[0].abs())
    if shared is not None:
        v, ev = ffn(shared, 0, x)
        y, err = y + v, err + ev + 4 * U * v.abs()
    half = torch.finfo(out).eps / 2
    return y, err + half * (y.abs() + err)


# ----------------------------------------------------------------------------
# AdamW
# ----------------------------------------------------------------------------

STATE_BLOCK = 256


def adamw64(p, g, m, v, step, lr, b1, b2, eps, decay, gs=1.0):
    """(p, m, v) in float64."""
    g = g * gs
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = torch.sqrt(v) / (1 - b2 ** step) ** 0.5 + eps
    return p * (1 - lr * decay) - lr / (1 - b1 ** step) * (m / den), m, v


def adamw32(p, g, m, v, step, lr, b1, b2, eps, decay, gs=None):
    """(p, m, v, sqrt(v)) with every operation rounded to float32, as documented."""
    f = np.float32
    g = g * f(1 if gs is None else gs)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + g * g * f(1 - b2)
    size, root = f(lr / (1 - b1 ** step)), f(1 / np.sqrt(1 - b2 ** step))
    r = np.sqrt(v)
    assert r.dtype == g.dtype == np.float32
    return p * f(1 - lr * decay) - m / (r * root + f(eps)) * size, m, v, r


def root_values():
    """What the 256 codes of sqrt(v) stand for."""
    return np.array([(c - 32 * max(c // 32 - 1, 0)) * 2.0 ** max(c // 32 - 1, 0) for c in range(256)])


def _blocks(a):
    return np.pad(a, (0, -len(a) % STATE_BLOCK)).reshape(-1, STATE_BLOCK)


def _scales(top, limit):
    n = np.full(len(top), -126)
    for i, t in enumerate(top):
        while t > limit * 2.0 ** n[i]:
            n[i] += 1
    return np.where(top == 0, 1.0, 2.0 ** n)


def _nearest(values, a):
    """Index of the nearest of the ascending values, ties to the even index."""
    hi = np.clip(np.searchsorted(values, a), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = a - values[lo], values[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def m_codes(m):
    """(e4m3 values float64, scales) of a float32 array, by search."""
    from block_ref import e4m3_values
    b = _blocks(m.astype(np.float64))
    s = _scales(np.abs(b).max(1), 448.0)
    t = e4m3_values().numpy()
    q = t[_nearest(t, np.abs(b / s[:, None]))] * np.sign(b)
    return q.reshape(-1)[:len(m)], s.astype(np.float32)


def v_codes(r):
    """(codes, scales) of a float32 array of roots, by search."""
    b = _blocks(r.astype(np.float64))
    s = _scales(b.max(1), 4032.0)
    c = _nearest(root_values(), b / s[:, None])
    c = np.where((b > 0) & (c == 0), 1, c)
    return c.reshape(-1)[:len(r)].astype(np.uint8), s.astype(np.float32)
