"""Plain form, on the CPU, of 8-bit moments: codes rounded up or down by a hash of
the step's number and the element's place (or, for step None, to the nearest), in
the documented float32 operations; blocks with roots that are not finite; and what
a run of AdamW steps does with them.

The draws are two 16-bit numbers and a half each, so a code's probability is off by
2^-17 at most."""
import numpy as np

from more_ref import _blocks, adamw32, root_values

F = np.float32
U32 = np.uint32


def mix(h):
    h = np.atleast_1d(h).astype(U32)
    h = (h ^ (h >> U32(16))) * U32(0x6A09E667)
    h = (h ^ (h >> U32(15))) * U32(0x9E3779B9)
    return h ^ (h >> U32(16))


def draws(step, first, n):
    """(for m, for v) of elements first .. first + n - 1 of a tensor."""
    step = max(step, 1)
    key = mix(U32(step & 0xFFFFFFFF) + mix(U32(step >> 32)))
    i = first + np.arange(n, dtype=np.uint64)
    h = mix((i & np.uint64(0xFFFFFFFF)).astype(U32) + mix(key + (i >> np.uint64(32)).astype(U32)))
    return tuple((k.astype(F) + F(0.5)) * F(2.0 ** -16) for k in (h & U32(0xFFFF), h >> U32(16)))


def exponent(a):
    """floor(log2(a)) of float32 numbers, at least -127."""
    return (a.view(U32) >> U32(23) & U32(0xFF)).astype(np.int32) - 127


def scales(top, limit):
    """The smallest powers of two, 2^-126 at least, with top <= limit times them; 1 for 0."""
    m, e = np.frexp(top.astype(np.float64) / limit)  # top / limit = m 2^e, m in [1/2, 1)
    n = np.maximum(np.where(m == 0.5, e - 1, e), -126)
    return np.where(top == 0, 1.0, np.exp2(n)).astype(F)


def m_codes(m, step, first=0, r=None):
    """(e4m3 values, scales) of a float32 array whose first element is `first`; of
    elements whose root r is not finite only the nearest within the others' scale."""
    b = np.where(np.isfinite(m if r is None else m * F(0) + r), m, F(0))
    s = scales(np.abs(_blocks(b)).max(1), 448.0)
    # by a power of two: exact
    a = np.abs(np.where(np.isfinite(m), m, F(0))) * np.repeat(F(1) / s, 256)[:len(m)]
    a = np.minimum(a, F(448))
    place = np.exp2(np.maximum(exponent(a), -6) - 3).astype(F)
    t = a / place
    q = (np.rint(t) if step is None else np.floor(t + draws(step, first, len(m))[0])) * place
    return np.where(np.isfinite(m), np.copysign(q, m), F(np.nan)).astype(F), s


def v_codes(r, step, first=0):
    """(codes, scales) of a float32 array of roots."""
    b = np.where(np.isfinite(r), r, F(0))
    odd = ~np.isfinite(_blocks(r)).all(1)
    s = scales(_blocks(b).max(1), np.where(odd, 3968.0, 4032.0))
    a = b * np.repeat(F(1) / s, 256)[:len(r)]
    e = np.maximum(exponent(a) - 5, 0)
    t = a * np.exp2(-e).astype(F)
    low = np.floor(t)
    if step is None:
        low, up = np.rint(t), False
    else:
        up = (t - low) * (t + low) > draws(step, first, len(r))[1] * (F(2) * low + F(1))
    c = 32 * e + low.astype(np.int32) + up
    c = np.where(np.isfinite(r), np.where((r > 0) & (c == 0), 1, c), 255)
    marks = (U32(0x7FC00000) | (s.view(U32) >> U32(23))).view(F)
    return c.astype(np.uint8), np.where(odd, marks, s)


def m_of(q, s):
    return q * np.repeat(s, 256)[:len(q)]


def v_of(c, s):
    """v of codes and their blocks' scales."""
    odd, exp = np.isnan(s), s.view(U32) & U32(0xFF)
    s = np.where(odd & (exp != 0), (exp << U32(23)).view(F), s)
    r = root_values().astype(F)[c] * np.repeat(s, 256)[:len(c)]
    return np.where(np.repeat(odd, 256)[:len(c)] & (c == 255), F(np.inf), r * r)


def moments(m, r, step, first=0):
    """What the codes of m and of the root r stand for, as m and v."""
    return m_of(*m_codes(m, step, first, r)), v_of(*v_codes(r, step, first))


KINDS = ("normal", "constant", "shrinking")


def gradients(kind, steps, sizes, seed):
    """Yields a gradient a step: normal; the same each time; or normal, 20 times
    smaller after a third of the steps."""
    rng = np.random.default_rng(seed)
    signs = np.where(rng.random(len(sizes)) < 0.5, -1, 1).astype(F) * sizes
    for t in range(steps):
        g = signs if kind == "constant" else rng.standard_normal(len(sizes)).astype(F) * sizes
        yield g * F(0.05) if kind == "shrinking" and t >= steps // 3 else g


def update_ratio(kind, steps, b1, b2, sizes, encode, seed=0):
    """Norm of the updates of a run's last third with moments as `encode` holds
    them, over the norm with float32 moments."""
    z = np.zeros(len(sizes), F)
    states, norms = [(z, z), (z, z)], [0.0, 0.0]
    for t, g in enumerate(gradients(kind, steps, sizes, seed), 1):
        for i, (m, v) in enumerate(states):
            p, m, v, r = adamw32(z, g, m, v, t, 1.0, b1, b2, 1e-12, 0.0)
            if 3 * t > 2 * steps:
                norms[i] += float((p.astype(np.float64) ** 2).sum())
            states[i] = encode(m, r, t) if i else (m, v)
    return (norms[1] / norms[0]) ** 0.5
