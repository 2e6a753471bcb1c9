"""Plain form, on the CPU, of the 8-bit moments of slow betas: codes rounded up or
down by a hash of the step's number and the element's place, in the documented
float32 operations; and what a run of AdamW steps does with them.

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


def m_codes(m, step, first=0):
    """(e4m3 values, scales) of a float32 array whose first element is `first`."""
    b = _blocks(m)
    s = scales(np.abs(b).max(1), 448.0)
    a = (np.abs(b) * (F(1) / s)[:, None]).reshape(-1)[:len(m)]  # a power of two: exact
    place = np.exp2(np.maximum(exponent(a), -6) - 3).astype(F)
    q = np.floor(a / place + draws(step, first, len(m))[0]) * place
    return np.copysign(q, m).astype(F), s


def v_codes(r, step, first=0):
    """(codes, scales) of a float32 array of roots."""
    b = _blocks(r)
    s = scales(b.max(1), 4032.0)
    a = (b * (F(1) / s)[:, None]).reshape(-1)[:len(r)]
    e = np.maximum(exponent(a) - 5, 0)
    t = a * np.exp2(-e).astype(F)
    low = np.floor(t)
    up = (t - low) * (t + low) > draws(step, first, len(r))[1] * (F(2) * low + F(1))
    c = 32 * e + low.astype(np.int32) + up
    return np.where((r > 0) & (c == 0), 1, c).astype(np.uint8), s


def moments(m, r, step, first=0):
    """What the codes of m and of the root r stand for, as m and v."""
    q, s = m_codes(m, step, first)
    c, z = v_codes(r, step, first)
    z = root_values().astype(F)[c] * np.repeat(z, 256)[:len(r)]
    return q * np.repeat(s, 256)[:len(m)], z * z


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
