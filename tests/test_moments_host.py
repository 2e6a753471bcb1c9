"""8-bit moments over many steps, in their plain form (no GPU needed): codes rounded
by the hash keep the moments' means and follow float32 AdamW for slow betas, where
the nearest codes do not."""
import numpy as np
import pytest

import moments_ref as mom
import more_ref as ref
from block_ref import e4m3_values

F = np.float32
SIZES = {"equal": np.full(256, 1e-2, F),
         "mixed": np.exp(np.random.default_rng(1).uniform(np.log(1e-4), np.log(1e-2), 256)).astype(F)}


def hashed(m, r, step):
    return mom.moments(m, r, step)


def nearest(m, r, step):
    return mom.moments(m, r, None)


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("kind", mom.KINDS)
@pytest.mark.parametrize("b2", [0.95, 0.99, 0.999])
def test_hashed_moments_follow_float32(b2, kind, sizes):
    """Within a tenth of the update's norm after 3000 steps."""
    assert abs(mom.update_ratio(kind, 3000, 0.9, b2, SIZES[sizes], hashed) - 1) < 0.1


def test_nearest_codes_do_not_at_slow_betas():
    """What the rule for the betas keeps apart, on few elements."""
    few = SIZES["equal"][:64]
    for kind, b2, low, high in (("shrinking", 0.99, 0, 0.1), ("normal", 0.999, 1.3, 9),
                                ("constant", 0.999, 2, 9), ("normal", 0.95, 0.9, 1.1),
                                ("shrinking", 0.95, 0.9, 1.1)):
        assert low < mom.update_ratio(kind, 1500, 0.9, b2, few, nearest) < high, (kind, b2)


@pytest.mark.parametrize("b1,b2", [(0.9, 0.95), (0.8, 0.9), (0.8, 0.95), (0.7, 0.94), (0.5, 0.75),
                                   (0.5, 0.9), (0.0, 0.5), (0.0, 0.8)])
def test_nearest_codes_where_they_are_kept(b1, b2):
    """Within an eighth: v falls, and the lags of m and v nearly cancel."""
    for kind in mom.KINDS:
        for sizes in SIZES.values():
            assert abs(mom.update_ratio(kind, 400, b1, b2, sizes, nearest) - 1) < 0.125, kind


def test_the_mean_over_steps_is_the_value():
    """Means of N draws of a value between two codes: the standard deviation is half
    their distance over sqrt(N) at most, and six of them are allowed."""
    n, steps = 256, 4000
    rng = np.random.default_rng(2)
    m = (rng.standard_normal(n) * np.exp(rng.uniform(-12, 0, n))).astype(F)
    r = np.exp(rng.uniform(-6, 0, n)).astype(F)
    sm, sv = np.zeros(n), np.zeros(n)
    for t in range(1, steps + 1):
        a, b = mom.moments(m, r, t)
        sm, sv = sm + a, sv + b
    scale = ref._scales(np.array([np.abs(m).max()], np.float64), 448.0)[0]
    place = np.exp2(np.maximum(np.floor(np.log2(np.abs(m) / scale)), -6) - 3) * scale
    assert (np.abs(sm / steps - m) <= 3 * place / steps ** 0.5).all()
    v = r.astype(np.float64) ** 2
    root = ref._scales(np.array([r.max()], np.float64), 4032.0)[0]
    e = np.exp2(np.maximum(np.floor(np.log2(r / root)) - 5, 0))
    low = np.floor(r / root / e)
    assert low.min() >= 1
    assert (np.abs(sv / steps - v) <= 3 * (2 * low + 1) * (e * root) ** 2 / steps ** 0.5).all()


def test_scales_are_those_of_the_nearest_codes():
    tops = np.concatenate([F(2) ** np.arange(-149, 127, 3), F(448) * F(2) ** np.arange(-120, 100, 7),
                           np.nextafter(F(4032) * F(2) ** np.arange(-120, 100, 7), F(9e9)), [0, 3.3e38]]).astype(F)
    for limit in (448.0, 4032.0):
        assert np.array_equal(mom.scales(tops, limit), ref._scales(tops.astype(np.float64), limit).astype(F))


def test_nearest_codes_are_those_found_by_search():
    rng = np.random.default_rng(5)
    m = (rng.standard_normal(1500) * np.exp(rng.uniform(-15, 0, 1500))).astype(F)
    for got, want in zip(mom.m_codes(m, None) + mom.v_codes(np.abs(m), None),
                         ref.m_codes(m) + ref.v_codes(np.abs(m))):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("step", [None, 3])
def test_a_root_that_is_not_finite_keeps_to_itself(step):
    """Its code is 255, its block's scale a NaN that holds the scale, and the others
    mean what they mean without it, where it is not the largest."""
    r = np.exp(np.random.default_rng(6).uniform(-6, 0, 700)).astype(F)
    for bad in (np.nan, np.inf):
        x = r.copy()
        x[300] = bad
        (c, s), (c0, s0) = mom.v_codes(x, step), mom.v_codes(r, step)
        assert np.isnan(s).tolist() == [False, True, False] and c[300] == 255
        same = np.arange(700) != 300
        assert np.array_equal(c[same], c0[same]) and (c[256:512] == 255).sum() == 1
        v = mom.v_of(c, s)
        assert np.array_equal(v[same], mom.v_of(c0, s0)[same]) and v[300] == np.inf
    # a root that would be code 255 takes the next scale beside a mark
    x = np.array([4032, 5, np.inf], F)
    c, s = mom.v_codes(x, step)
    assert c[0] == 223 and mom.v_of(c, s)[0] == F(4032) ** 2 and mom.v_of(c, s)[2] == np.inf
    # a NaN that holds no scale makes a block of NaN
    assert np.isnan(mom.v_of(np.array([3, 0], np.uint8), np.array([np.nan], F))).all()


def test_values_that_codes_hold_stay():
    """Every code's own value, whatever the draw."""
    e4m3 = np.abs(e4m3_values().numpy())
    m = np.zeros(256, F)
    m[:len(e4m3)] = e4m3
    r = ref.root_values().astype(F)
    for t in (1, 2, 77, 2 ** 40, 2 ** 62):
        q, s = mom.m_codes(m, t)
        c, z = mom.v_codes(r, t)
        assert s[0] == 1 and z[0] == 1
        assert np.array_equal(q, m) and np.array_equal(c, np.arange(256))


def test_draws():
    """Different by step and by element, far ones too; each half even over (0, 1)."""
    a = mom.draws(5, 0, 4096)
    for k in (0, 1):
        for other in (mom.draws(6, 0, 4096), mom.draws(5 + 2 ** 32, 0, 4096), mom.draws(5, 2 ** 32, 4096)):
            assert (a[k] != other[k]).mean() > 0.99
        assert abs(a[k].mean() - 0.5) < 6 / (12 * 4096) ** 0.5 and 0 < a[k].min() and a[k].max() < 1
    assert np.array_equal(mom.draws(0, 0, 9), mom.draws(1, 0, 9))
    assert np.array_equal(mom.draws(5, 1000, 96)[0], a[0][1000:1096])
