"""The plain implementations that the 4-bit operators are tested with: the cast
against a search for the nearest value, worked blocks, and the block's gradient
against differences."""
import numpy as np
import pytest

from tests import fp4_ref as r4
from tests import train_ref as ref


def test_nearest_by_search():
    t = np.concatenate([np.linspace(0, 8, 4097), r4.MIDDLES, np.nextafter(r4.MIDDLES, 0), np.nextafter(r4.MIDDLES, 9)])
    got = r4.round_e2m1(t)
    for v, c in zip(t, got):
        d = np.abs(r4.TABLE - min(v, 6.0))
        near = np.flatnonzero(d == d.min())
        assert c in near and (len(near) == 1 or c % 2 == 0), (v, c)


def test_worked_block():
    x = np.zeros((1, 64))
    x[0, :8] = [6.0, -6.0, 7.9, 0.25, 0.75, -0.0, 2.5, 5.0]     # amax 7.9: 2^0
    x[0, 32:36] = [1.0, 0.125, 0.0625, -0.1875]                 # amax 1: 2^-2
    q, s = r4.cast4(x)
    assert s.tolist() == [[127, 125]]
    assert q[0, :8].tolist() == [7, 15, 7, 0, 2, 8, 4, 6] and q[0, 32:36].tolist() == [6, 1, 0, 10]
    assert np.array_equal(r4.unpack(r4.pack(q)), q)
    assert r4.values4(q, s)[0, :8].tolist() == [6, -6, 6, 0, 1, 0, 2, 4]


def test_special_blocks():
    x = np.ones((4, 32))
    x[0, 3], x[1, 5], x[2] = np.inf, np.nan, 0.0
    x[3] = 2.0 ** -140
    q, s = r4.cast4(x)
    assert s[:, 0].tolist() == [254, 255, 0, 0]
    assert q[0, 3] == 7 and q[0, 0] == 0 and not q[1].any() and not q[2].any() and not q[3].any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """d sum(D * ((act(g) u) Wd^T)) by g and u."""
    rng = np.random.default_rng(3)
    g, u, wd, d = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal((3, 5))
    dg, du = ref.gated_act_backward(d @ wd, g, u, act)

    def value(g, u):
        return float((d * (ref.gated_act(g, u, act) @ wd.T)).sum())

    step = 1e-5   # error of a central difference: step^2 / 6 times a third derivative of order 10
    for grad, which in ((dg, 0), (du, 1)):
        for i in np.ndindex(grad.shape):
            e = np.zeros_like(g)
            e[i] = step
            hi, lo = ((value(g + e, u), value(g - e, u)), (value(g, u + e), value(g, u - e)))[which]
            assert abs((hi - lo) / (2 * step) - grad[i]) < 1e-7


def test_checkpoint_range_holds_the_cast(oracle_mod):
    """Without an error the range is the oracle's cast itself."""
    rng = np.random.default_rng(4)
    h = ref.bf16_round(rng.standard_normal((32, 64)) * np.exp2(rng.integers(-6, 7, (32, 64))))
    q, s, v = ref.checkpoint(oracle_mod, h)
    lo, hi, held = r4.checkpoint_range(h, np.zeros_like(h))
    assert np.array_equal(lo, s) and np.array_equal(hi, s)
    a, b = held(s)
    assert np.array_equal(a, v) and np.array_equal(b, v)
