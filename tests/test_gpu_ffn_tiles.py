"""The gated feed-forward block and its gradient in the forms of their kernels
that take several groups in large tiles, more groups than a scalar loop places,
and GELU in large tiles and in quarters of them.  Checks and tolerances are
those of tests/test_gpu_ffn.py."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import fp4_ref as r4
from tests.gpu_util import device, sentinel, to_dev_u8
from tests.test_gpu_ffn import NAMES, PAIRS, _check_backward, _check_forward, _kept, _operands

pytestmark = pytest.mark.gpu


def _forward(oracle_mod, rows, f, k, fx, fw, act, ends):
    dev = device()
    rng = np.random.default_rng([rows, f, k])
    args, off, x, w = _operands(oracle_mod, rng, dev, rows, 2 * f, k, fx, fw, ends)
    out = (torch.full((rows, f), -77.0, dtype=torch.bfloat16, device=dev), sentinel((rows, 2 * f), dev),
           sentinel((rows, f // 16), dev))
    y, q, s = mx.mx_gated_ffn(*args, act=act, group_end_offsets=off, a_format=NAMES[fx], w_format=NAMES[fw], out=out,
                              raw=True)
    hi = 0
    for i, (lo, hi) in enumerate(r4.bounds([rows] if ends is None else ends, rows)):
        if hi > lo:
            _check_forward(y[lo:hi], q[lo:hi], s[lo:hi], x[lo:hi], w[i], fx, fw, act, "group %d" % i)
    assert bool((y[hi:] == -77).all()) and bool((q[hi:] == 0xCD).all()) and bool((s[hi:] == 0xCD).all())


def _backward(oracle_mod, rows, f, k, fx, fw, act, ends):
    dev = device()
    rng = np.random.default_rng([rows, f, k, 8])
    args, off, d, w = _operands(oracle_mod, rng, dev, rows, f, k, fx, fw, ends)
    q, s, h = _kept(rng, rows, f)
    out = tuple(torch.full((rows, n), -77.0, dtype=torch.bfloat16, device=dev) for n in (2 * f, f))
    dh, y = mx.mx_gated_ffn_backward(*args, to_dev_u8(q, dev), to_dev_u8(s, dev), act=act, group_end_offsets=off,
                                     a_format=NAMES[fx], w_format=NAMES[fw], recompute=True, out=out)
    hi = 0
    for i, (lo, hi) in enumerate(r4.bounds([rows] if ends is None else ends, rows)):
        if hi > lo:
            _check_backward(dh[lo:hi], y[lo:hi], d[lo:hi], w[i], h[lo:hi], fx, fw, act, "group %d" % i)
    assert bool((dh[hi:] == -77).all()) and bool((y[hi:] == -77).all())


RAGGED = [700, 701, 701, 2900]   # of 3100 rows: one row, none, and rows past the last end


@pytest.mark.parametrize("fx,fw", PAIRS)
def test_groups_in_large_tiles(fx, fw, oracle_mod):
    """At least 192 tiles of 256 rows: the larger ones are taken."""
    _forward(oracle_mod, 3100, 2080, 160, fx, fw, "gelu", RAGGED)
    _backward(oracle_mod, 3100, 4160, 96, fx, fw, "silu", RAGGED)


@pytest.mark.parametrize("fx,fw", PAIRS)
def test_one_group_in_large_tiles(fx, fw, oracle_mod):
    _forward(oracle_mod, 3333, 2048, 64, fx, fw, "silu", [3300])
    _backward(oracle_mod, 3333, 4128, 64, fx, fw, "gelu", [3300])


@pytest.mark.parametrize("groups", [33, 150])
@pytest.mark.parametrize("fx,fw", PAIRS)
def test_many_groups(groups, fx, fw, oracle_mod):
    ends = np.sort(np.random.default_rng(groups).integers(0, 700, groups))
    _forward(oracle_mod, 717, 64, 96, fx, fw, "silu", ends)
    _backward(oracle_mod, 717, 64, 96, fx, fw, "gelu", ends)


@pytest.mark.parametrize("fx,fw", PAIRS)
def test_many_groups_in_large_tiles(fx, fw, oracle_mod):
    ends = np.sort(np.random.default_rng(5).integers(0, 1900, 40))
    _forward(oracle_mod, 2000, 640, 64, fx, fw, "silu", ends)
    _backward(oracle_mod, 2000, 1280, 32, fx, fw, "silu", ends)


@pytest.mark.parametrize("fx,fw", PAIRS)
@pytest.mark.parametrize("forward,backward", [((4100, 1568, 160), (3333, 3680, 96)), ((4100, 2112, 96), (4353, 4096, 32))])
def test_gelu_in_large_tiles_and_quarters(forward, backward, fx, fw, oracle_mod):
    _forward(oracle_mod, *forward, fx, fw, "gelu", None)
    _backward(oracle_mod, *backward, fx, fw, "gelu", None)
