"""The products of a few bf16 rows with MX weights on the GPU against binary64.

Tolerance: a code times its scale and a bf16 x are exact, their products too;
K sums of binary32 in any order are within K 2^-24 of the magnitudes that meet;
the gate and the output's rounding as in tests/fp4_ref.py."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import fp4_ref as r4
from tests import train_ref as ref
from tests.gpu_util import device, to_dev_u8

pytestmark = pytest.mark.gpu

FORMATS = ["e2m1", "e4m3"]


def _np(t):
    return t.detach().double().cpu().numpy()


def _x(rng, m, k, dev, pad=0, first=0):
    v = ref.bf16_round(rng.standard_normal((m, k)) * np.exp2(rng.integers(-4, 3, (m, k))))
    wide = torch.full((m, k + pad + first), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, first:first + k] = torch.from_numpy(v).to(dev).bfloat16()
    return v, wide[:, first:first + k]


def _weights(oracle_mod, rng, n, k, fmt, dev):
    q, s = r4.operand(rng, n, k, fmt)
    return to_dev_u8(q, dev), to_dev_u8(oracle_mod.to_blocked(s), dev), r4.values(q, s, fmt)


def _sum_error(mag, k):
    return mag * k * 2.0 ** -24


SIZES = [(1, 1, 32), (1, 17, 64), (2, 16, 96), (1, 300, 5120), (7, 129, 160), (16, 64, 1056), (17, 33, 128),
         (32, 100, 544), (33, 48, 416), (64, 250, 1024), (48, 16, 8192), (64, 1, 32)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear(m, n, k, fmt, oracle_mod):
    dev = device()
    rng = np.random.default_rng([m, n, k, fmt == "e2m1"])
    v, x = _x(rng, m, k, dev)
    qw, sw, w = _weights(oracle_mod, rng, n, k, fmt, dev)
    want, mag = r4.product(v, w)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((m * n + 2,), 7.0, dtype=dt, device=dev)
        y = mx.mx_linear_decode(x, qw, sw, out_dtype=dt, out=out[1:-1].view(m, n))
        ref.assert_close(_np(y), want, r4.round_tol(want, _sum_error(mag, k), dt == torch.bfloat16), "y")
        assert out[0] == 7 and out[-1] == 7
        assert torch.equal(y, mx.mx_linear_decode(x, qw, sw, out_dtype=dt))


@pytest.mark.parametrize("m,f,k", [(1, 1, 32), (1, 5, 64), (3, 256, 160), (16, 33, 1056), (20, 96, 288), (64, 130, 512),
                                   (40, 16, 5120)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(m, f, k, fmt, act, oracle_mod):
    dev = device()
    rng = np.random.default_rng([m, f, k, fmt == "e2m1"])
    v, x = _x(rng, m, k, dev)
    v, x = v * 2.0 ** -4, x * 2.0 ** -4     # gates where the activation bends
    qw, sw, w = _weights(oracle_mod, rng, 2 * f, k, fmt, dev)
    h, mag = r4.product(v, w)
    y = mx.mx_gated_ffn_decode(x, qw, sw, act=act)
    want = r4.gated(h, act)
    ref.assert_close(_np(y), want, r4.round_tol(want, r4.gated_tol(h, _sum_error(mag, k), act), True), "y")
    assert torch.equal(y, mx.mx_gated_ffn_decode(x, qw, sw, act=act))


@pytest.mark.parametrize("pad,first", [(1, 0), (8, 0), (3, 5), (0, 1)])
def test_rows_at_any_pitch_and_start(pad, first, oracle_mod):
    dev = device()
    rng = np.random.default_rng([pad, first])
    m, n, k = 19, 70, 416
    v, x = _x(rng, m, k, dev, pad, first)
    qw, sw, w = _weights(oracle_mod, rng, n, k, "e2m1", dev)
    y = mx.mx_linear_decode(x, qw, sw, out_dtype=torch.float32)
    want, mag = r4.product(v, w)
    ref.assert_close(_np(y), want, r4.round_tol(want, _sum_error(mag, k), False), "y")
    assert torch.equal(y, mx.mx_linear_decode(x.contiguous(), qw, sw, out_dtype=torch.float32))


@pytest.mark.parametrize("m,pitch", [(5, (1 << 25) + 32), (2, 1 << 28)])
def test_last_tokens_of_long_sequences(m, pitch, oracle_mod):
    """Rows of x far apart, as the last tokens of (batch, tokens, K) lie."""
    dev = device()
    rng = np.random.default_rng(m)
    n, k = 40, 160
    qw, sw, w = _weights(oracle_mod, rng, n, k, "e2m1", dev)
    v, x = _x(rng, m, k, dev)
    wide = torch.full(((m - 1) * pitch + k,), float("nan"), dtype=torch.bfloat16, device=dev)
    far = wide.as_strided((m, k), (pitch, 1))
    far.copy_(x)
    assert torch.equal(mx.mx_linear_decode(far, qw, sw), mx.mx_linear_decode(x, qw, sw))
    assert torch.equal(mx.mx_gated_ffn_decode(far, qw, sw), mx.mx_gated_ffn_decode(x, qw, sw))


def test_nan_blocks_and_infinite_x(oracle_mod):
    """A block of scale 0xFF makes its column NaN; Inf and NaN of x stay in
    their row; the other rows and columns do not see them."""
    dev = device()
    rng = np.random.default_rng(3)
    m, n, k = 18, 40, 160
    for fmt in FORMATS:
        q, s = r4.operand(rng, n, k, fmt)
        s[5, 1], s[37, 4] = 255, 255
        v, x = _x(rng, m, k, dev)
        v[2, 50], v[17, 3] = np.inf, np.nan
        x = torch.from_numpy(v).to(dev).bfloat16()
        y = mx.mx_linear_decode(x, to_dev_u8(q, dev), to_dev_u8(oracle_mod.to_blocked(s), dev), out_dtype=torch.float32)
        with np.errstate(invalid="ignore"):
            want = v @ r4.values(q, s, fmt).T
            mag = np.abs(np.nan_to_num(v, posinf=0)) @ np.abs(np.nan_to_num(r4.values(q, s, fmt))).T
        ref.assert_close(_np(y), want, _sum_error(mag, k) + np.abs(np.nan_to_num(want)) * 2.0 ** -24 + 1e-40, fmt)


def test_empty():
    dev = device()
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    w, s = torch.zeros(8, 32, dtype=torch.uint8, device=dev), torch.zeros(128, 4, dtype=torch.uint8, device=dev)
    assert mx.mx_linear_decode(x, w, s).shape == (0, 8) and mx.mx_gated_ffn_decode(x, w, s).shape == (0, 4)
    none = torch.zeros(8, 0, dtype=torch.uint8, device=dev)
    y = mx.mx_linear_decode(torch.zeros(3, 0, dtype=torch.bfloat16, device=dev), none, none[:0].reshape(0),
                            out=torch.ones(3, 8, dtype=torch.bfloat16, device=dev))
    assert bool((y == 0).all())
