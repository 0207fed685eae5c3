"""Layer norm and its gradients on the GPU against binary64.

Tolerances, from the arithmetic (u = 2^-24).  A row sum is formed over at most
32 terms in a lane and 10 pairings of lanes and waves, so it is within 48 u of
the sum of its terms' magnitudes; a result adds a handful of roundings: 64 u
times the magnitudes that meet in it covers both.  An error of the mean enters
y through x - mean, with rstd |w|.  Weight gradients sum over rows in some
order: (rows + 64) u times the sum of magnitudes.  bf16 results are rounded
once more (half a bf16 ulp)."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import train_ref as ref
from tests.gpu_util import assert_bytes_equal, device, host, sentinel

pytestmark = pytest.mark.gpu

U, HALF = ref.U32, ref.half_ulp16
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _values(rng, shape, dtype, scale=1.0, offset=0.0):
    a = (rng.standard_normal(shape) * scale + offset).astype(np.float32).astype(np.float64)
    return ref.bf16_round(a) if dtype == "bf16" else a


def _dev(a, dtype, dev, pad=0):
    """On the device, rows `pad` elements wider than the matrix, NaN there."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TORCH[dtype]).to(dev)
    if pad == 0:
        return t
    wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=TORCH[dtype], device=dev)
    wide[:, :a.shape[1]] = t
    return wide[:, :a.shape[1]]


def _np(t):
    return t.detach().double().cpu().numpy()


def _fwd_check(x, w, b, eps, y, mean, rstd, bf16):
    wy, wm, wr = ref.layernorm(x, w, b, eps)
    mag = np.abs(x).mean(1)
    ref.assert_close(mean, wm, 64 * U * mag + 1e-44, "mean")
    ref.assert_close(rstd, wr, wr * (32 * U + (48 * U * mag * wr) ** 2 + 4 * U), "rstd")
    d = np.abs(x - wm[:, None]) * wr[:, None] * np.abs(w)
    tol = 64 * U * (d + (wr * mag)[:, None] * np.abs(w) + (0.0 if b is None else np.abs(b)))
    tol = tol + d * (48 * U * mag * wr)[:, None] ** 2
    ref.assert_close(y, wy, tol + (HALF(np.abs(wy) + tol) if bf16 else 0.0) + 1e-38, "y")


# columns: one, around a wave, one- and four-wave rows, longest; odd ones and
# whole 16-byte words
SHAPES = [(1, 1), (3, 7), (5, 64), (130, 96), (33, 511), (64, 512), (9, 1000), (17, 1024), (31, 1111), (2, 2048),
          (600, 2080), (3, 5120), (2, 6152), (2, 8192), (2, 10007), (1, 16384), (3, 16384)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_backward(rows, cols, dtype):
    dev = device()
    rng = np.random.default_rng([rows, cols, dtype == "f32"])
    wtype = "f32" if cols % 2 else dtype
    pad = [0, 8, 3][(rows + cols) % 3]
    x = _values(rng, (rows, cols), dtype, 1.5, 0.3)
    w = _values(rng, cols, wtype, 0.3, 1.0)
    b = _values(rng, cols, wtype, 0.2) if rows % 2 else None
    dy = _values(rng, (rows, cols), dtype)
    tx, tw = _dev(x, dtype, dev, pad), _dev(w, wtype, dev)
    y, mean, rstd = mx.mx_layernorm(tx, tw, None if b is None else _dev(b, wtype, dev), eps=1e-5)
    _fwd_check(x, w, b, 1e-5, _np(y), _np(mean), _np(rstd), dtype == "bf16")

    # backward of the statistics that the forward pass left
    dx, dw, db = mx.mx_layernorm_backward(_dev(dy, dtype, dev, pad), tx, tw, mean, rstd, bias=True)
    wx, ww, wb, xh, g = ref.layernorm_backward(dy, x, w, _np(mean), _np(rstd))
    tol = 64 * U * _np(rstd)[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                         + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    ref.assert_close(_np(dx), wx, tol + (HALF(np.abs(wx) + tol) if dtype == "bf16" else 0.0) + 1e-38, "dx")
    ref.assert_close(_np(dw), ww, (rows + 64) * U * np.abs(dy * xh).sum(0) + 1e-38, "dweight")
    ref.assert_close(_np(db), wb, (rows + 64) * U * np.abs(dy).sum(0) + 1e-38, "dbias")


@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 512), (70, 1056), (3, 5120), (2, 16384)])
def test_checkpoint_is_the_cast_of_y(rows, cols, oracle_mod):
    dev = device()
    rng = np.random.default_rng([7, rows, cols])
    x = _values(rng, (rows, cols), "bf16", 2.0)
    x[0, :32] = 0.0
    w = _values(rng, cols, "bf16", 0.3, 1.0)
    w[-32:] = 0.0                                  # blocks of zeros
    out = (torch.empty(rows, cols, dtype=torch.bfloat16, device=dev), torch.empty(rows, device=dev),
           torch.empty(rows, device=dev), sentinel((rows, cols), dev), sentinel((rows, cols // 32), dev))
    y, _, _, q, s = mx.mx_layernorm(_dev(x, "bf16", dev), _dev(w, "bf16", dev), checkpoint=True, out=out, raw=True)
    r_q, r_s, _ = ref.checkpoint(oracle_mod, _np(y))
    assert_bytes_equal(host(q), r_q, "codes")
    assert_bytes_equal(host(s), r_s, "scales")


def test_checkpoint_of_infinities_and_nan(oracle_mod):
    """A weight of Inf or NaN reaches y; the checkpoint is still y's cast."""
    dev = device()
    rng = np.random.default_rng(8)
    x = _values(rng, (4, 128), "bf16")
    w = np.ones(128)
    w[3], w[40], w[70] = np.inf, np.nan, -np.inf
    y, _, _, q, s = mx.mx_layernorm(_dev(x, "bf16", dev), _dev(w, "bf16", dev), checkpoint=True, raw=True)
    bits = y.view(torch.int16).cpu().numpy().view(np.uint16)
    r_q, r_s = oracle_mod.cast_dim0(np.concatenate([bits, np.zeros((28, 128), np.uint16)]))
    assert_bytes_equal(host(q), r_q[:4], "codes")
    assert_bytes_equal(host(s), r_s[:4], "scales")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_from_zero(dtype):
    """The variance is taken around the mean: rows at 1000 +- 1 keep it."""
    dev = device()
    rng = np.random.default_rng(9)
    x = 1000.0 + rng.integers(-4, 5, (5, 768)) * (8.0 if dtype == "bf16" else 0.25)
    w = np.ones(768)
    y, mean, rstd = mx.mx_layernorm(_dev(x, dtype, dev), _dev(w, "f32", dev))
    _fwd_check(x, w, None, 1e-5, _np(y), _np(mean), _np(rstd), dtype == "bf16")


def test_constant_rows_and_non_finite_rows():
    """A row without spread gives the bias (rstd = 1 / sqrt(eps)); a row with
    a NaN or an infinity is all NaN and leaves the other rows alone."""
    dev = device()
    x = np.tile(np.linspace(-1, 1, 96), (4, 1))
    x[0] = 2.0
    x[1, 5] = np.nan
    x[2, 7] = np.inf
    b = np.linspace(0, 1, 96).astype(np.float32).astype(np.float64)
    y, mean, rstd = mx.mx_layernorm(_dev(x, "f32", dev), _dev(np.ones(96), "f32", dev), _dev(b, "f32", dev))
    y = _np(y)
    assert np.array_equal(y[0], b)
    assert abs(_np(rstd)[0] * np.sqrt(1e-5) - 1) < 4 * U
    assert np.isnan(y[1]).all() and np.isnan(y[2]).all() and np.isfinite(y[3]).all()


def test_no_rows():
    dev = device()
    x = torch.empty(0, 96, device=dev)
    w = torch.ones(96, device=dev)
    y, mean, rstd = mx.mx_layernorm(x, w)
    assert y.shape == (0, 96) and mean.shape == (0,) and rstd.shape == (0,)
    out = (x.clone(), torch.full((96,), 7.0, device=dev), torch.full((96,), 7.0, device=dev))
    _, dw, db = mx.mx_layernorm_backward(x, x, w, mean, rstd, out=out)
    assert not dw.any() and not db.any()


def test_gradients_against_differences():
    """Along a random direction: (L(p + h v) - L(p - h v)) / 2h of L = sum(dy *
    y) in binary64, h = 2^-10, against the kernels' gradients.  The quotient is
    off by h^2 times a third derivative of order one per element; the
    gradients by about 2^-20 of their magnitudes."""
    dev = device()
    rng = np.random.default_rng(10)
    rows, cols, h = 6, 200, 2.0 ** -10
    x, w, b, dy = (_values(rng, s, "f32", 1.0, o) for s, o in (((rows, cols), 0.5), (cols, 1.0), (cols, 0.0),
                                                               ((rows, cols), 0.0)))
    _, mean, rstd = mx.mx_layernorm(_dev(x, "f32", dev), _dev(w, "f32", dev), _dev(b, "f32", dev))
    grads = mx.mx_layernorm_backward(_dev(dy, "f32", dev), _dev(x, "f32", dev), _dev(w, "f32", dev), mean, rstd)
    for i, p in enumerate((x, w, b)):
        v = rng.standard_normal(p.shape)
        args = [x, w, b]
        diff = []
        for sign in (1, -1):
            args[i] = p + sign * h * v
            diff.append(float((dy * ref.layernorm(*args, 1e-5)[0]).sum()))
        want = (diff[0] - diff[1]) / (2 * h)
        got = float((_np(grads[i]) * v).sum())
        size = float(np.abs(_np(grads[i]) * v).sum())
        assert abs(got - want) <= 2.0 ** -16 * size, (i, got, want)


def test_same_bits_every_time():
    dev = device()
    rng = np.random.default_rng(11)
    x = _dev(_values(rng, (3001, 1056), "bf16"), "bf16", dev)
    w = _dev(_values(rng, 1056, "f32"), "f32", dev)
    y, mean, rstd = mx.mx_layernorm(x, w)
    first = mx.mx_layernorm_backward(x, x, w, mean, rstd)
    for _ in range(3):
        for a, b in zip(first, mx.mx_layernorm_backward(x, x, w, mean, rstd)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Elements past 2^31: the last rows of a tall matrix."""
    dev = device()
    rows, cols = (1 << 17) + 37, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=dev)
    tail = _values(np.random.default_rng(12), (40, cols), "bf16")
    x[-40:] = _dev(tail, "bf16", dev)
    w = torch.ones(cols, device=dev)
    y, mean, rstd = mx.mx_layernorm(x, w)
    _fwd_check(tail, np.ones(cols), None, 1e-5, _np(y[-40:]), _np(mean[-40:]), _np(rstd[-40:]), True)
    assert not y[:-40].any()
    dx, dw, db = mx.mx_layernorm_backward(x, x, w, mean, rstd)
    wx, ww, wb, xh, g = ref.layernorm_backward(tail, tail, np.ones(cols), _np(mean[-40:]), _np(rstd[-40:]))
    tol = 64 * U * _np(rstd[-40:])[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                               + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    ref.assert_close(_np(dx[-40:]), wx, tol + HALF(np.abs(wx) + tol) + 1e-38, "dx")
    ref.assert_close(_np(dw), ww, (40 + 64) * U * np.abs(tail * xh).sum(0) + 1e-38, "dweight")


def test_refusals():
    dev = device()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    m = torch.zeros(4, device=dev)
    for call in (lambda: mx.mx_layernorm(x.cpu(), w), lambda: mx.mx_layernorm(x.half(), w),
                 lambda: mx.mx_layernorm(x, w[:32]), lambda: mx.mx_layernorm(x, w.half()),
                 lambda: mx.mx_layernorm(x, w, w.bfloat16()), lambda: mx.mx_layernorm(x.t(), w[:4]),
                 lambda: mx.mx_layernorm(x[0], w), lambda: mx.mx_layernorm(x[:1].expand(4, 64), w),
                 lambda: mx.mx_layernorm(x.float(), w, checkpoint=True),
                 lambda: mx.mx_layernorm(x[:, :40], w[:40], checkpoint=True),
                 lambda: mx.mx_layernorm(x, w, out=(x, m)),
                 lambda: mx.mx_layernorm(x, w, out=(x.float(), m, m)),
                 lambda: mx.mx_layernorm_backward(x.float(), x, w, m, m),
                 lambda: mx.mx_layernorm_backward(x[:2], x, w, m, m),
                 lambda: mx.mx_layernorm_backward(x, x, w, m[:2], m)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mx.MxError):
        mx.mx_layernorm(torch.zeros(1, 16385, device=dev), torch.ones(16385, device=dev))
    with pytest.raises(mx.MxError):   # too small a workspace
        mx.mx_layernorm_backward(x, x, w, m, m, workspace=torch.empty(16, device=dev))
