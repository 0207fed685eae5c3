"""The MoE router and its gradient on the GPU against binary64.  Choices,
counts and group ends must be equal.

Tolerances (u = 2^-24).  e^x is formed as 2^(x log2 e): its relative error is
at most 2 |x| u for the rounded product and 4 u for the function; a row's sum
adds at most 48 u.  So a probability is within (64 + 4 |z - zmax|) u of
itself, and lse within 64 u + 2 u |lse|.  The loss sums rows in some order:
(rows + 256) u more.  A gradient is within (128 + 8 |z - lse|) u of the
magnitudes that meet in it (+ half a bf16 ulp)."""
import math

import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import train_ref as ref
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

U, HALF = ref.U32, ref.half_ulp16
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _logits(rng, rows, experts, dtype, shut=0.0):
    z = (rng.standard_normal((rows, experts)) * 2).astype(np.float32).astype(np.float64)
    z = ref.bf16_round(z)          # many ties, in either type
    if shut:
        z[rng.random((rows, experts)) < shut] = -math.inf
    return z


def _dev(z, dtype, dev, pad=0):
    t = torch.from_numpy(np.ascontiguousarray(z)).to(TORCH[dtype]).to(dev)
    if pad == 0:
        return t
    wide = torch.full((z.shape[0], z.shape[1] + pad), float("nan"), dtype=TORCH[dtype], device=dev)
    wide[:, :z.shape[1]] = t
    return wide[:, :z.shape[1]]


def _np(t):
    return t.detach().double().cpu().numpy()


def _check_forward(z, got, want, topk):
    chosen, gates, lse, counts, ends, balance, loss = got
    assert np.array_equal(chosen.cpu().numpy(), want["chosen"]), "chosen"
    assert np.array_equal(counts.cpu().numpy(), want["counts"]), "counts"
    assert np.array_equal(ends.cpu().numpy(), want["ends"]), "ends"
    here = want["here"]
    with np.errstate(invalid="ignore"):
        span = np.where(np.isfinite(z), z.max(1, initial=-1e30, where=np.isfinite(z))[:, None] - z, 0.0)
    span = np.where(here[:, None], span, 0.0)
    at = np.where(want["chosen"] >= 0, want["chosen"], 0)
    far = np.take_along_axis(span, at, 1)
    ref.assert_close(_np(gates), want["gates"], (192 + 8 * far) * U * np.abs(np.nan_to_num(want["gates"])) + 1e-37,
                     "gates")
    ref.assert_close(_np(lse), want["lse"], 64 * U + 2 * U * np.abs(np.nan_to_num(want["lse"])), "lse")
    ref.assert_close(_np(balance), want["balance"], 8 * U * want["balance"], "balance")
    reach = span.max() if span.size else 0.0
    ref.assert_close(_np(loss), [want["loss"]],
                     (256 + z.shape[0] + 4 * min(reach, 100.0)) * U * abs(np.nan_to_num(want["loss"])), "loss")


CASES = [(1, 1, 1), (1, 2, 2), (3, 5, 1), (64, 16, 2), (7, 17, 4), (100, 32, 8), (65, 33, 3), (33, 64, 6), (50, 96, 8),
         (40, 100, 32), (300, 256, 8), (17, 255, 5), (9, 257, 2), (20, 512, 8), (6, 1000, 32), (5, 1024, 16),
         (2111, 24, 2)]


@pytest.mark.parametrize("rows,experts,topk", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_backward(rows, experts, topk, dtype):
    dev = device()
    rng = np.random.default_rng([rows, experts, topk, dtype == "f32"])
    normalize = (rows + topk) % 2 == 0
    align = [1, 32][experts % 2]
    pad = [0, 8, 5][(rows + experts) % 3]
    valid = rng.random(rows) > 0.2 if rows > 2 else None
    z = _logits(rng, rows, experts, dtype, 0.1 if rows % 2 else 0.0)
    want = ref.router(z, topk, valid, normalize, align)
    t = _dev(z, dtype, dev, pad)
    v = None if valid is None else torch.from_numpy(valid).to(dev)
    got = mx.mx_router_balance(t, topk, valid=v, normalize=normalize, align=align)
    _check_forward(z, got, want, topk)

    dgates = rng.standard_normal((rows, topk)).astype(np.float32)
    dloss = np.float32(0.37)
    dz = mx.mx_router_balance_backward(t, got[2], got[0], got[1], got[5], torch.from_numpy(dgates).to(dev),
                                       torch.tensor([dloss], device=dev), normalize=normalize)
    wz, mag = ref.router_backward(z, want["p"], want["chosen"], want["here"], normalize, want["balance"],
                                  dgates.astype(np.float64), float(dloss))
    span = np.where(np.isfinite(z), np.abs(z - want["lse"][:, None]), 0.0)
    tol = (128 + 8 * span.max(1, keepdims=True)) * U * 3 * mag
    ref.assert_close(_np(dz), wz, tol + (HALF(np.abs(wz) + tol) if dtype == "bf16" else 0.0) + 1e-37, "dlogits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [8, 48, 300])
def test_rows_that_take_no_part(dtype, experts):
    """Rows that valid drops, whatever they hold, and rows of -inf only: no
    choice, zero gates, no count, zero gradient; nothing of them leaks."""
    dev = device()
    rng = np.random.default_rng([3, experts])
    z = _logits(rng, 40, experts, dtype)
    valid = np.ones(40, bool)
    for r, junk in ((0, math.nan), (5, math.inf), (6, -math.inf), (39, math.nan)):
        valid[r] = False
        z[r] = junk
    z[10] = -math.inf
    z[11, 1:] = -math.inf                # one expert left
    z[12] = np.finfo(np.float32).min if dtype == "f32" else ref.bf16_round(np.float32(-3.38e38))   # all at the lowest
    want = ref.router(z, 4, valid, True, 32)
    got = mx.mx_router_balance(_dev(z, dtype, dev), 4, valid=torch.from_numpy(valid).to(dev), normalize=True, align=32)
    _check_forward(z, got, want, 4)
    assert (got[0][[0, 5, 6, 39, 10]] == -1).all()
    assert got[0][11].tolist() == [0, -1, -1, -1] and got[1][11].tolist() == [1, 0, 0, 0]
    assert got[0][12].tolist() == [0, 1, 2, 3]
    dz = mx.mx_router_balance_backward(_dev(z, dtype, dev), got[2], got[0], got[1], got[5],
                                       torch.ones(40, 4, device=dev), torch.ones(1, device=dev), normalize=True)
    assert not dz[[0, 5, 6, 39, 10]].any() and torch.isfinite(dz).all()


def test_no_row_takes_part():
    dev = device()
    for z, valid in ((torch.randn(70, 24, device=dev), torch.zeros(70, dtype=torch.bool, device=dev)),
                     (torch.full((3000, 24), -math.inf, device=dev), None), (torch.empty(0, 24, device=dev), None)):
        chosen, gates, lse, counts, ends, balance, loss = mx.mx_router_balance(z, 2, valid=valid)
        assert (chosen == -1).all() and not gates.any() and not lse.any()
        assert not counts.any() and not ends.any() and not balance.any() and loss.item() == 0.0
        dz = mx.mx_router_balance_backward(z, lse, chosen, gates, balance, torch.ones_like(gates),
                                           torch.ones(1, device=dev))
        assert not dz.any()


@pytest.mark.parametrize("experts", [16, 100, 600])
def test_infinities_and_nan_in_rows_that_count(experts):
    """NaN is chosen before +inf, +inf before the rest; the row's
    probabilities are NaN (as the formula gives), the choices whole."""
    dev = device()
    z = np.tile(np.linspace(-1, 1, experts), (3, 1)).astype(np.float32).astype(np.float64)
    z[0, 7], z[0, 3] = math.nan, math.inf
    z[1, 9] = math.inf
    want = ref.router(z, 3, None, False, 1)
    got = mx.mx_router_balance(_dev(z, "f32", dev), 3)
    assert np.array_equal(got[0].cpu().numpy(), want["chosen"])
    assert got[0][0].tolist()[:2] == [7, 3] and got[0][1].tolist()[0] == 9
    assert np.array_equal(got[3].cpu().numpy(), want["counts"])
    assert np.isnan(_np(got[1])[:2]).all() and np.isfinite(_np(got[1])[2]).all() and math.isnan(got[6].item())


def test_equal_logits_and_signed_zeros():
    """Ties go to the lowest index; -0 equals +0."""
    dev = device()
    for experts in (8, 40, 200, 700):
        for dtype in ("bf16", "f32"):
            z = torch.zeros(5, experts, dtype=TORCH[dtype], device=dev)
            z[1] = -0.0
            z[2, ::2] = -0.0
            z[3] = -1.0
            z[3, experts - 1] = z[3, experts // 2] = 2.0
            chosen = mx.mx_router_balance(z, 4)[0].tolist()
            for r in (0, 1, 2, 4):
                assert chosen[r] == [0, 1, 2, 3], (experts, dtype, r)
            assert chosen[3] == [experts // 2, experts - 1, 0, 1]


def test_gradient_against_differences():
    """(f(z + h v) - f(z - h v)) / 2h in binary64 for the fixed choice, h =
    2^-12: off by h^2 and by the gradient's own 2^-18."""
    dev = device()
    rng = np.random.default_rng(5)
    for normalize in (False, True):
        z = rng.standard_normal((30, 12)).astype(np.float32).astype(np.float64)
        want = ref.router(z, 3, None, normalize, 1)
        dgates = rng.standard_normal((30, 3)).astype(np.float32)
        got = mx.mx_router_balance(_dev(z, "f32", dev), 3, normalize=normalize)
        dz = mx.mx_router_balance_backward(_dev(z, "f32", dev), got[2], got[0], got[1], got[5],
                                           torch.from_numpy(dgates).to(dev), torch.tensor([2.0], device=dev),
                                           normalize=normalize)
        v, h = rng.standard_normal(z.shape), 2.0 ** -12
        f = [ref.router_value(z + s * h * v, want["chosen"], want["here"], normalize, want["balance"],
                              dgates.astype(np.float64), 2.0) for s in (1, -1)]
        got_d, size = float((_np(dz) * v).sum()), float(np.abs(_np(dz) * v).sum())
        assert abs(got_d - (f[0] - f[1]) / (2 * h)) <= 2.0 ** -17 * size


def test_either_gradient_may_be_absent():
    dev = device()
    z = torch.randn(50, 20, device=dev)
    chosen, gates, lse, _, _, balance, _ = mx.mx_router_balance(z, 3, normalize=True)
    dg, dl = torch.randn(50, 3, device=dev), torch.tensor([0.5], device=dev)
    both = mx.mx_router_balance_backward(z, lse, chosen, gates, balance, dg, dl, normalize=True)
    g = mx.mx_router_balance_backward(z, lse, chosen, gates, balance, dg, None, normalize=True)
    b = mx.mx_router_balance_backward(z, lse, chosen, gates, balance, None, dl, normalize=True)
    none = mx.mx_router_balance_backward(z, lse, chosen, gates, balance, None, None, normalize=True)
    assert not none.any()
    # linear in the two: equal up to a few roundings of the parts
    assert (both - g - b).abs().max().item() <= 16 * U * (g.abs() + b.abs()).max().item()


def test_same_bits_every_time():
    dev = device()
    z = torch.randn(9000, 60, device=dev)
    first = mx.mx_router_balance(z, 4)
    for _ in range(3):
        for a, b in zip(first, mx.mx_router_balance(z, 4)):
            assert torch.equal(a, b)


def test_refusals():
    dev = device()
    z = torch.zeros(4, 8, device=dev)
    chosen, gates, lse, _, _, balance, _ = mx.mx_router_balance(z, 2)
    for call in (lambda: mx.mx_router_balance(z.cpu(), 2), lambda: mx.mx_router_balance(z.half(), 2),
                 lambda: mx.mx_router_balance(z, 0), lambda: mx.mx_router_balance(z, 9),
                 lambda: mx.mx_router_balance(z, 2, align=0), lambda: mx.mx_router_balance(z.t(), 2),
                 lambda: mx.mx_router_balance(torch.zeros(4, 1025, device=dev), 2),
                 lambda: mx.mx_router_balance(torch.zeros(4, 64, device=dev), 33),
                 lambda: mx.mx_router_balance(z, 2, valid=torch.ones(3, dtype=torch.bool, device=dev)),
                 lambda: mx.mx_router_balance(z, 2, valid=torch.ones(4, device=dev)),
                 lambda: mx.mx_router_balance_backward(z, lse[:2], chosen, gates, balance),
                 lambda: mx.mx_router_balance_backward(z, lse, chosen.long(), gates, balance),
                 lambda: mx.mx_router_balance_backward(z, lse, chosen, gates[:, :1], balance),
                 lambda: mx.mx_router_balance_backward(z, lse, chosen, gates, balance, gates.bfloat16()),
                 lambda: mx.mx_router_balance_backward(z, lse, chosen, gates, balance, gates[:1].expand(4, 2))):
        with pytest.raises(ValueError):
            call()
    big = torch.zeros(5000, 8, device=dev)
    with pytest.raises(mx.MxError):
        mx.mx_router_balance(big, 2, workspace=torch.empty(4, device=dev))
