"""Layer norm at the ends of its range: gradients of rows far out, lengths of
zero and past the longest, checkpoints of rows at any pitch and start.

Tolerances as for the layer norm's other tests (u = 2^-24): 64 u of the
magnitudes that meet in a result, (rows + 64) u of those that meet in a weight
gradient, and half a bf16 ulp where a result is bf16."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import train_ref as ref
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

U, HALF = ref.U32, ref.half_ulp16
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev(a, dtype, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(TORCH[dtype]).to(dev)


def _np(t):
    return t.detach().double().cpu().numpy()


# lengths that fill the lanes' last words and lengths that leave lanes empty
@pytest.mark.parametrize("cols", [96, 512, 1000, 5120, 8192, 9000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_a_constant_row_far_out(cols, dtype):
    """A row of 2^120 throughout: every x - mean is 0 and the gradient finite,
    although mean * rstd (rstd = 1 / sqrt(1e-5)) is past binary32's largest."""
    dev = device()
    rng = np.random.default_rng([31, cols])
    x = ref.bf16_round(rng.standard_normal((6, cols)))
    x[2] = 2.0 ** 120
    dy = ref.bf16_round(rng.standard_normal((6, cols)))
    w = ref.bf16_round(1.0 + 0.3 * rng.standard_normal(cols))
    mean, rstd = x.mean(1).astype(np.float32), (1.0 / np.sqrt(x.var(1) + 1e-5)).astype(np.float32)
    assert mean[2] == 2.0 ** 120 and float(mean[2]) * float(rstd[2]) > float(np.finfo(np.float32).max)
    dx, dw, db = mx.mx_layernorm_backward(_dev(dy, dtype, dev), _dev(x, dtype, dev), _dev(w, "f32", dev),
                                          torch.from_numpy(mean).to(dev), torch.from_numpy(rstd).to(dev))
    m64, r64 = mean.astype(np.float64), rstd.astype(np.float64)
    wx, ww, wb, xh, g = ref.layernorm_backward(dy, x, w, m64, r64)
    tol = 64 * U * r64[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                   + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    ref.assert_close(_np(dx), wx, tol + (HALF(np.abs(wx) + tol) if dtype == "bf16" else 0.0) + 1e-38, "dx")
    ref.assert_close(_np(dw), ww, (6 + 64) * U * np.abs(dy * xh).sum(0) + 1e-38, "dweight")
    ref.assert_close(_np(db), wb, (6 + 64) * U * np.abs(dy).sum(0) + 1e-38, "dbias")
