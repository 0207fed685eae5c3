"""The weight gradient from an 8-bit checkpoint: dy in rows that no 16-byte
word fits although n is a multiple of 8, in both tile sizes; and the smallest
values of a checkpoint."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import train_ref as ref
from tests.gpu_util import device, to_dev_u8

pytestmark = pytest.mark.gpu

# rows, n, k, columns of dy past its n and before them, group ends.  256 x 256
# tiles: whole, cut along the tokens, whole and cut together, short, groups not
# cut and cut; 128 x 128 tiles: the last three
SLICES = [(3000, 3104, 3104, 3, 0, None), (16640, 2048, 2048, 0, 1, None), (5000, 5120, 4352, 2, 5, None),
          (700, 3104, 3104, 0, 3, None), (16640, 3000, 4096, 5, 0, [100, 14000, 14100, 16640]),
          (16640, 2048, 4096, 1, 2, [15000, 15000, 16000, 16600]), (1664, 4128, 4128, 7, 0, None),
          (8192, 2048, 1024, 1, 1, None), (3000, 3104, 3104, 0, 5, [1000, 1001, 2999])]


@pytest.mark.parametrize("rows,n,k,pad,start,ends", SLICES)
def test_slices_of_a_wider_gradient(rows, n, k, pad, start, ends):
    """Against products in binary64 on the GPU.  Products are exact in binary32
    and at most one ulp (2^-23) is lost per addition: within (T + 32) 2^-23 of
    the sum of T products' magnitudes, and half a bf16 ulp as bf16.  dy lies
    between NaN, and so does what its last row ends in."""
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(rows + n + k)
    wide = torch.full((rows, start + n + pad), float("nan"), dtype=torch.bfloat16, device=dev)
    dy = wide[:, start:start + n]
    dy.copy_(torch.randn(rows, n, device=dev, generator=gen))
    assert dy.data_ptr() % 16 or dy.stride(0) % 8
    q = (torch.randn(rows, k, device=dev, generator=gen) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.randint(118, 130, (rows, k // 32), device=dev, generator=gen, dtype=torch.uint8)
    x = q.double().view(rows, k // 32, 32) * torch.exp2(s.double() - 127)[:, :, None]
    x = x.view(rows, k)
    e = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=dev)
    space = torch.full((max(mx.mx_wgrad_checkpoint_workspace_bytes(rows, n, k, 1 if ends is None else len(ends)), 16),),
                       0xFF, dtype=torch.uint8, device=dev)
    for dtype in (torch.float32, torch.bfloat16):
        got = mx.mx_wgrad_checkpoint(dy, q, s, e, out_dtype=dtype, workspace=space)
        lo = 0
        for g, hi in enumerate([rows] if ends is None else ends):
            a, b = dy[lo:hi].double(), x[lo:hi]
            want, mag = a.t().contiguous() @ b, a.abs().t().contiguous() @ b.abs()
            tol = (hi - lo + 32) * 2.0 ** -23 * mag
            if dtype == torch.bfloat16:
                tol += torch.exp2(torch.floor(torch.log2((want.abs() + tol).clamp(min=2.0 ** -126))) - 8)
            off = ((got if ends is None else got[g]).double() - want).abs()
            assert bool((off <= tol).all()), (dtype, g, int((off > tol).sum()))   # (NaN is not)
            lo = hi


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_below_the_normal_range(dtype):
    """One token with dy = 1, every code under every scale byte: a value below
    2^-126 is rounded to the nearest multiple of 2^-133 (bf16's smallest step),
    ties to even, and not taken as 0; from scale byte 3 on it is exact."""
    dev = device()
    codes = np.tile(np.arange(256, dtype=np.uint8), 256)[None]
    scales = np.repeat(np.arange(256, dtype=np.uint8), 8)[None]
    got = mx.mx_wgrad_checkpoint(torch.ones(1, 1, dtype=torch.bfloat16, device=dev), to_dev_u8(codes, dev),
                                 to_dev_u8(scales, dev), out_dtype=dtype).double().cpu().numpy()[0]
    want = ref.values(codes, scales)[0]
    low = np.isfinite(want) & (np.abs(want) < 2.0 ** -126)
    assert low.sum() > 1000 and (want[low] != 0).sum() > 500
    assert np.array_equal(got[low], np.rint(want[low] * 2.0 ** 133) * 2.0 ** -133)
    exact = low & (np.repeat(scales[0], 32) >= 3)
    assert exact.any() and np.array_equal(got[exact], want[exact])
