"""Codes and scales of another 8-bit type than the operators read are refused
(they were read as e4m3 or e2m1 codes, or as e8m0 scales).  The checks run on the
host, so that tensors of any device serve here."""
import pytest
import torch

from fp8_precision_quantization_amd import _fp4, _train

OTHER_CODES = [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.float8_e8m0fnu]
OTHER_SCALES = [torch.float8_e5m2, torch.float8_e4m3fn, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz]


@pytest.fixture(autouse=True)
def any_device(monkeypatch):
    calls = []
    for module in (_fp4, _train):
        monkeypatch.setattr(module, "_gpu", lambda t, name: None)
    monkeypatch.setattr(_fp4, "_typed", lambda t, dtypes, name: None)
    monkeypatch.setattr(_fp4, "_call", lambda name, *a: calls.append(name))
    return calls


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


X = torch.zeros(3, 64, dtype=torch.bfloat16)
ENDS = torch.zeros(2, dtype=torch.int32)


def _calls(q, s):
    """Every call with q and s as the cast of its codes and scales."""
    q4, q8, sb = q(_u8(3, 32)), q(_u8(3, 64)), s(_u8(128, 4))
    w4, w8, wb = q(_u8(64, 32)), q(_u8(64, 64)), s(_u8(128, 4))
    yield "mx_dequantize_mxfp4", lambda: _fp4.mx_dequantize_mxfp4(q4, s(_u8(3, 2)))
    yield "mx_dequantize_mxfp4", lambda: _fp4.mx_dequantize_mxfp4(q4, sb, blocked=True)
    yield "mx_gemm_mxfp4", lambda: _fp4.mx_gemm_mxfp4(q8, sb, w4, wb)
    yield "mx_grouped_gemm_mxfp4", lambda: _fp4.mx_grouped_gemm_mxfp4(q8, s(_u8(3 + 256, 4)), q(_u8(2, 64, 32)),
                                                                      s(_u8(256, 4)), ENDS)
    yield "mx_linear_decode", lambda: _fp4.mx_linear_decode(X, w8, wb)
    yield "mx_gated_ffn_decode", lambda: _fp4.mx_gated_ffn_decode(X, w8, wb)
    yield "mx_gated_ffn", lambda: _fp4.mx_gated_ffn(q8, sb, w8, wb)
    yield "mx_gated_ffn_backward", lambda: _fp4.mx_gated_ffn_backward(q8, sb, w8, wb, q(_u8(3, 128)), s(_u8(3, 4)))


def _same(t):
    return t


def test_bytes_are_taken(any_device):
    names = [name for name, call in _calls(_same, _same) if call() is not None]
    assert any_device == names
    for name, call in _calls(_same, lambda t: t.view(torch.float8_e8m0fnu)):
        call()


@pytest.mark.parametrize("dtype", OTHER_CODES)
def test_other_codes(dtype, any_device):
    for name, call in _calls(lambda t: t.view(dtype), _same):
        with pytest.raises(ValueError, match="codes|holds"):
            call()
    assert not any_device


@pytest.mark.parametrize("dtype", OTHER_SCALES)
def test_other_scales(dtype, any_device):
    for name, call in _calls(_same, lambda t: t.view(dtype)):
        with pytest.raises(ValueError, match="scales"):
            call()
    assert not any_device


@pytest.mark.parametrize("dtype", OTHER_CODES)
def test_other_checkpoints(dtype, any_device):
    """The checkpoint's codes alone."""
    with pytest.raises(ValueError, match="codes"):
        _fp4.mx_gated_ffn_backward(_u8(3, 64), _u8(128, 4), _u8(64, 64), _u8(128, 4), _u8(3, 128).view(dtype), _u8(3, 4))
    with pytest.raises(ValueError, match="codes"):
        _fp4.mx_gated_ffn_backward(_u8(3, 64), _u8(128, 4), _u8(64, 64), _u8(128, 4),
                                   _u8(3, 128).view(torch.float4_e2m1fn_x2), _u8(3, 4))
