"""The third part of the C ABI (include/mxfp4.h) on a machine without a GPU:
every declared symbol is exported and bound, and bad arguments are rejected on
the host before any HIP call."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxfp4.h")

OK, NULL, SHAPE, GROUPS, HIP, ALIGN, WORKSPACE = range(7)
P = ctypes.c_void_p(0x10000)       # well aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10002)
FOUR = ctypes.c_void_p(0x10004)
EIGHT = ctypes.c_void_p(0x10008)
BIG = 1 << 40
HUGE = (1 << 63) - 32              # a multiple of 32


@pytest.fixture(scope="module")
def lib():
    import fp8_precision_quantization_amd as mx
    from fp8_precision_quantization_amd import build
    if not os.path.exists(mx.LIB_PATH):
        build.build()
    return mx.lib()


def test_every_declared_symbol_is_exported_and_bound(lib):
    import fp8_precision_quantization_amd as mx
    from fp8_precision_quantization_amd import _fp4
    names = re.findall(r"MX_API\s+[\w\s\*]+?\b(mx_\w+)\s*\(", open(HEADER).read())
    assert sorted(names) == sorted(_fp4.SIGNATURES)
    for n in names:
        assert hasattr(lib, n) and hasattr(mx, n), n


def test_cast_validation(lib):
    def f(x=P, t=0, batch=2, rows=64, cols=64, ldx=64, q0=P, s0=P, q1=P, s1=P, blocked=0):
        return lib.mx_cast_mxfp4(x, t, batch, rows, cols, ldx, q0, s0, q1, s1, blocked, None)
    for bad in (dict(t=2), dict(batch=-1), dict(rows=-32), dict(cols=-32), dict(cols=48, ldx=48), dict(ldx=63),
                dict(rows=33), dict(ldx=(1 << 31) + 1), dict(rows=HUGE), dict(batch=HUGE), dict(cols=HUGE, ldx=HUGE),
                dict(batch=1 << 21, rows=128, cols=128, ldx=128), dict(batch=1, rows=1 << 28, cols=128, ldx=128),
                dict(batch=1 << 20, rows=97, cols=128, ldx=128, q1=None, s1=None)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(q0=None), dict(s0=None), dict(q1=None), dict(s1=None),
                dict(q0=None, s0=None, q1=None, s1=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(x=ODD), dict(t=1, x=HALF), dict(q0=HALF), dict(s0=ODD), dict(q1=EIGHT), dict(s1=HALF)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=0, x=None, q0=None, s0=None, q1=None, s1=None) == OK and f(batch=0) == OK and f(cols=0, ldx=0) == OK

    def g(q=P, s=P, batch=1, rows=33, cols=64, blocked=1, x=P, t=0):
        return lib.mx_dequantize_mxfp4(q, s, batch, rows, cols, blocked, x, t, None)
    for bad in (dict(t=-1), dict(batch=-1), dict(rows=-1), dict(cols=33), dict(rows=BIG), dict(batch=BIG, rows=128)):
        assert g(**bad) == SHAPE, bad
    for bad in (dict(q=None), dict(s=None), dict(x=None)):
        assert g(**bad) == NULL, bad
    assert g(q=HALF) == ALIGN and g(x=EIGHT) == ALIGN and g(rows=0, q=None) == OK


def test_gemm_validation(lib):
    def f(qa=P, sa=P, fa=1, qb=P, sb=P, m=8, n=8, k=64, c=P, t=0):
        return lib.mx_gemm_mxfp4(qa, sa, fa, qb, sb, m, n, k, c, t, None)

    def g(qa=P, sa=P, fa=0, qb=P, sb=P, ends=P, groups=2, m=8, n=8, k=64, c=P, t=1):
        return lib.mx_grouped_gemm_mxfp4(qa, sa, fa, qb, sb, ends, groups, m, n, k, c, t, None)
    for call in (f, g):
        for bad in (dict(fa=2), dict(fa=-1), dict(t=2), dict(m=-1), dict(n=-1), dict(k=-32), dict(k=48),
                    dict(k=(1 << 23) + 32), dict(n=1 << 14, k=1 << 22), dict(m=(1 << 31) - 1), dict(n=(1 << 24) + 1), dict(n=1 << 31),
                    dict(m=1 << 30, n=1 << 30), dict(m=1 << 30, n=1 << 30, k=32), dict(m=HUGE), dict(n=HUGE), dict(k=HUGE)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(qa=None), dict(sa=None), dict(qb=None), dict(sb=None), dict(c=None)):
            assert call(**bad) == NULL, bad
        for bad in (dict(qa=EIGHT), dict(sa=EIGHT), dict(qb=EIGHT), dict(sb=EIGHT), dict(c=ODD), dict(t=1, c=HALF)):
            assert call(**bad) == ALIGN, bad
        assert call(m=0, qa=None, c=None) == OK and call(n=0, c=None) == OK
    assert g(groups=0) == GROUPS and g(groups=1025) == GROUPS and g(ends=None) == NULL and g(ends=HALF) == ALIGN
    assert g(groups=1024, m=(1 << 31) - 1 - 256 * 1024) == SHAPE


def test_decode_validation(lib):
    def f(x=P, ldx=64, qw=P, sw=P, fw=1, m=8, n=8, k=64, c=P, t=0):
        return lib.mx_linear_decode(x, ldx, qw, sw, fw, m, n, k, c, t, None)

    def g(x=P, ldx=64, qw=P, sw=P, fw=0, m=8, n=8, k=64, c=P, act=0):
        return lib.mx_gated_ffn_decode(x, ldx, qw, sw, fw, m, n, k, act, c, None)
    for call in (f, g):
        for bad in (dict(fw=2), dict(m=-1), dict(m=65), dict(n=-1), dict(k=-32), dict(k=40), dict(ldx=63),
                    dict(ldx=BIG), dict(ldx=(1 << 28) + 1), dict(k=(1 << 23) + 32, ldx=1 << 24), dict(n=1 << 31), dict(n=HUGE),
                    dict(n=1 << 14, k=1 << 22, ldx=1 << 22)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(x=None), dict(qw=None), dict(sw=None), dict(c=None)):
            assert call(**bad) == NULL, bad
        for bad in (dict(x=ODD), dict(qw=EIGHT), dict(sw=EIGHT), dict(c=ODD)):
            assert call(**bad) == ALIGN, bad
        assert call(m=0, x=None, c=None) == OK and call(n=0, c=None) == OK
    assert f(t=3) == SHAPE and f(t=1, c=HALF) == ALIGN and g(act=2) == SHAPE and g(n=(1 << 30) + 1) == SHAPE


def test_ffn_validation(lib):
    def f(qx=P, sx=P, fx=0, qw=P, sw=P, fw=0, ends=None, groups=1, rows=8, cols=64, k=64, act=0, y=P, q=P, s=P):
        return lib.mx_gated_ffn(qx, sx, fx, qw, sw, fw, ends, groups, rows, cols, k, act, y, q, s, None)

    def g(qx=P, sx=P, fx=0, qw=P, sw=P, fw=0, ends=None, groups=1, rows=8, cols=64, k=64, act=0, y=P, q=P, s=P, dh=P):
        return lib.mx_gated_ffn_backward(qx, sx, fx, qw, sw, fw, ends, groups, rows, cols, k, act, q, s, dh, y, None)
    for call in (f, g):
        for bad in (dict(fx=2), dict(fw=-1), dict(fx=1, fw=0), dict(act=2), dict(rows=-1), dict(cols=-32), dict(cols=48),
                    dict(k=40), dict(k=-32), dict(k=(1 << 23) + 32), dict(rows=(1 << 31) - 1), dict(cols=1 << 31), dict(cols=(1 << 24) + 32),
                    dict(cols=HUGE), dict(rows=HUGE), dict(k=HUGE), dict(cols=1 << 14, k=1 << 22),
                    dict(rows=1 << 30, cols=1 << 24, k=32)):
            assert call(**bad) == SHAPE, bad
        assert call(groups=0) == call(groups=2) == call(ends=P, groups=1025) == GROUPS
        for bad in (dict(qx=None), dict(sx=None), dict(qw=None), dict(sw=None), dict(q=None), dict(s=None)):
            assert call(**bad) == NULL, bad
        for bad in (dict(qx=EIGHT), dict(sx=EIGHT), dict(qw=EIGHT), dict(sw=EIGHT), dict(ends=HALF), dict(y=EIGHT),
                    dict(q=EIGHT)):
            assert call(**bad) == ALIGN, bad
        assert call(rows=0, qx=None, y=None) == OK and call(cols=0, y=None, q=None, s=None) == OK
    assert f(y=None) == NULL and g(dh=None) == NULL and g(dh=EIGHT) == ALIGN
    assert f(cols=1 << 13, k=1 << 22) == SHAPE     # two halves


def test_binding_needs_gpu_tensors():
    import torch
    import fp8_precision_quantization_amd as mx
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    b, s = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((128, 4), dtype=torch.uint8)
    e = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mx.mx_cast_mxfp4(x), lambda: mx.mx_dequantize_mxfp4(b, s), lambda: mx.mx_gemm_mxfp4(b, s, b, s),
                 lambda: mx.mx_grouped_gemm_mxfp4(b, s, b[None], s, e), lambda: mx.mx_linear_decode(x, b, s),
                 lambda: mx.mx_gated_ffn_decode(x, b, s), lambda: mx.mx_gated_ffn(b, s, b, s),
                 lambda: mx.mx_gated_ffn_backward(b, s, b, s, b, s)):
        with pytest.raises(ValueError):
            call()
