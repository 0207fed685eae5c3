"""The second half of the C ABI (include/mxtrain.h) on a machine without a
GPU: every declared symbol is exported and bound, and bad arguments are
rejected on the host before any HIP call."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxtrain.h")

OK, NULL, SHAPE, GROUPS, HIP, ALIGN, WORKSPACE = range(7)
P = ctypes.c_void_p(0x10000)       # well aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10002)    # aligned for bf16 only
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import fp8_precision_quantization_amd as mx
    from fp8_precision_quantization_amd import build
    if not os.path.exists(mx.LIB_PATH):
        build.build()
    return mx.lib()


def test_every_declared_symbol_is_exported_and_bound(lib):
    import fp8_precision_quantization_amd as mx
    from fp8_precision_quantization_amd import _train
    names = re.findall(r"MX_API\s+[\w\s\*]+?\b(mx_\w+)\s*\(", open(HEADER).read())
    assert sorted(names) == sorted(_train.SIGNATURES)
    for n in names:
        assert hasattr(lib, n) and hasattr(mx, n), n


def test_layernorm_validation(lib):
    def f(x=P, ldx=64, xt=0, w=P, b=P, wt=1, rows=4, cols=64, y=P, mean=P, rstd=P, q=None, s=None):
        return lib.mx_layernorm(x, ldx, xt, w, b, wt, rows, cols, 1e-5, y, mean, rstd, q, s, None)
    for bad in (dict(xt=2), dict(wt=-1), dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(ldx=63),
                dict(cols=16385, ldx=16385), dict(ldx=(1 << 31) + 1), dict(cols=48, q=P, s=P), dict(xt=1, q=P, s=P)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(q=P), dict(s=P)):
        assert f(**bad) == NULL, bad
    for bad in (dict(x=ODD), dict(y=ODD), dict(w=HALF), dict(b=HALF), dict(mean=HALF), dict(rstd=HALF),
                dict(xt=1, x=HALF), dict(q=ctypes.c_void_p(0x10004), s=P), dict(x=HALF, q=P, s=P),
                dict(ldx=65, q=P, s=P)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=0, x=None, w=None, y=None, mean=None, rstd=None) == OK
    assert f(cols=0, ldx=0) == OK


def test_layernorm_backward_validation(lib):
    ws = lib.mx_layernorm_backward_workspace_bytes
    assert ws(-1, 64) == ws(4, -1) == ws(4, 16385) == ws(1 << 31, 64) == -1
    assert ws(0, 64) == 0 and ws(4, 64) == 4 * 64 * 8 and ws(1 << 20, 64) == ws(1 << 21, 64)

    def f(dy=P, lddy=64, x=P, ldx=64, xt=0, w=P, wt=1, mean=P, rstd=P, rows=4, cols=64, dx=P, dw=P, db=P, work=P,
          nbytes=1 << 20):
        return lib.mx_layernorm_backward(dy, lddy, x, ldx, xt, w, wt, mean, rstd, rows, cols, dx, dw, db, work, nbytes,
                                         None)
    for bad in (dict(lddy=63), dict(lddy=BIG), dict(ldx=8), dict(xt=7), dict(rows=-4), dict(cols=20000, ldx=20000)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dx=None),
                dict(dw=None), dict(work=None), dict(rows=0, dw=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(dy=ODD), dict(dx=ODD), dict(dw=HALF), dict(db=HALF), dict(work=ctypes.c_void_p(0x10008))):
        assert f(**bad) == ALIGN, bad
    assert f(nbytes=4 * 64 * 8 - 1) == WORKSPACE
    assert f(cols=0, lddy=0, ldx=0, dw=None) == OK


def test_router_validation(lib):
    ws = lib.mx_router_workspace_bytes
    assert ws(-1, 8) == ws(8, 0) == ws(8, 1025) == ws(1 << 31, 8) == -1
    assert ws(0, 8) == 0 and ws(1, 1024) == 0 and ws(1 << 20, 256) == 256 * (8 * 256 + 4)

    def f(z=P, ld=16, t=1, valid=None, rows=4, experts=16, topk=2, align=1, chosen=P, gates=P, lse=P, counts=P, ends=P,
          balance=P, loss=P, work=P, nbytes=1 << 24):
        return lib.mx_router_balance(z, ld, t, valid, rows, experts, topk, 0, align, chosen, gates, lse, counts, ends,
                                     balance, loss, work, nbytes, None)
    assert f(experts=0) == GROUPS and f(experts=1025, ld=1025) == GROUPS
    for bad in (dict(t=2), dict(ld=15), dict(rows=-1), dict(topk=0), dict(topk=17), dict(align=0),
                dict(experts=64, ld=64, topk=33), dict(rows=1 << 30), dict(align=1 << 30), dict(ld=BIG)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(z=None), dict(chosen=None), dict(gates=None), dict(lse=None), dict(counts=None), dict(ends=None),
                dict(balance=None), dict(loss=None), dict(rows=100000, work=None), dict(rows=0, loss=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(z=HALF), dict(chosen=HALF), dict(loss=ODD), dict(work=ctypes.c_void_p(0x10004))):
        assert f(**bad) == ALIGN, bad
    assert f(rows=100000, nbytes=64) == WORKSPACE

    def g(z=P, ld=16, t=1, lse=P, chosen=P, gates=P, balance=P, dg=P, dl=P, rows=4, experts=16, topk=2, out=P):
        return lib.mx_router_balance_backward(z, ld, t, lse, chosen, gates, balance, dg, dl, rows, experts, topk, 0,
                                              out, None)
    assert g(experts=2000, ld=2000) == GROUPS
    assert g(topk=20) == SHAPE and g(ld=3) == SHAPE and g(t=5) == SHAPE and g(rows=-1) == SHAPE
    for bad in (dict(z=None), dict(lse=None), dict(chosen=None), dict(gates=None), dict(balance=None), dict(out=None)):
        assert g(**bad) == NULL, bad
    for bad in (dict(z=HALF), dict(out=HALF), dict(dg=ODD), dict(dl=HALF)):
        assert g(**bad) == ALIGN, bad
    assert g(rows=0, z=None, out=None) == OK


def test_gated_act_validation(lib):
    def f(h=P, rows=4, cols=64, act=0, y=P, q=P, s=P):
        return lib.mx_gated_act(h, rows, cols, act, y, q, s, None)

    def g(dy=P, q=P, s=P, rows=4, cols=64, act=0, dh=P, y=None):
        return lib.mx_gated_act_backward(dy, q, s, rows, cols, act, dh, y, None)
    for call in (f, g):
        for bad in (dict(rows=-1), dict(cols=-32), dict(cols=48), dict(act=2), dict(rows=BIG, cols=BIG),
                    dict(rows=(1 << 62), cols=1 << 62), dict(rows=1 << 20, cols=1 << 15)):
            assert call(**bad) == SHAPE, bad
    for bad in (dict(h=None), dict(y=None), dict(q=None), dict(s=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(dy=None), dict(q=None), dict(s=None), dict(dh=None)):
        assert g(**bad) == NULL, bad
    eight = ctypes.c_void_p(0x10008)
    assert f(h=eight) == ALIGN and f(y=eight) == ALIGN and f(q=ctypes.c_void_p(0x10004)) == ALIGN
    assert g(dy=eight) == ALIGN and g(dh=eight) == ALIGN and g(y=eight) == ALIGN and g(q=ODD) == ALIGN
    assert f(rows=0, h=None, y=None) == OK and g(cols=0, dy=None) == OK


def test_wgrad_validation(lib):
    ws = lib.mx_wgrad_checkpoint_workspace_bytes
    assert ws(-1, 8, 32, 1) == ws(8, -1, 32, 1) == ws(8, 8, 33, 1) == ws(8, 8, 32, 0) == ws(8, 8, 32, 1025) == -1
    assert ws(8, 8, 32, 1) == 0 and ws(0, 0, 0, 1) == 0 and ws(100000, 64, 64, 1) > 0

    def f(dy=P, lddy=64, q=P, s=P, rows=8, n=64, k=64, ends=None, groups=1, dw=P, t=1, work=P, nbytes=1 << 30):
        return lib.mx_wgrad_checkpoint(dy, lddy, q, s, rows, n, k, ends, groups, dw, t, work, nbytes, None)
    for bad in (dict(rows=-1), dict(rows=(1 << 31) - 512), dict(n=-1), dict(k=48), dict(lddy=63), dict(t=2),
                dict(k=(1 << 22) + 32), dict(n=(1 << 22) + 1, lddy=1 << 23), dict(lddy=(1 << 22) + 1)):
        assert f(**bad) == SHAPE, bad
    assert f(groups=0) == GROUPS and f(groups=2) == GROUPS and f(ends=P, groups=1025) == GROUPS
    assert f(ends=P, groups=1024, n=1 << 22, lddy=1 << 22, k=1 << 22) == SHAPE    # too many tiles for a launch
    for bad in (dict(dy=None), dict(q=None), dict(s=None), dict(dw=None), dict(rows=100000, work=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(dy=ODD), dict(q=ctypes.c_void_p(0x10008)), dict(dw=HALF), dict(ends=HALF), dict(work=ODD)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=100000, nbytes=16) == WORKSPACE
    assert f(n=0, dy=None, dw=None) == OK and f(k=0, q=None, dw=None) == OK


def test_binding_needs_gpu_tensors():
    import torch
    import fp8_precision_quantization_amd as mx
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    v = torch.zeros(4)
    b = torch.zeros((4, 64), dtype=torch.uint8)
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: mx.mx_layernorm(x, x[0]), lambda: mx.mx_layernorm_backward(x, x, x[0], v, v),
                 lambda: mx.mx_router_balance(x, 2), lambda: mx.mx_router_balance_backward(x, v, i, v, v),
                 lambda: mx.mx_gated_act(x), lambda: mx.mx_gated_act_backward(x, b, b),
                 lambda: mx.mx_wgrad_checkpoint(x, b, b)):
        with pytest.raises(ValueError):
            call()
