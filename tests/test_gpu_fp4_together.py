"""The MXFP4 and gated feed-forward operators as they are used: one after the
other for serving and for a training step, captured in a HIP graph, on a
stream of the caller's, with scale layouts whose padding holds anything, and
calls that must be refused.

In a chain each operator is held against binary64 of what it was given, so that
the tolerances are those of the operators alone (tests/fp4_ref.py); casts are
compared byte for byte."""
import numpy as np
import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests import fp4_ref as r4
from tests import train_ref as ref
from tests.gpu_util import assert_bytes_equal, device, host, to_dev_u8

pytestmark = pytest.mark.gpu

REPLAYS = 4
MXFP4 = dict(a_format="mxfp4", w_format="mxfp4")


def _np(t):
    return t.detach().double().cpu().numpy()


def _normal(rng, dev, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dev).bfloat16()


def _cast4(oracle_mod, x):
    """The library's blocked cast of x along its rows, checked: (q, s, values)."""
    q, s, _, _ = mx.mx_cast_mxfp4(x, dim1=False, blocked=True, raw=True)
    codes, scales = r4.cast4(_np(x))
    assert_bytes_equal(host(q), r4.pack(codes), "codes")
    assert_bytes_equal(host(s).reshape(-1), oracle_mod.to_blocked(scales).reshape(-1), "scales")
    return q, s, r4.values4(codes, scales)


def _cast8(x, dim0=True, dim1=False):
    """(q_row, s_row, q_col, s_col), blocked, and the values along the rows or columns."""
    out = mx.mx_cast_dim0_dim1_blocked(x, dim0=dim0, dim1=dim1, raw=True)
    plain = mx.mx_cast_dim0_dim1(x, dim0=dim0, dim1=dim1, raw=True)
    i = 0 if dim0 else 2
    return out[i], out[i + 1], plain[i + 1], ref.values(host(plain[i]), host(plain[i + 1]))


def _close_product(got, a, w, fa, fw, bf16, what):
    want, mag = r4.product(a, w)
    tol = r4.product_error(mag, a.shape[1], fa, fw)
    ref.assert_close(_np(got), want, r4.round_tol(want, tol, bf16), what)


@pytest.mark.parametrize("rows,model,hidden", [(1, 64, 32), (33, 160, 96), (320, 288, 416)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_serving(rows, model, hidden, act, oracle_mod):
    """Weights once to MXFP4; a prompt in 4-bit products, and its first rows as
    single tokens."""
    dev = device()
    rng = np.random.default_rng([rows, model])
    x = _normal(rng, dev, rows, model)
    wg, wd = _normal(rng, dev, 2 * hidden, model, scale=model ** -0.5), _normal(rng, dev, model, hidden, scale=hidden ** -0.5)
    qg, sg, vg = _cast4(oracle_mod, wg)
    qd, sd, vd = _cast4(oracle_mod, wd)
    assert np.array_equal(_np(mx.mx_dequantize_mxfp4(qg, sg, blocked=True)), vg)
    qx, sx, vx = _cast4(oracle_mod, x)
    y, = mx.mx_gated_ffn(qx, sx, qg, sg, act=act, checkpoint=False, **MXFP4)
    h, mag = r4.product(vx, vg)
    want = r4.gated(h, act)
    eh = r4.product_error(mag, model, "e2m1", "e2m1")
    ref.assert_close(_np(y), want, r4.round_tol(want, r4.gated_tol(h, eh, act), True), "y")
    qy, sy, vy = _cast4(oracle_mod, y)
    _close_product(mx.mx_gemm_mxfp4(qy, sy, qd, sd), vy, vd, "e2m1", "e2m1", True, "out")
    if rows % 32 == 0:    # (what the 8-bit cast takes)
        q8, s8, _, v8 = _cast8(y)
        _close_product(mx.mx_gemm_mxfp4(q8, s8, qd, sd, out_dtype=torch.float32), v8, vd, "e4m3", "e2m1", False, "out 8")

    few = x[:min(rows, 5)]
    y = mx.mx_gated_ffn_decode(few, qg, sg, act=act)
    h, mag = r4.product(_np(few), vg)
    want = r4.gated(h, act)
    ref.assert_close(_np(y), want, r4.round_tol(want, r4.gated_tol(h, mag * model * 2.0 ** -24, act), True), "y of a few")
    out = mx.mx_linear_decode(y, qd, sd)
    want, mag = r4.product(_np(y), vd)
    ref.assert_close(_np(out), want, r4.round_tol(want, mag * hidden * 2.0 ** -24, True), "out of a few")


@pytest.mark.parametrize("rows,model,hidden", [(32, 64, 32), (320, 160, 96), (480, 416, 288)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_step(rows, model, hidden, act):
    """Both directions of the block, out = y Wd^T, in MXFP8: every product of the
    step against binary64 of its operands' values, and the gradient that the
    block's kernel forms against differences of the loss."""
    dev = device()
    rng = np.random.default_rng([rows, model, 1])
    x, dout = _normal(rng, dev, rows, model), _normal(rng, dev, rows, model)
    wg, wd = _normal(rng, dev, 2 * hidden, model, scale=model ** -0.5), _normal(rng, dev, model, hidden, scale=hidden ** -0.5)
    qx, sx, px, vx = _cast8(x)
    qg, sg, _, vg = _cast8(wg)
    y, q, s = mx.mx_gated_ffn(qx, sx, qg, sg, act=act, raw=True)
    h = ref.values(host(q), host(s))
    true_h, mag = r4.product(vx, vg)
    lo, hi, held = r4.checkpoint_range(true_h, r4.product_error(mag, model, "e4m3", "e4m3"))
    a, b = held(host(s))
    assert np.all((h >= a) & (h <= b))
    qy, sy, _, vy = _cast8(y)
    qd, sd, _, vd = _cast8(wd)
    _close_product(mx.mx_gemm_mxfp8(qy, sy, qd, sd), vy, vd, "e4m3", "e4m3", True, "out")

    # backward: dy through Wd's columns, the block's inside, and its weights and input
    qo, so, _, vo = _cast8(dout)
    qc, sc, _, vc = _cast8(wd, dim0=False, dim1=True)
    dh, again = mx.mx_gated_ffn_backward(qo, so, qc, sc, q, s, act=act, recompute=True)
    dy, mag = r4.product(vo, vc)
    edy = r4.product_error(mag, model, "e4m3", "e4m3")
    g, u = h[:, :hidden], h[:, hidden:]

    # differences of sum(dy act(g) u), element by element, over +-d: the third
    # derivative of act is below 3 and of act(g) u in u there is none, so the
    # difference is within d^2 / 2 |dy u| of the derivative, and binary64's
    # rounding of values below |dy u| (|g| + 1) over d adds 2^-50 / d of that.
    d = 2.0 ** -10
    slope_g = (ref.gated_act(g + d, u, act) - ref.gated_act(g - d, u, act)) / (2 * d)
    slope_u = (ref.gated_act(g, u + d, act) - ref.gated_act(g, u - d, act)) / (2 * d)
    got = _np(dh)
    for part, slope, size in ((got[:, :hidden], slope_g, np.abs(u)), (got[:, hidden:], slope_u, np.abs(g))):
        want = dy * slope
        t = np.minimum(np.abs(ref.gate_t(g, act)[0]), 200.0)
        # (an activation's slope is below 1.13 and its evaluation within (18 + 8 t) 2^-24 of the magnitudes 1 + |g|)
        rel = 2 * (18 + 8 * t) * ref.U32 * (1.13 + np.abs(g))
        tol = edy * 1.13 * size + (np.abs(dy) + edy) * size * (rel + d * d / 2 + 2.0 ** -50 / d * (1 + np.abs(g))) + 1e-30
        ref.assert_close(part, want, r4.round_tol(want, tol, True), "gradient against differences")
    want = ref.gated_act(g, u, act)
    t = np.minimum(np.abs(ref.gate_t(g, act)[0]), 200.0)
    ref.assert_close(_np(again), want, r4.round_tol(want, (18 + 8 * t) * ref.U32 * np.abs(want) + 1e-30, True), "y again")

    # dx = dh Wg through the columns of Wg; dWg = dh^T x from x's checkpoint
    qh, sh, _, vh = _cast8(dh)
    qgc, sgc, _, vgc = _cast8(wg, dim0=False, dim1=True)
    _close_product(mx.mx_gemm_mxfp8(qh, sh, qgc, sgc), vh, vgc, "e4m3", "e4m3", True, "dx")
    dw = mx.mx_wgrad_checkpoint(dh, qx, px)
    want, mag = _np(dh).T @ vx, np.abs(_np(dh)).T @ np.abs(vx)
    ref.assert_close(_np(dw), want, r4.round_tol(want, mag * (rows + 8) * ref.U32, False), "dW")


def _work(dev):
    """(fn, outputs): every operator, with its outputs given."""
    rng = np.random.default_rng(5)
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32

    def empty(*shape, dtype=u8):
        return torch.empty(*shape, dtype=dtype, device=dev)

    t, c, f, e = 512, 256, 128, 3
    x, w, wd = _normal(rng, dev, t, c), _normal(rng, dev, e, 2 * f, c, scale=1 / 16), _normal(rng, dev, e, c, f, scale=1 / 16)
    few = x[:9]
    ends = torch.tensor([100, 100, 470], dtype=i32, device=dev)
    ox = [empty(t, c // 2), empty(t, c // 32), empty(c, t // 2), empty(c, t // 32)]
    ow = [empty(e, 2 * f, c // 2), empty(e, 2 * f, c // 32)]
    od = [empty(e, c, f // 2), empty(e, c, f // 32), empty(e, f, c // 2), empty(e, 128, c // 32)]
    sxg = empty(t + 128 * e, c // 32)
    y, q, s = empty(t, f, dtype=bf), empty(t, 2 * f), empty(t, 2 * f // 32)
    dh, ya = empty(t, 2 * f, dtype=bf), empty(t, f, dtype=bf)
    one = [empty(t, f, dtype=bf), empty(t, 2 * f), empty(t, 2 * f // 32)]
    back, gm, gg = empty(t, c, dtype=f32), empty(t, 2 * f, dtype=f32), empty(t, 2 * f, dtype=bf)
    yd, zd = empty(9, f, dtype=bf), empty(9, c, dtype=f32)
    mm = [empty(t, c // 2), empty(t, c // 32)]

    def fn():
        mx.mx_cast_mxfp4(x, out=ox, raw=True)
        mx.mx_dequantize_mxfp4(ox[0], ox[1], out=back, out_dtype=f32)
        mx.mx_cast_mxfp4(x, dim1=False, blocked=True, out=mm + [None, None], raw=True)
        mx.mx_cast_mxfp4(w, dim1=False, blocked=True, out=ow + [None, None], raw=True)
        mx.mx_cast_mxfp4(wd, blocked=True, out=od, raw=True)
        mx.mx_scales_to_blocked_grouped(ox[1], ends, group_axis=0, out=sxg)
        mx.mx_gated_ffn(ox[0], sxg, ow[0], ow[1], group_end_offsets=ends, out=(y, q, s), raw=True, **MXFP4)
        mx.mx_gated_ffn_backward(ox[0], sxg, od[2], od[3], q, s, group_end_offsets=ends, recompute=True, out=(dh, ya),
                                 **MXFP4)
        mx.mx_gated_ffn(*mm, ow[0][1], ow[1][1], act="gelu", out=one, raw=True, **MXFP4)
        mx.mx_gemm_mxfp4(*mm, ow[0][2], ow[1][2], out=gm, out_dtype=f32)
        mx.mx_grouped_gemm_mxfp4(ox[0], sxg, ow[0], ow[1], ends, out=gg)
        mx.mx_gated_ffn_decode(few, ow[0][1], ow[1][1], out=yd)
        mx.mx_linear_decode(yd, od[0][1], od[1][1], out=zd, out_dtype=f32)

    return fn, ox + ow + od + [sxg, y, q, s, dh, ya] + one + [back, gm, gg, yd, zd] + mm


def _fill(outs):
    for o in outs:
        o.view(torch.uint8).fill_(0x3A)


def _same(outs, want, what):
    for i, (o, r) in enumerate(zip(outs, want)):
        assert torch.equal(o.view(torch.uint8), r), (what, i)


def test_graph_replays():
    """Captured once, replayed with eager work and synchronisations between:
    every replay, and every eager run after it, gives the same bytes, and those
    past the last group are left as they were."""
    dev = device()
    fn, outs = _work(dev)
    _fill(outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    side.synchronize()
    want = [o.view(torch.uint8).clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    for i in range(REPLAYS):
        _fill(outs)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _same(outs, want, "replay %d" % i)
        _fill(outs)
        fn()
        torch.cuda.synchronize()
        _same(outs, want, "eager after replay %d" % i)


def test_two_streams_at_once():
    """Two streams' calls, neither waiting for the other, and inputs that a long
    queue on the caller's own stream writes last."""
    dev = device()
    rng = np.random.default_rng(2)
    final = [_normal(rng, dev, 2048, 512) for _ in range(2)]
    w = [_normal(rng, dev, 1024, 512, scale=1 / 16) for _ in range(2)]
    x = [torch.zeros_like(f) for f in final]

    def fn(x, w):
        qx, sx, _, _ = mx.mx_cast_mxfp4(x, dim1=False, blocked=True, raw=True)
        qw, sw, _, _ = mx.mx_cast_mxfp4(w, dim1=False, blocked=True, raw=True)
        return mx.mx_gated_ffn(qx, sx, qw, sw, raw=True, **MXFP4) + (mx.mx_gemm_mxfp4(qx, sx, qw, sw),
                                                                    mx.mx_gated_ffn_decode(x[:40], qw, sw))

    want = [fn(f, v) for f, v in zip(final, w)]
    big = [torch.randn(4096, 4096, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    sides, got = [torch.cuda.Stream() for _ in range(2)], []
    for i, side in enumerate(sides):
        with torch.cuda.stream(side):
            for _ in range(4):
                big[i] = (big[i] @ big[i]).clamp(-1, 1)
            x[i].copy_(final[i])
            got.append(fn(x[i], w[i]))
    for side in sides:
        side.synchronize()
    for a, b in zip(got, want):
        for o, r in zip(a, b):
            assert torch.equal(o, r)


@pytest.mark.parametrize("k", [32, 64, 96, 160, 416])
@pytest.mark.parametrize("fa", ["e2m1", "e4m3"])
def test_padding_of_scale_layouts_is_not_read(k, fa, oracle_mod):
    """Bytes of the layouts that belong to no block, NaN scales among them, do
    not reach a result."""
    dev = device()
    m, n = 40, 96
    rng = np.random.default_rng(k)
    (qa, sa), (qb, sb) = r4.operand(rng, m, k, fa), r4.operand(rng, n, k, "e2m1")
    kept_q, kept_s = rng.integers(0, 120, (m, 2 * n)), rng.integers(118, 122, (m, n // 16))

    def layout(s, fill):
        full = np.full(((s.shape[0] + 127) // 128 * 128, (s.shape[1] + 3) // 4 * 4), fill, np.uint8)
        full[:s.shape[0], :s.shape[1]] = s
        return to_dev_u8(oracle_mod.to_blocked(full), dev)

    x = _normal(rng, dev, 7, k)
    a_format = {"e2m1": "mxfp4", "e4m3": "mxfp8"}[fa]
    results = []
    for fill in (0, 255):
        a, b = (to_dev_u8(qa, dev), layout(sa, fill)), (to_dev_u8(qb, dev), layout(sb, fill))
        f = dict(a_format=a_format, w_format="mxfp4")
        results.append((mx.mx_gemm_mxfp4(*a, *b), *mx.mx_gated_ffn(*a, b[0][:64], layout(sb[:64], fill), raw=True, **f),
                        *mx.mx_gated_ffn_backward(*a, *b, to_dev_u8(kept_q, dev), to_dev_u8(kept_s, dev), **f),
                        mx.mx_linear_decode(x, *b), mx.mx_gated_ffn_decode(x, *b),
                        mx.mx_dequantize_mxfp4(*b, blocked=True)))
        if fa == "e4m3":
            both = (a[0][:32].repeat(2, 1), layout(np.tile(sa[:32], (2, 1)), fill))
            results[-1] += (mx.mx_linear_decode(x, *a), *mx.mx_gated_ffn(*a, *both, checkpoint=False))
    for i, (o, r) in enumerate(zip(*results)):
        assert not torch.isnan(o.float()).any() and torch.equal(o, r), i


def test_refusals():
    """Shapes, formats, sizes of scales and devices that do not fit."""
    dev = device()

    def u8(*shape):
        return torch.zeros(*shape, dtype=torch.uint8, device=dev)

    x = torch.zeros(64, 64, dtype=torch.bfloat16, device=dev)
    s, half = u8(128, 4), u8(64, 32)
    ends = torch.zeros(1, dtype=torch.int32, device=dev)
    e4 = u8(64, 64).view(torch.float8_e4m3fn)
    gs = u8((64 + 128) * 4)
    good = [lambda: mx.mx_gemm_mxfp4(half, s, half, s), lambda: mx.mx_gated_ffn(half, s, half, s, **MXFP4),
            lambda: mx.mx_gated_ffn_backward(half, s, half, s, u8(64, 128), u8(64, 4), **MXFP4),
            lambda: mx.mx_grouped_gemm_mxfp4(half, gs, half[None], s, ends), lambda: mx.mx_linear_decode(x, half, s),
            lambda: mx.mx_gated_ffn_decode(x, half, s), lambda: mx.mx_gemm_mxfp4(e4, s, half, s)]
    for call in good:
        call()
    bad = [lambda: mx.mx_cast_mxfp4(x.half()), lambda: mx.mx_cast_mxfp4(x[:, :48]), lambda: mx.mx_cast_mxfp4(x[:40]),
           lambda: mx.mx_cast_mxfp4(x, dim0=False, dim1=False), lambda: mx.mx_cast_mxfp4(x[None, :, :32]),
           lambda: mx.mx_cast_mxfp4(x, out=(u8(64, 31), None, None, None)), lambda: mx.mx_cast_mxfp4(x.t()),
           lambda: mx.mx_dequantize_mxfp4(e4, u8(64, 2)), lambda: mx.mx_dequantize_mxfp4(half, u8(64, 3)),
           lambda: mx.mx_dequantize_mxfp4(half, u8(64, 2), blocked=True),
           lambda: mx.mx_dequantize_mxfp4(half, u8(64, 2), out_dtype=torch.float16),
           lambda: mx.mx_gemm_mxfp4(half, s, e4, s), lambda: mx.mx_gemm_mxfp4(half, u8(127, 4), half, s),
           lambda: mx.mx_gemm_mxfp4(half, s, half, u8(128, 8)), lambda: mx.mx_gemm_mxfp4(u8(64, 48), s, half, s),
           lambda: mx.mx_gemm_mxfp4(half, s, half, s, out_dtype=torch.float16),
           lambda: mx.mx_gemm_mxfp4(half, s, half, s, out=x[:32]), lambda: mx.mx_gemm_mxfp4(half, s, half.cpu(), s),
           lambda: mx.mx_gemm_mxfp4(half.t(), s, half, s), lambda: mx.mx_gemm_mxfp4(half, s, half[:, :24], s),
           lambda: mx.mx_grouped_gemm_mxfp4(half, s, half[None], s, ends),
           lambda: mx.mx_grouped_gemm_mxfp4(half, gs, half[None], s, ends.long()),
           lambda: mx.mx_grouped_gemm_mxfp4(half, gs, half[None], s, ends.repeat(2)),
           lambda: mx.mx_grouped_gemm_mxfp4(half, gs, half[None], s, ends.cpu()),
           lambda: mx.mx_linear_decode(torch.cat([x, x]), half, s), lambda: mx.mx_linear_decode(x.float(), half, s),
           lambda: mx.mx_linear_decode(x[:, :40], half, s), lambda: mx.mx_linear_decode(x.t(), half, s),
           lambda: mx.mx_gated_ffn_decode(x, half[:63], s), lambda: mx.mx_gated_ffn_decode(x, half, s, act="relu"),
           lambda: mx.mx_gated_ffn(half, s, half, s, a_format="mxfp4"),
           lambda: mx.mx_gated_ffn(e4, s, half, s, **MXFP4), lambda: mx.mx_gated_ffn(half, s, half[:32], s, **MXFP4),
           lambda: mx.mx_gated_ffn(half, s, half, s, a_format="fp4", w_format="mxfp4"),
           lambda: mx.mx_gated_ffn(half, s, half, s, act="tanh", **MXFP4),
           lambda: mx.mx_gated_ffn(half, s, half, s, out=(x,), **MXFP4),
           lambda: mx.mx_gated_ffn(half, s, half[None], s, **MXFP4),
           lambda: mx.mx_gated_ffn_backward(half, s, half, s, u8(64, 64), u8(64, 4), **MXFP4),
           lambda: mx.mx_gated_ffn_backward(half, s, half, s, u8(64, 128), u8(64, 2), **MXFP4),
           lambda: mx.mx_gated_ffn_backward(half, s, half[:48], s, u8(64, 96), u8(64, 3), **MXFP4)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            call()
            pytest.fail("call %d was taken" % i)


def test_offsets_past_32_bits(oracle_mod):
    """Rows of codes, results and checkpoints that lie more than 2^32 bytes from
    the first: the last rows of long operands, against the same rows alone."""
    dev = device()
    rng = np.random.default_rng(4)
    rows, k, f = 1 << 21, 64, 1056          # y 4.4e9 bytes, the checkpoint as many
    qx = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device=dev)
    sx = torch.full((rows, 4), 126, dtype=torch.uint8, device=dev)
    wq, ws = r4.operand(rng, 2 * f, k, "e2m1", spread=1)
    w = (to_dev_u8(wq, dev), to_dev_u8(oracle_mod.to_blocked(ws), dev))
    tail = rows - 256
    y, q, s = mx.mx_gated_ffn(qx, sx, *w, raw=True, **MXFP4)
    few = mx.mx_gated_ffn(qx[tail:].clone(), sx[:256], *w, raw=True, **MXFP4)
    for a, b in zip((y[tail:], q[tail:], s[tail:]), few):
        assert torch.equal(a, b)
    c = mx.mx_gemm_mxfp4(qx, sx, *w, out=torch.empty(rows, 2 * f, dtype=torch.bfloat16, device=dev))
    assert torch.equal(c[tail:], mx.mx_gemm_mxfp4(qx[tail:].clone(), sx[:256], *w))
    # the gradient reads the checkpoint of those rows
    wd = (w[0][:f].clone(), to_dev_u8(oracle_mod.to_blocked(ws[:f]), dev))
    dh, = mx.mx_gated_ffn_backward(qx, sx, *wd, q, s, out=(c,), **MXFP4)
    only, = mx.mx_gated_ffn_backward(qx[tail:].clone(), sx[:256], *wd, q[tail:].clone(), s[tail:].clone(), **MXFP4)
    assert torch.equal(dh[tail:], only)
    # and the cast of as many elements, both directions
    c0 = mx.mx_cast_mxfp4(c, dim1=False, raw=True)
    want = mx.mx_cast_mxfp4(c[tail:].clone(), dim1=False, raw=True)
    assert torch.equal(c0[0][tail:], want[0]) and torch.equal(c0[1][tail:], want[1])
    back = mx.mx_dequantize_mxfp4(c0[0], c0[1], out=c)
    assert torch.equal(back[tail:], mx.mx_dequantize_mxfp4(want[0], want[1]))
