"""ctypes binding of the third part of libmxcast (include/mxfp4.h): the MXFP4
cast, products with MXFP4 weights and the gated feed-forward block on MX
operands.

Argument marshalling only, as in _binding and _train: shapes and dtypes are
checked, outputs are allocated with torch, every call goes to the C ABI on
torch's current stream of the inputs' device, and there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import MX_BLOCK, MX_MAX_GROUPS, _pad, lib
from ._train import _TYPES, _act, _bytes, _call, _gpu, _matrix, _new, _new_bytes, _outs, _p, _same_device, _typed

MX_MAX_DECODE_ROWS = 64
FORMATS = {"mxfp8": 0, "mxfp4": 1}

# Types that codes come in, with the format that they say (None: bytes, of either
# format), and those of scales.  (Looked up, not asked: 0.2 us of a call's 10.)
_CODES = {torch.float8_e4m3fn: 0, torch.uint8: None, torch.int8: None, torch.bool: None}
_SCALES = {torch.float8_e8m0fnu, torch.uint8, torch.int8, torch.bool}
_FP4 = getattr(torch, "float4_e2m1fn_x2", None)   # two codes to an element, as stored here
if _FP4 is not None:
    _CODES[_FP4] = 1


def _code_type(t, name):
    """The format that a dtype says (None: bytes)."""
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise ValueError("%s must hold e4m3 or e2m1 codes or bytes, got %s" % (name, t.dtype)) from None


def _codes(t, fmt, name, ndim=2):
    """(tensor, format, rows.., k) of an operand's codes; fmt None: by dtype,
    MXFP4 for plain bytes."""
    _gpu(t, name)
    if t.dim() != ndim or not t.is_contiguous() or t.element_size() != 1:
        raise ValueError("%s must be a contiguous one-byte tensor of %d dimensions" % (name, ndim))
    own = _code_type(t, name)
    if fmt is None:
        f = 1 if own is None else own
    elif fmt in FORMATS:
        f = FORMATS[fmt]
        if own is not None and own != f:
            raise ValueError("%s holds %s, not %s" % (name, t.dtype, fmt))
    else:
        raise ValueError("a format must be one of %s" % ", ".join(sorted(FORMATS)))
    k = t.shape[-1] * (2 if f else 1)
    if k % MX_BLOCK:
        raise ValueError("%s must hold a multiple of %d elements a row" % (name, MX_BLOCK))
    return f, k


def _scale_type(s, name):
    if s.dtype not in _SCALES:
        raise ValueError("%s must hold e8m0 scales or bytes, got %s" % (name, s.dtype))


def _blocked_scales(s, nbytes, name):
    _gpu(s, name)
    if s.element_size() != 1 or not s.is_contiguous():
        raise ValueError("%s must be a contiguous one-byte tensor" % name)
    _scale_type(s, name)
    if s.numel() != nbytes:
        raise ValueError("%s: %d bytes of blocked scales expected, got %d" % (name, nbytes, s.numel()))


def _blocked_numel(rows, k):
    return _pad(rows, 128) * _pad(k // MX_BLOCK, 4)


def _ends(offs):
    _typed(offs, (torch.int32,), "group_end_offsets")
    if offs.dim() != 1 or not offs.is_contiguous():
        raise ValueError("group_end_offsets must be a contiguous vector")
    if not 1 <= offs.numel() <= MX_MAX_GROUPS:
        raise ValueError("1 to %d groups" % MX_MAX_GROUPS)
    return offs.numel()


def _out_type(dtype):
    if dtype not in _TYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    return _TYPES[dtype]


def _views(q, s, raw):
    if raw or q is None:
        return q, s
    return q if _FP4 is None else q.view(_FP4), s.view(torch.float8_e8m0fnu)


def mx_cast_mxfp4(x, dim0: bool = True, dim1: bool = True, blocked: bool = False, out=None, raw: bool = False):
    """(R, C) or (B, R, C) of bf16 or float32 -> MXFP4: (q_row (.., R, C / 2),
    s_row (.., R, C / 32), q_col (.., C, R / 2), s_col (.., C, R / 32)), two
    codes to a byte, the column cast a row for each column.  With blocked each
    matrix's scales are in the 128x4 blocked layout, (.., ceil128(R), ceil4(C /
    32)) and (.., ceil128(C), ceil4(R / 32)).  C a multiple of 32, and R with
    dim1; rows of a 2D x may lie any distance apart.  A direction turned off
    returns None for its pair.  `out` may hold preallocated uint8 outputs in
    that order.  float4_e2m1fn_x2 / e8m0 views, or uint8 if raw."""
    _typed(x, (torch.bfloat16, torch.float32), "x")
    if x.dim() == 3:
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        lead, ldx = (x.shape[0],), x.shape[2]
    else:
        lead, ldx = (), _matrix(x, "x")[2]
    rows, cols = x.shape[-2:]
    if cols % MX_BLOCK or (dim1 and rows % MX_BLOCK):
        raise ValueError("x must have a multiple of %d columns%s" % (MX_BLOCK, " and rows" if dim1 else ""))
    if not dim0 and not dim1:
        raise ValueError("dim0 or dim1 must be asked for")
    o, dev = _outs(out, 4), x.device

    def pair(i, r, c, names):
        scales = (_pad(r, 128), _pad(c // MX_BLOCK, 4)) if blocked else (r, c // MX_BLOCK)
        return (_new_bytes(o[i], lead + (r, c // 2), dev, names[0]),
                _new_bytes(o[i + 1], lead + scales, dev, names[1]))

    q0, s0 = pair(0, rows, cols, ("q_row", "s_row")) if dim0 else (None, None)
    q1, s1 = pair(2, cols, rows, ("q_col", "s_col")) if dim1 else (None, None)
    _call("mx_cast_mxfp4", dev, x.data_ptr(), _TYPES[x.dtype], lead[0] if lead else 1, rows, cols, ldx, _p(q0), _p(s0),
          _p(q1), _p(s1), int(blocked))
    return _views(q0, s0, raw) + _views(q1, s1, raw)


def mx_dequantize_mxfp4(q, s, blocked: bool = False, out_dtype=torch.bfloat16, out=None):
    """The values of an MXFP4 cast: (R, C) or (B, R, C), bf16 or float32, from
    codes (.., R, C / 2) and scales, plain or in the blocked layout.  Exact."""
    _gpu(q, "q")
    if q.dim() not in (2, 3):
        raise ValueError("q must have 2 or 3 dimensions")
    fmt, cols = _codes(q, None, "q", q.dim())
    if not fmt:
        raise ValueError("q must hold MXFP4 codes")
    lead, rows = tuple(q.shape[:-2]), q.shape[-2]
    batch = lead[0] if lead else 1
    if blocked:
        _blocked_scales(s, batch * _blocked_numel(rows, cols), "s")
    else:
        _bytes(s, lead + (rows, cols // MX_BLOCK), "s")
        _scale_type(s, "s")
    _same_device(q.device, s=s)
    code = _out_type(out_dtype)
    x = _new(out, lead + (rows, cols), out_dtype, q.device, "out")
    _call("mx_dequantize_mxfp4", q.device, q.data_ptr(), s.data_ptr(), batch, rows, cols, int(blocked), x.data_ptr(),
          code)
    return x


def _a_operand(qa, k, name):
    """Format of A's codes: MXFP4 or MXFP8 by the bytes of a row."""
    _gpu(qa, name)
    if qa.dim() != 2 or qa.shape[1] not in (k, k // 2):
        raise ValueError("%s: codes (M, %d) of MXFP8 or (M, %d) of MXFP4 expected" % (name, k, k // 2))
    fmt = "mxfp8" if qa.shape[1] == k and (k or qa.dtype == torch.float8_e4m3fn) else "mxfp4"
    return _codes(qa, fmt, name)[0]


def mx_gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None):
    """C (M, N) = A @ B^T with MXFP4 weights B: qb (N, K / 2) codes, sb the
    blocked layout of their (N, K / 32) scales; qa (M, K / 2) MXFP4 or (M, K)
    MXFP8 codes with sa likewise."""
    fb, k = _codes(qb, "mxfp4", "B")
    fa = _a_operand(qa, k, "A")
    m, n, dev = qa.shape[0], qb.shape[0], qa.device
    _blocked_scales(sa, _blocked_numel(m, k), "A")
    _blocked_scales(sb, _blocked_numel(n, k), "B")
    _same_device(dev, sa=sa, qb=qb, sb=sb)
    code = _out_type(out_dtype)
    c = _new(out, (m, n), out_dtype, dev, "out")
    _call("mx_gemm_mxfp4", dev, qa.data_ptr(), sa.data_ptr(), fa, qb.data_ptr(), sb.data_ptr(), m, n, k, c.data_ptr(),
          code)
    return c


def mx_grouped_gemm_mxfp4(qa, sa, qb, sb, group_end_offsets, out_dtype=torch.bfloat16, out=None):
    """Grouped along M: rows of group g of A times group g's weights.  sa is
    the M-grouped blocked layout of A's scales (mx_scales_to_blocked_grouped
    with group_axis 0), qb (G, N, K / 2) the weights' codes and sb the G blocked
    layouts of their scales one after another; offsets int32 [G] on the device.
    Rows past the last end are left as they were in `out`."""
    _, k = _codes(qb, "mxfp4", "B", 3)
    fa = _a_operand(qa, k, "A")
    groups = _ends(group_end_offsets)
    if groups != qb.shape[0]:
        raise ValueError("one offset per group of B")
    m, n, dev = qa.shape[0], qb.shape[1], qa.device
    _blocked_scales(sa, (m + 128 * groups) * _pad(k // MX_BLOCK, 4), "A")
    _blocked_scales(sb, groups * _blocked_numel(n, k), "B")
    _same_device(dev, sa=sa, qb=qb, sb=sb, group_end_offsets=group_end_offsets)
    code = _out_type(out_dtype)
    c = _new(out, (m, n), out_dtype, dev, "out")
    _call("mx_grouped_gemm_mxfp4", dev, qa.data_ptr(), sa.data_ptr(), fa, qb.data_ptr(), sb.data_ptr(),
          group_end_offsets.data_ptr(), groups, m, n, k, c.data_ptr(), code)
    return c


def _decode_operands(x, qw, sw):
    """Checked (m, ldx, k, format, rows of W) of the decode forms."""
    _typed(x, (torch.bfloat16,), "x")
    m, k, ldx = _matrix(x, "x")
    if m > MX_MAX_DECODE_ROWS:
        raise ValueError("x must have at most %d rows" % MX_MAX_DECODE_ROWS)
    fmt = _a_operand(qw, k, "W")
    n = qw.shape[0]
    _blocked_scales(sw, _blocked_numel(n, k), "W")
    _same_device(x.device, qw=qw, sw=sw)
    return m, ldx, k, fmt, n


def mx_linear_decode(x, qw, sw, out_dtype=torch.bfloat16, out=None):
    """x @ W^T (M, N) of a few bf16 rows x (M, K), M at most 64, with weights
    held in MXFP4, qw (N, K / 2), or MXFP8, qw (N, K); sw their blocked scales.
    x is not rounded.  Rows of x may lie any distance apart."""
    m, ldx, k, fmt, n = _decode_operands(x, qw, sw)
    code = _out_type(out_dtype)
    c = _new(out, (m, n), out_dtype, x.device, "out")
    _call("mx_linear_decode", x.device, x.data_ptr(), ldx, qw.data_ptr(), sw.data_ptr(), fmt, m, n, k, c.data_ptr(),
          code)
    return c


def mx_gated_ffn_decode(x, qw, sw, act: str = "silu", out=None):
    """act(x Wg^T) * (x Wu^T), bf16 (M, F), of a few bf16 rows x (M, K), M at
    most 64; qw holds Wg's F rows and then Wu's, as for mx_linear_decode."""
    code = _act(act)
    m, ldx, k, fmt, n = _decode_operands(x, qw, sw)
    if n % 2:
        raise ValueError("W must hold a gate and a factor half")
    y = _new(out, (m, n // 2), torch.bfloat16, x.device, "out")
    _call("mx_gated_ffn_decode", x.device, x.data_ptr(), ldx, qw.data_ptr(), sw.data_ptr(), fmt, m, n // 2, k, code,
          y.data_ptr())
    return y


def _ffn_operands(qx, sx, qw, sw, group_end_offsets, formats, halves, name):
    """Checked (rows, F, k, formats, groups) of the block's operands."""
    groups = 0 if group_end_offsets is None else _ends(group_end_offsets)
    fx, k = _codes(qx, formats[0], name)
    fw, kw = _codes(qw, formats[1], "W", 3 if groups else 2)
    if (fx, fw) == (1, 0):
        raise ValueError("MXFP4 %s goes with MXFP4 weights" % name)
    if k != kw:
        raise ValueError("%s and W must have rows of one length" % name)
    if groups and groups != qw.shape[0]:
        raise ValueError("one offset per group of W")
    rows, n = qx.shape[0], qw.shape[-2]
    if n % (halves * MX_BLOCK):
        raise ValueError("W must have a multiple of %d rows" % (halves * MX_BLOCK))
    if groups:
        _blocked_scales(sx, (rows + 128 * groups) * _pad(k // MX_BLOCK, 4), name)
    else:
        _blocked_scales(sx, _blocked_numel(rows, k), name)
    _blocked_scales(sw, max(1, groups) * _blocked_numel(n, k), "W")
    _same_device(qx.device, sx=sx, qw=qw, sw=sw, group_end_offsets=group_end_offsets)
    return rows, n // halves, k, fx, fw, max(1, groups)


def mx_gated_ffn(qx, sx, qw, sw, act: str = "silu", checkpoint: bool = True, group_end_offsets=None,
                 a_format: str = "mxfp8", w_format: str = "mxfp8", out=None, raw: bool = False):
    """act(x Wg^T) * (x Wu^T) on MX operands in one kernel, bf16 (R, F): (y,),
    or with checkpoint (y, q, s) with the 8-bit checkpoint of both products that
    mx_gated_ffn_backward and mx_gated_act_backward take: codes (R, 2 F), scales
    (R, 2 F / 32).
    qx (R, K) MXFP8 or (R, K / 2) MXFP4 codes, sx the blocked layout of their
    scales; qw (2 F, ..) codes, Wg's rows and then Wu's, sw likewise.  With
    group_end_offsets (int32 [G] on the device, cumulative END rows) qw is (G, 2
    F, ..) and sx the M-grouped blocked layout; rows past the last end are left
    as they were in `out`.  Formats "mxfp8" or "mxfp4"; MXFP4 x goes with MXFP4
    weights."""
    code = _act(act)
    rows, f, k, fx, fw, groups = _ffn_operands(qx, sx, qw, sw, group_end_offsets, (a_format, w_format), 2, "x")
    o, dev = _outs(out, 3 if checkpoint else 1), qx.device
    y = _new(o[0], (rows, f), torch.bfloat16, dev, "y")
    q = s = None
    if checkpoint:
        q = _new_bytes(o[1], (rows, 2 * f), dev, "q")
        s = _new_bytes(o[2], (rows, 2 * f // MX_BLOCK), dev, "s")
    _call("mx_gated_ffn", dev, qx.data_ptr(), sx.data_ptr(), fx, qw.data_ptr(), sw.data_ptr(), fw,
          _p(group_end_offsets), groups, rows, f, k, code, y.data_ptr(), _p(q), _p(s))
    if not checkpoint:
        return (y,)
    return (y, q, s) if raw else (y, q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))


def mx_gated_ffn_backward(qd, sd, qw, sw, q, s, act: str = "silu", group_end_offsets=None, a_format: str = "mxfp8",
                          w_format: str = "mxfp8", recompute: bool = False, out=None):
    """Gradient of mx_gated_ffn's (g, u) through the second projection, in one
    kernel: (dh,) bf16 (R, 2 F), or with recompute (dh, y) with y formed again
    from the checkpoint (q, s).
    qd (R, ..) codes of the block's output gradient along its rows, sd their
    blocked scales; qw (F, ..) the second projection's weight (K, F) cast along
    the axis that is summed (its dim1 cast), sw likewise; groups and formats as
    for mx_gated_ffn."""
    code = _act(act)
    rows, f, k, fd, fw, groups = _ffn_operands(qd, sd, qw, sw, group_end_offsets, (a_format, w_format), 1, "d")
    dev = qd.device
    _bytes(q, (rows, 2 * f), "q")
    _bytes(s, (rows, 2 * f // MX_BLOCK), "s")
    if _code_type(q, "q"):
        raise ValueError("q must hold e4m3 codes or bytes, got %s" % q.dtype)
    _scale_type(s, "s")
    _same_device(dev, q=q, s=s)
    o = _outs(out, 2 if recompute else 1)
    dh = _new(o[0], (rows, 2 * f), torch.bfloat16, dev, "dh")
    y = _new(o[1], (rows, f), torch.bfloat16, dev, "y") if recompute else None
    _call("mx_gated_ffn_backward", dev, qd.data_ptr(), sd.data_ptr(), fd, qw.data_ptr(), sw.data_ptr(), fw,
          _p(group_end_offsets), groups, rows, f, k, code, q.data_ptr(), s.data_ptr(), dh.data_ptr(), _p(y))
    return (dh, y) if recompute else (dh,)


_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
SIGNATURES = {
    "mx_cast_mxfp4": ([_vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp], ctypes.c_int),
    "mx_dequantize_mxfp4": ([_vp, _vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp], ctypes.c_int),
    "mx_gemm_mxfp4": ([_vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp], ctypes.c_int),
    "mx_grouped_gemm_mxfp4": ([_vp, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp], ctypes.c_int),
    "mx_linear_decode": ([_vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp], ctypes.c_int),
    "mx_gated_ffn": ([_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp],
                     ctypes.c_int),
    "mx_gated_ffn_decode": ([_vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp], ctypes.c_int),
    "mx_gated_ffn_backward": ([_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp,
                               _vp], ctypes.c_int),
}
