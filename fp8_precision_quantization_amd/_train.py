"""ctypes binding of the second part of libmxcast (include/mxtrain.h): layer
norm, the MoE router, the gated activation and the weight gradient that work
from 8-bit activation checkpoints.

Argument marshalling only, as in _binding: shapes and dtypes are checked,
outputs and workspaces are allocated with torch, every call goes to the C ABI
on torch's current stream of the inputs' device, and there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import MX_BLOCK, MX_MAX_GROUPS, _check, lib

MX_MAX_NORM_COLS = 16384
MX_MAX_TOPK = 32
ACTS = {"silu": 0, "gelu": 1}

_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor" % name)


def _typed(t, dtypes, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _gpu(t, name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s must be on %s" % (name, device))


def _matrix(t, name):
    """(rows, cols, leading dimension) of a matrix whose rows are contiguous;
    a single row has no pitch of its own."""
    if t.dim() != 2:
        raise ValueError("%s must have 2 dimensions" % name)
    rows, cols = t.shape
    sr, sc = t.stride()
    if rows == 0 or cols == 0:
        return rows, cols, cols
    if cols > 1 and sc != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if rows == 1:
        return rows, cols, cols
    if sr < cols:
        raise ValueError("%s has overlapping rows" % name)
    return rows, cols, sr


def _vector(t, dtypes, n, name):
    _typed(t, dtypes, name)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d elements" % (name, n))


def _dense(t, dtypes, shape, name):
    _typed(t, dtypes, name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor" % (name, tuple(shape)))


def _bytes(t, shape, name):
    """A contiguous one-byte tensor of that shape (codes, scale bytes)."""
    _gpu(t, name)
    if t.element_size() != 1 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous one-byte %s tensor" % (name, tuple(shape)))


def _outs(out, count):
    if out is None:
        return (None,) * count
    if len(out) != count:
        raise ValueError("out must hold %d tensors (or None)" % count)
    return out


def _new(t, shape, dtype, device, name):
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device)   # sizes one by one: 0.4 us less than as a tuple
    _dense(t, (dtype,), shape, name)
    _same_device(device, **{name: t})
    return t


def _new_bytes(t, shape, device, name):
    if t is None:
        return torch.empty(*shape, dtype=torch.uint8, device=device)
    _bytes(t, shape, name)
    _same_device(device, **{name: t})
    return t


def _workspace(t, nbytes, device):
    """(tensor to keep until the call is enqueued, address, bytes).  A size
    below 0 is of a shape that the call itself will refuse."""
    if t is None:
        if nbytes <= 0:
            return None, None, 0
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        _gpu(t, "workspace")
        if not t.is_contiguous():
            raise ValueError("workspace must be contiguous")
        _same_device(device, workspace=t)
    return t, t.data_ptr(), t.numel() * t.element_size()


def _p(t):
    return None if t is None else t.data_ptr()


def _call(name, device, *args):
    """The C call on the device's current stream, with that device current."""
    f = getattr(lib(), name)
    # the stream's handle without the Stream object around it: 0.1 instead of
    # 1.9 us, of about 10 for a small call
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        status = f(*args, stream)
    else:
        with torch.cuda.device(device):
            status = f(*args, stream)
    if status:
        _check(status, name)


def _fp8(q, s, raw):
    return (q, s) if raw else (q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))


def mx_layernorm(x, weight, bias=None, eps: float = 1e-5, checkpoint: bool = False, out=None, raw: bool = False):
    """Layer norm over the rows of x (R, C), bf16 or float32: (y, mean, rstd),
    y as x, mean and rstd float32 (R).  weight (C) and bias (C) or None, bf16
    or float32, both of one type.  With checkpoint=True (bf16, C a multiple of
    32) also the 8-bit checkpoint of y: (y, mean, rstd, q, s), e4m3 / e8m0
    views, or uint8 if raw.  Rows of x may lie any distance apart.  With C = 0
    mean and rstd are NaN (0 / 0)."""
    _typed(x, (torch.bfloat16, torch.float32), "x")
    rows, cols, ldx = _matrix(x, "x")
    dev = x.device
    _vector(weight, (torch.bfloat16, torch.float32), cols, "weight")
    if bias is not None:
        _vector(bias, (weight.dtype,), cols, "bias")
    _same_device(dev, weight=weight, bias=bias)
    o = _outs(out, 5 if checkpoint else 3)
    y = _new(o[0], (rows, cols), x.dtype, dev, "y")
    mean = _new(o[1], (rows,), torch.float32, dev, "mean")
    rstd = _new(o[2], (rows,), torch.float32, dev, "rstd")
    if cols == 0:   # the C call writes nothing then
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    if checkpoint:
        if x.dtype != torch.bfloat16 or cols % MX_BLOCK:
            raise ValueError("a checkpoint needs a bfloat16 x and a multiple of %d columns" % MX_BLOCK)
        q = _new_bytes(o[3], (rows, cols), dev, "q")
        s = _new_bytes(o[4], (rows, cols // MX_BLOCK), dev, "s")
        _call("mx_layernorm_checkpoint", dev, x.data_ptr(), ldx, weight.data_ptr(), _p(bias), _TYPES[weight.dtype],
              rows, cols, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), q.data_ptr(), s.data_ptr())
        return (y, mean, rstd) + _fp8(q, s, raw)
    _call("mx_layernorm", dev, x.data_ptr(), ldx, _TYPES[x.dtype], weight.data_ptr(), _p(bias),
          _TYPES[weight.dtype], rows, cols, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), None, None)
    return y, mean, rstd


def mx_layernorm_checkpoint(x, weight, bias=None, eps: float = 1e-5, out=None, raw: bool = False):
    """mx_layernorm with checkpoint=True: (y, mean, rstd, q, s).  x, weight,
    bias and a caller's y and s may start at any element, a caller's q at any
    eight bytes."""
    return mx_layernorm(x, weight, bias, eps, True, out, raw)


def mx_layernorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return lib().mx_layernorm_backward_workspace_bytes(rows, cols)


def mx_layernorm_backward(dy, x, weight, mean, rstd, bias: bool = True, out=None, workspace=None):
    """Gradients of mx_layernorm: (dx, dweight, dbias), dx as x, the others
    float32 (C); dbias None if bias is False (the layer has none).  x, weight,
    mean and rstd as in the forward call, dy (R, C) of x's type."""
    _typed(x, (torch.bfloat16, torch.float32), "x")
    rows, cols, ldx = _matrix(x, "x")
    dev = x.device
    _typed(dy, (x.dtype,), "dy")
    if dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape")
    lddy = _matrix(dy, "dy")[2]
    _vector(weight, (torch.bfloat16, torch.float32), cols, "weight")
    _vector(mean, (torch.float32,), rows, "mean")
    _vector(rstd, (torch.float32,), rows, "rstd")
    _same_device(dev, dy=dy, weight=weight, mean=mean, rstd=rstd)
    o = _outs(out, 3)
    dx = _new(o[0], (rows, cols), x.dtype, dev, "dx")
    dw = _new(o[1], (cols,), torch.float32, dev, "dweight")
    db = _new(o[2], (cols,), torch.float32, dev, "dbias") if bias else None
    ws = _workspace(workspace, mx_layernorm_backward_workspace_bytes(rows, cols), dev)
    _call("mx_layernorm_backward", dev, dy.data_ptr(), lddy, x.data_ptr(), ldx, _TYPES[x.dtype], weight.data_ptr(),
          _TYPES[weight.dtype], mean.data_ptr(), rstd.data_ptr(), rows, cols, dx.data_ptr(), dw.data_ptr(), _p(db),
          ws[1], ws[2])
    return dx, dw, db


def mx_router_workspace_bytes(rows: int, experts: int) -> int:
    return lib().mx_router_workspace_bytes(rows, experts)


def mx_router_balance(logits, topk: int, valid=None, normalize: bool = False, align: int = 1, out=None,
                      workspace=None):
    """MoE router over logits (R, E), bf16 or float32: (chosen int32 (R, topk),
    gates (R, topk), lse (R), counts int32 (E), ends int32 (E), balance (E),
    loss (1)), the rest float32.  valid (R), bool or uint8, drops rows; ends
    are the group END offsets with every group padded to a multiple of
    `align`, as the grouped casts and GEMMs take them.  include/mxtrain.h has
    the definitions."""
    _typed(logits, (torch.bfloat16, torch.float32), "logits")
    rows, experts, ld = _matrix(logits, "logits")
    dev = logits.device
    if not 1 <= experts <= MX_MAX_GROUPS:
        raise ValueError("logits must have 1 to %d columns" % MX_MAX_GROUPS)
    if not 1 <= topk <= min(experts, MX_MAX_TOPK):
        raise ValueError("topk must be 1 to %d" % min(experts, MX_MAX_TOPK))
    if not 1 <= align <= 0x7FFFFFFF:
        raise ValueError("align must be positive and fit 32 bits")   # (ctypes would cut it off)
    if valid is not None:
        _vector(valid, (torch.bool, torch.uint8), rows, "valid")
        _same_device(dev, valid=valid)
    o = _outs(out, 7)
    f32, i32 = torch.float32, torch.int32
    chosen = _new(o[0], (rows, topk), i32, dev, "chosen")
    gates = _new(o[1], (rows, topk), f32, dev, "gates")
    lse = _new(o[2], (rows,), f32, dev, "lse")
    counts = _new(o[3], (experts,), i32, dev, "counts")
    ends = _new(o[4], (experts,), i32, dev, "ends")
    balance = _new(o[5], (experts,), f32, dev, "balance")
    loss = _new(o[6], (1,), f32, dev, "loss")
    ws = _workspace(workspace, mx_router_workspace_bytes(rows, experts), dev)
    _call("mx_router_balance", dev, logits.data_ptr(), ld, _TYPES[logits.dtype], _p(valid), rows, experts, topk,
          int(normalize), align, chosen.data_ptr(), gates.data_ptr(), lse.data_ptr(), counts.data_ptr(),
          ends.data_ptr(), balance.data_ptr(), loss.data_ptr(), ws[1], ws[2])
    return chosen, gates, lse, counts, ends, balance, loss


def mx_router_balance_backward(logits, lse, chosen, gates, balance, dgates=None, dloss=None,
                               normalize: bool = False, out=None):
    """Gradient of the logits (R, E), of their type, from dgates float32 (R,
    topk) and dloss float32 (1), either of them None for zero; the others as
    mx_router_balance took and returned them."""
    _typed(logits, (torch.bfloat16, torch.float32), "logits")
    rows, experts, ld = _matrix(logits, "logits")
    dev = logits.device
    _typed(chosen, (torch.int32,), "chosen")
    if chosen.dim() != 2:
        raise ValueError("chosen must have 2 dimensions")
    topk = chosen.shape[1]
    f32 = torch.float32
    _dense(chosen, (torch.int32,), (rows, topk), "chosen")
    _dense(gates, (f32,), (rows, topk), "gates")
    _vector(lse, (f32,), rows, "lse")
    _vector(balance, (f32,), experts, "balance")
    if dgates is not None:
        _dense(dgates, (f32,), (rows, topk), "dgates")
    if dloss is not None:
        _typed(dloss, (f32,), "dloss")
        if dloss.numel() != 1:
            raise ValueError("dloss must hold one element")
    _same_device(dev, chosen=chosen, gates=gates, lse=lse, balance=balance, dgates=dgates, dloss=dloss)
    dlogits = _new(out, (rows, experts), logits.dtype, dev, "dlogits")
    _call("mx_router_balance_backward", dev, logits.data_ptr(), ld, _TYPES[logits.dtype], lse.data_ptr(),
          chosen.data_ptr(), gates.data_ptr(), balance.data_ptr(), _p(dgates), _p(dloss), rows, experts, topk,
          int(normalize), dlogits.data_ptr())
    return dlogits


def _act(act):
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTS)))
    return ACTS[act]


def mx_gated_act(h, act: str = "silu", checkpoint: bool = True, out=None, raw: bool = False):
    """act(h[:, :C]) * h[:, C:] of a contiguous bf16 h (R, 2 C), C a multiple
    of 32, act "silu" or "gelu" (tanh form): (y,), or with checkpoint (y, q, s)
    with the 8-bit checkpoint of h: codes (R, 2 C), scales (R, 2 C / 32)."""
    code = _act(act)
    _typed(h, (torch.bfloat16,), "h")
    if h.dim() != 2 or h.shape[1] % (2 * MX_BLOCK) or not h.is_contiguous():
        raise ValueError("h must be a contiguous matrix with a multiple of %d columns" % (2 * MX_BLOCK))
    rows, cols, dev = h.shape[0], h.shape[1] // 2, h.device
    o = _outs(out, 3 if checkpoint else 1)
    y = _new(o[0], (rows, cols), torch.bfloat16, dev, "y")
    q = s = None
    if checkpoint:
        q = _new_bytes(o[1], (rows, 2 * cols), dev, "q")
        s = _new_bytes(o[2], (rows, 2 * cols // MX_BLOCK), dev, "s")
    _call("mx_gated_act", dev, h.data_ptr(), rows, cols, code, y.data_ptr(), _p(q), _p(s))
    return (y,) + _fp8(q, s, raw) if checkpoint else (y,)


def mx_gated_act_backward(dy, q, s, act: str = "silu", recompute: bool = False, out=None):
    """Gradient of mx_gated_act from its checkpoint: (dh,) bf16 (R, 2 C), or
    with recompute (dh, y) with y formed again from the checkpoint."""
    code = _act(act)
    _typed(dy, (torch.bfloat16,), "dy")
    if dy.dim() != 2 or dy.shape[1] % MX_BLOCK or not dy.is_contiguous():
        raise ValueError("dy must be a contiguous matrix with a multiple of %d columns" % MX_BLOCK)
    rows, cols, dev = dy.shape[0], dy.shape[1], dy.device
    _bytes(q, (rows, 2 * cols), "q")
    _bytes(s, (rows, 2 * cols // MX_BLOCK), "s")
    _same_device(dev, q=q, s=s)
    o = _outs(out, 2 if recompute else 1)
    dh = _new(o[0], (rows, 2 * cols), torch.bfloat16, dev, "dh")
    y = _new(o[1], (rows, cols), torch.bfloat16, dev, "y") if recompute else None
    _call("mx_gated_act_backward", dev, dy.data_ptr(), q.data_ptr(), s.data_ptr(), rows, cols, code, dh.data_ptr(),
          _p(y))
    return (dh, y) if recompute else (dh,)


def mx_wgrad_checkpoint_workspace_bytes(rows: int, n: int, k: int, num_groups: int = 1) -> int:
    return lib().mx_wgrad_checkpoint_workspace_bytes(rows, n, k, num_groups)


def mx_wgrad_checkpoint(dy, q, s, group_end_offsets=None, out_dtype=torch.float32, out=None, workspace=None):
    """Weight gradient of a linear layer from bf16 dy (R, N) and the 8-bit
    checkpoint of its input, codes q (R, K) and scales s (R, K / 32): dy^T x,
    (N, K), float32 or bf16.  With group_end_offsets (int32 [G] on the device,
    cumulative END rows) one product per group of rows, (G, N, K).  Rows of dy
    may lie any distance apart."""
    _typed(dy, (torch.bfloat16,), "dy")
    rows, n, lddy = _matrix(dy, "dy")
    dev = dy.device
    _gpu(q, "q")
    if q.dim() != 2 or q.shape[1] % MX_BLOCK:
        raise ValueError("q must be a matrix with a multiple of %d columns" % MX_BLOCK)
    k = q.shape[1]
    _bytes(q, (rows, k), "q")
    _bytes(s, (rows, k // MX_BLOCK), "s")
    groups, shape = 1, (n, k)
    if group_end_offsets is not None:
        _typed(group_end_offsets, (torch.int32,), "group_end_offsets")
        groups = group_end_offsets.numel()
        _vector(group_end_offsets, (torch.int32,), groups, "group_end_offsets")
        if not 1 <= groups <= MX_MAX_GROUPS:
            raise ValueError("1 to %d groups" % MX_MAX_GROUPS)
        shape = (groups, n, k)
    _same_device(dev, q=q, s=s, group_end_offsets=group_end_offsets)
    if out_dtype not in _TYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    dw = _new(out, shape, out_dtype, dev, "out")
    ws = _workspace(workspace, mx_wgrad_checkpoint_workspace_bytes(rows, n, k, groups), dev)
    _call("mx_wgrad_checkpoint", dev, dy.data_ptr(), lddy, q.data_ptr(), s.data_ptr(), rows, n, k,
          _p(group_end_offsets), groups, dw.data_ptr(), _TYPES[out_dtype], ws[1], ws[2])
    return dw


_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
SIGNATURES = {
    "mx_layernorm": ([_vp, _i64, _i32, _vp, _vp, _i32, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mx_layernorm_checkpoint": ([_vp, _i64, _vp, _vp, _i32, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp],
                                ctypes.c_int),
    "mx_layernorm_backward_workspace_bytes": ([_i64, _i64], _i64),
    "mx_layernorm_backward": ([_vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64,
                               _vp], ctypes.c_int),
    "mx_router_workspace_bytes": ([_i64, _i64], _i64),
    "mx_router_balance": ([_vp, _i64, _i32, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _i64, _vp], ctypes.c_int),
    "mx_router_balance_backward": ([_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp],
                                   ctypes.c_int),
    "mx_gated_act": ([_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mx_gated_act_backward": ([_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp], ctypes.c_int),
    "mx_wgrad_checkpoint_workspace_bytes": ([_i64, _i64, _i64, _i32], _i64),
    "mx_wgrad_checkpoint": ([_vp, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _i64, _vp],
                            ctypes.c_int),
}
