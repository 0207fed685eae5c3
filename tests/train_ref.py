"""The training-step operators in binary64 numpy, straight from their
definitions, and inputs for their tests.  Nothing of the library is used
here; the checkpoint's codes come from the oracle's cast."""
import math

import numpy as np

U32 = 2.0 ** -24      # half an ulp of binary32, relative


def half_ulp16(a):
    """Half the spacing of bf16 (8 significant bits) at magnitude a: what one
    rounding of a number up to that magnitude may change."""
    e = np.floor(np.log2(np.maximum(np.abs(np.nan_to_num(a, posinf=0.0, neginf=0.0)), 2.0 ** -126)))
    return np.exp2(e - 8)


def bf16_round(a):
    """binary64 -> the nearest bf16 (through binary32: inputs here are made
    from binary32 numbers), as binary64."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16) << np.uint64(16)).astype(np.uint32)
    return r.view(np.float32).astype(np.float64)


def bits_of(a):
    """bf16 bit patterns of values that are bf16 numbers."""
    return (np.ascontiguousarray(a, dtype=np.float32).view(np.uint32) >> np.uint32(16)).astype(np.uint16)


def layernorm(x, w, b, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + (0.0 if b is None else b), mean, rstd


def layernorm_backward(dy, x, w, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def router(z, topk, valid, normalize, align):
    """One row at a time, plainly."""
    rows, experts = z.shape
    chosen = np.full((rows, topk), -1, np.int64)
    gates = np.zeros((rows, topk))
    lse = np.zeros(rows)
    p = np.zeros((rows, experts))
    here = np.zeros(rows, bool)
    for r in range(rows):
        if valid is not None and not valid[r]:
            continue
        if all(v == -math.inf for v in z[r]):
            continue
        here[r] = True
        top = z[r].max()
        with np.errstate(invalid="ignore"):
            e = np.exp(z[r] - top)
            p[r] = e / e.sum()
            lse[r] = top + np.log(e.sum())
        # NaN first, then descending, equal ones by index; -inf never
        order = sorted((i for i in range(experts) if z[r][i] != -math.inf),
                       key=lambda i: (not math.isnan(z[r][i]), -z[r][i] if not math.isnan(z[r][i]) else 0.0, i))
        for j, i in enumerate(order[:topk]):
            chosen[r, j], gates[r, j] = i, p[r, i]
        if normalize:
            gates[r] /= gates[r].sum()
    counts = np.bincount(chosen[chosen >= 0], minlength=experts)
    n = int(here.sum())
    balance = experts * counts / (topk * n * n) if n else np.zeros(experts)
    return dict(chosen=chosen, gates=gates, lse=lse, counts=counts, p=p, here=here, balance=balance,
                ends=np.cumsum(-(-counts // align) * align), loss=float((balance * p.sum(0)).sum()) if n else 0.0)


def router_value(z, chosen, here, normalize, balance, dgates, dloss):
    """sum(dgates * gates) + dloss * sum(balance * p) for a fixed choice: the
    function whose gradient the backward pass is."""
    total = 0.0
    for r in range(z.shape[0]):
        if not here[r]:
            continue
        e = np.exp(z[r] - z[r].max())
        p = e / e.sum()
        total += dloss * float((balance * p).sum())
        on = chosen[r] >= 0
        g = p[chosen[r][on]]
        if normalize:
            g = g / g.sum()
        total += float((dgates[r][on] * g).sum())
    return total


def router_backward(z, p, chosen, here, normalize, balance, dgates, dloss):
    """(dlogits, sum of the magnitudes that meet in each of them)."""
    rows, experts = z.shape
    dz = np.zeros((rows, experts))
    mag = np.zeros((rows, experts))
    for r in range(rows):
        if not here[r]:
            continue
        dp = dloss * balance.astype(np.float64)
        mp = np.abs(dp)
        on = np.flatnonzero(chosen[r] >= 0)
        d = dgates[r][on].astype(np.float64)
        md = np.abs(d)
        if normalize:
            s = p[r][chosen[r][on]].sum()
            g = p[r][chosen[r][on]] / s
            d, md = (d - (d * g).sum()) / s, (md + (md * g).sum()) / s
        dp[chosen[r][on]] += d
        mp[chosen[r][on]] += md
        dz[r] = p[r] * (dp - (p[r] * dp).sum())
        mag[r] = p[r] * (mp + (p[r] * mp).sum())
    return dz, mag


def gate_t(g, act):
    if act == "silu":
        return g, np.ones_like(g)
    a, b = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
    return a * (g + b * g ** 3), a * (1.0 + 3.0 * b * g ** 2)


def logistic(t):
    return np.where(t >= 0, 1.0 / (1.0 + np.exp(-np.abs(t))), np.exp(-np.abs(t)) / (1.0 + np.exp(-np.abs(t))))


def gated_act(g, u, act):
    return g * logistic(gate_t(g, act)[0]) * u


def gated_act_backward(dy, g, u, act):
    t, dt = gate_t(g, act)
    s = logistic(t)
    return dy * u * (s + g * dt * s * logistic(-t)), dy * g * s


def checkpoint(oracle_mod, x):
    """The oracle's dim0 cast of a matrix of bf16 values with any number of
    rows: codes, scale bytes and the values they stand for."""
    rows, cols = x.shape
    pad = (-rows) % 32
    bits = bits_of(np.concatenate([x, np.zeros((pad, cols))]) if pad else x)
    q, s = oracle_mod.cast_dim0(bits)
    q, s = np.ascontiguousarray(q[:rows]), np.ascontiguousarray(s[:rows])
    return q, s, values(q, s)


def values(q, s):
    """code * 2^(scale - 127) in binary64; NaN codes and scales give NaN."""
    table = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
        table[c] = math.nan if (c & 127) == 127 else -v if c & 128 else v
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127.0))
    return table[q] * np.repeat(scale, 32, axis=1)


def wgrad(dy, x, ends):
    """Per group, and the sum of the products' magnitudes."""
    rows = dy.shape[0]
    prev, out, mag = 0, [], []
    for e in ([rows] if ends is None else ends):
        hi = min(max(prev, int(e)), rows)
        a, b = dy[prev:hi], x[prev:hi]
        out.append(a.T @ b)
        mag.append(np.abs(a).T @ np.abs(b))
        prev = hi
    return np.stack(out), np.stack(mag)


def assert_close(got, want, tol, what):
    got = np.asarray(got, np.float64)
    want = np.asarray(want, np.float64)
    assert got.shape == want.shape, "%s: shape %s, expected %s" % (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), "%s: NaN in other places" % what
    with np.errstate(invalid="ignore"):
        off = np.where(nan, 0.0, np.abs(got - want))
        off = np.where(got == want, 0.0, off)   # equal infinities
    bad = off > np.broadcast_to(tol, off.shape)
    assert not bad.any(), "%s: %d of %d outside tolerance, first at %s: got %r, want %r" % (
        what, int(bad.sum()), bad.size, np.argwhere(bad)[0], got[tuple(np.argwhere(bad)[0])],
        want[tuple(np.argwhere(bad)[0])])
