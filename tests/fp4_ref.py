"""The MXFP4 cast, products of MX operands and the gated feed-forward block in
binary64 numpy, straight from their definitions, and inputs for their tests.
Nothing of the library is used here."""
import numpy as np

from tests import train_ref as ref

TABLE = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLES = (TABLE[1:] + TABLE[:-1]) / 2
LARGEST = {"e2m1": (2, 6.0), "e4m3": (8, 448.0)}   # exponent and value of a format's largest code


def scale_bytes(amax, fmt):
    """Scale byte of a block's largest magnitude (NaN where it holds one)."""
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.frexp(np.where(np.isfinite(amax), amax, 1.0))[1] - 1 - LARGEST[fmt][0]
    e = np.where(amax == 0, -127, np.where(np.isinf(amax), 127, e))
    return np.where(np.isnan(amax), 255, np.clip(e, -127, 127) + 127).astype(np.uint8)


def round_e2m1(t):
    """Codes of |t|, nearest, ties to the even code, 6 at most."""
    t = np.abs(t)
    return sum(((t > m) | ((t == m) & (i % 2 == 1))).astype(np.uint8) for i, m in enumerate(MIDDLES))


def cast4(x):
    """One code (sign in bit 3) to an element and the scale bytes of the blocks
    along the rows of binary64 values; a block with a NaN has zero codes."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    s = scale_bytes(np.abs(b).max(-1), "e2m1")
    with np.errstate(invalid="ignore"):
        q = round_e2m1(b / np.exp2(np.minimum(s, 254).astype(np.float64) - 127.0)[:, :, None])
    q = np.where(s[:, :, None] == 255, 0, q | (np.signbit(b).astype(np.uint8) << 3)).astype(np.uint8)
    return q.reshape(rows, cols), s


def pack(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def unpack(p):
    out = np.empty(p.shape[:-1] + (2 * p.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = p & 15, p >> 4
    return out


def values4(q, s):
    """code * 2^(byte - 127) of one code to an element; byte 255 gives NaN."""
    v = np.where(q & 8, -1.0, 1.0) * TABLE[q & 7]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127.0))
    return v * np.repeat(scale, 32, axis=-1)


def values(codes, s, fmt):
    """Codes as stored -> binary64."""
    return values4(unpack(codes), s) if fmt == "e2m1" else ref.values(codes, s)


def operand(rng, rows, k, fmt, spread=4):
    """Random codes as stored and scale bytes: every code, scales over 2^spread."""
    s = rng.integers(127 - spread, 128, (rows, k // 32)).astype(np.uint8)
    if fmt == "e2m1":
        return rng.integers(0, 256, (rows, k // 2)).astype(np.uint8), s
    q = rng.integers(0, 256, (rows, k)).astype(np.uint8)
    return np.where((q & 127) == 127, q ^ 1, q).astype(np.uint8), s - 6


def product(a, w):
    """(A W^T, the sum of the products' magnitudes)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def product_error(mag, k, fa, fw):
    """How far a product's binary32 sums may be off.  Each 64-deep step is one
    instruction: of e2m1 by e2m1 it is within 2^-22 of its largest product
    (measured 2^-22.2), of any pair with e4m3 within 2^-11 (measured 4.1e-4);
    its result meets the accumulator with one binary32 rounding, of at most
    2^-24 of the magnitudes so far."""
    step = 2.0 ** -22 if fa == fw == "e2m1" else 2.0 ** -11
    return mag * (step + (k / 64 + 2) * 2.0 ** -24)


def gated(h, act):
    f = h.shape[1] // 2
    return ref.gated_act(h[:, :f], h[:, f:], act)


def gated_tol(h, eh, act):
    """What an error of eh in (g, u) and the evaluation may change in act(g) u:
    |act'| <= 1.13 for both activations, |act(g)| <= |g|; the evaluation as for
    the activation alone ((16 + 8 |t|) 2^-24 of the value)."""
    f = h.shape[1] // 2
    g, u, eg, eu = h[:, :f], h[:, f:], eh[:, :f], eh[:, f:]
    a = np.abs(ref.gated_act(g, np.ones_like(g), act))
    t = np.minimum(np.abs(ref.gate_t(g, act)[0]), 200.0)
    moved = 1.13 * eg * np.abs(u) + (a + 1.13 * eg) * eu
    return moved + (18 + 8 * t) * ref.U32 * (a * np.abs(u) + moved) + 2.0 ** -125 * (np.abs(g * u) + 1)


def checkpoint_range(h, eh):
    """Lowest and highest scale byte and, for a given byte, the range of values
    that the MXFP8 cast of numbers within eh of h may hold."""
    rows, cols = h.shape
    b, e = np.abs(h).reshape(rows, -1, 32), eh.reshape(rows, -1, 32)
    lo = scale_bytes(np.maximum(b - e, 0).max(-1), "e4m3")
    hi = scale_bytes((b + e).max(-1), "e4m3")

    def held(v, s):
        t = v.reshape(rows, -1, 32) / np.exp2(s.astype(np.float64) - 127)[:, :, None]
        ex = np.maximum(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -20))), -6)
        step = np.exp2(ex - 3)
        return (np.clip(np.round(t / step) * step, -448, 448) * np.exp2(s.astype(np.float64) - 127)[:, :, None]
                ).reshape(rows, cols)

    return lo, hi, lambda s: (held(h - eh, s), held(h + eh, s))


def round_tol(want, tol, bf16):
    """A tolerance before the output's one rounding -> after it."""
    half = ref.half_ulp16 if bf16 else lambda a: np.abs(a) * 2.0 ** -24
    return tol + half(np.abs(want) + tol) + 1e-40


def bounds(ends, rows):
    lo, out = 0, []
    for e in ends:
        hi = min(max(lo, int(e)), rows)
        out.append((lo, hi))
        lo = hi
    return out
