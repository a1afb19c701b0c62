"""Oracle of rows as E4M3 codes and of the matrix product with an epilogue, in 64 bits.

TEST INFRASTRUCTURE ONLY: imported by ``tests/`` alone; no code shared with the library.  A row's scale and codes are float32
operations by definition (one division for the scale, one per value); the norm and the product are real-number formulas, so
they come in float64 with bounds of what float32 arithmetic may be off.
"""
import numpy as np
from scipy.special import erfc

from oracle.k2_fp8 import E4M3_VALUES, e4m3_encode

F32 = np.float32
U = 2.0 ** -24  # half a step of float32


def encode_rows(x):
    """(codes, scales) of float32 rows: the definition, in float32."""
    x = np.asarray(x, dtype=F32)
    top = np.abs(x).max(1)  # NaN if one is there
    with np.errstate(all="ignore"):
        scale = (top / F32(448.0)).astype(F32)
        bad = ~np.isfinite(top)
        safe = np.where(bad | (scale == 0), F32(1), scale)[:, None]
        codes = e4m3_encode(np.where(bad[:, None], F32(0), (x / safe).astype(F32)))
    codes[scale == 0] = 0
    codes[bad] = 0x7F
    return codes, np.where(bad, F32(np.nan), scale).astype(F32)


def norm_rows(x, residual, gain, groups, eps):
    """The normalised sum in float64 of the float32 sum."""
    h = np.asarray(x, dtype=F32) if residual is None else (np.asarray(x, dtype=F32) + np.asarray(residual, dtype=F32)).astype(F32)
    parts = h.astype(np.float64).reshape(h.shape[0], groups, -1)
    y = parts / np.sqrt((parts ** 2).mean(2, keepdims=True) + np.float64(F32(eps)))
    return h, y.reshape(h.shape) * np.asarray(gain, dtype=np.float64)


def norm_error(size):
    """How far, relative to its value, y may be off: a sum of `size` squares in float32 whatever its order is off by at most
    size / 2 roundings where every partial sum is one, and the kernels add at least 8 partial sums apart; mean, eps, root,
    quotient and two products follow."""
    return (size / 8 + 16) / 2 * U + 6 * U


def codes_between(v, rel):
    """The lowest and highest code values that v (in units of the scale) may be rounded to when it is off by `rel`."""
    a, b = v * (1 - rel), v * (1 + rel)
    return tuple(E4M3_VALUES[e4m3_encode(np.clip(q, -448, 448))] for q in (np.minimum(a, b), np.maximum(a, b)))


def activate(z, kind):
    """(value, the largest slope) of an activation."""
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-z))
        if kind in (None, "none"):
            return z, 1.0
        if kind == "relu":
            return np.maximum(z, 0), 1.0
        if kind == "silu":
            return z * sig, 1.1
        if kind == "gelu":
            return 0.5 * z * erfc(-z / np.sqrt(2)), 1.13
        return z / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))), 1.13


def linear(w, x, w_scale=None, x_scale=None, bias=None, activation=None, residual=None):
    """(result, bound of its error before the last rounding) of operands given as real numbers.

    The products are exact.  A tensor core adds 32 bytes of K at a time (at least 16 values) and each such addition, its
    alignment included, loses at most two steps of the running sum of magnitudes; scales, bias, activation and residual are
    a dozen roundings of what they meet."""
    w, x = np.asarray(w, dtype=np.float64), np.asarray(x, dtype=np.float64)
    z, mass = x @ w.T, np.abs(x) @ np.abs(w).T
    if w_scale is not None:
        s = np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)
        z, mass = z * s, mass * np.abs(s)
    off = mass * (4 * U * (w.shape[1] // 16 + 8))
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    off = off + 2 * U * np.abs(z)
    if activation == "swiglu":
        g, u = z[:, 0::2], z[:, 1::2]
        a = activate(g, "silu")[0]
        y = a * u
        off = 1.1 * off[:, 0::2] * np.abs(u) + (np.abs(a) + 1.1 * off[:, 0::2]) * off[:, 1::2] + 12 * U * np.abs(y)
    else:
        y, slope = activate(z, activation)
        off = slope * off + 12 * U * np.abs(z)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
        off = off + U * np.abs(y)
    return y, off


class _RoundedMatrix:
    """A weight matrix that rounds the rows multiplied with it to E4M3 codes first (`before`: and to a 16-bit type before that)."""

    __array_ufunc__ = None  # x @ self asks self

    def __init__(self, w, before):
        self.w, self.before = w, before

    @property
    def T(self):
        return self

    def __rmatmul__(self, x):
        x = np.asarray(x, dtype=F32)
        if self.before == "f16":
            x = x.astype(np.float16).astype(F32)
        elif self.before == "bf16":
            u = x.view(np.uint32)
            x = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(F32)
        codes, scale = encode_rows(x)
        return (E4M3_VALUES[codes] * scale.astype(np.float64)[:, None]) @ self.w.T


def act8(model, attention="f16"):
    """The oracle model with the projections of its layers over E4M3 activations: the library keeps the attention's output as
    `attention` ("f16", or None: in fp32) and the SwiGLU's as bf16 until they are rounded to codes."""
    plain = model._w
    before = {"wq": None, "wk": None, "wv": None, "w_gate": None, "w_up": None, "wo": attention, "w_down": "bf16"}
    model._w = lambda name, layer=-1: _RoundedMatrix(plain(name, layer), before[name]) if name in before else plain(name, layer)
    return model
