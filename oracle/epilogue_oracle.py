"""Plain float64 numpy oracle of the layer's epilogue, the 8-bit activation
checkpoints and the gradients through them (formulas: include/qlora.h).

Test infrastructure only; the library never calls it.
"""

from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

F32, F64 = np.float32, np.float64
GROUP = 32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _tanh_arg(z):
    return np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)


def act(name: str, z):
    """act(z) in float64; -inf gives the limit 0, NaN stays NaN."""
    z = np.asarray(z, F64)
    if name == "none":
        return z
    lo = np.where(z == -np.inf, -1e30, z)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return lo * ndtr(lo)
    if name == "gelu_tanh":
        with np.errstate(over="ignore"):
            return lo * expit(2 * _tanh_arg(lo))
    if name == "silu":
        return lo * expit(lo)
    raise ValueError(name)


def slope(name: str, z):
    """act'(z) in float64 (relu'(0) = 0; limits at the infinities)."""
    z = np.asarray(z, F64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(np.isnan(z), z, (z > 0).astype(F64))
    c = np.clip(z, -400, 400)
    if name == "gelu":
        return ndtr(c) + c * np.exp(-0.5 * c * c) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        w = 2 * _tanh_arg(c)
        dw = 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * c * c)
        return expit(w) + c * dw * expit(w) * expit(-w)
    if name == "silu":
        return expit(c) * (1 + c * expit(-c))
    raise ValueError(name)


def write_groups(v):
    """v [M, C] float32 -> (codes int8 [M, C], bytes uint8 [M, ceil(C / 32)])."""
    v = np.asarray(v, F32)
    M, C = v.shape
    G = -(-C // GROUP)
    p = np.zeros((M, G * GROUP), F64)
    p[:, :C] = v
    p = p.reshape(M, G, GROUP)
    amax = np.abs(p).max(2)
    bad = ~np.isfinite(amax)
    e = np.full((M, G), -126, np.int64)
    live = (amax > 0) & ~bad
    m, x = np.frexp(np.where(live, amax, 1.0))       # amax = m 2^x, 1/2 <= m < 1
    e = np.where(live, np.maximum(np.where(m * 128 <= 127, x - 7, x - 6), -126), e)
    with np.errstate(invalid="ignore"):
        q = np.rint(p * 2.0 ** -e[:, :, None].astype(F64))
    q = np.where((q == 0) & (p != 0), np.sign(p), q)
    q = np.where(bad[:, :, None], 0, q)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return q.reshape(M, -1)[:, :C].astype(np.int8), byte


def read_groups(codes, byte):
    """The values of a group checkpoint, exact in float64 (and in bfloat16)."""
    C = codes.shape[1]
    b = np.repeat(byte.astype(np.int64), GROUP, axis=1)[:, :C]
    s = np.where(b == 255, np.nan, 2.0 ** (b.astype(F64) - 127))
    return codes.astype(F64) * s


def read_rows(codes, scales):
    """The values of a row checkpoint in float64."""
    return codes.astype(F64) * np.asarray(scales, F64)[:, None]
