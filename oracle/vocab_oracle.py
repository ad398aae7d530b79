"""Plain float64 numpy oracle of the vocabulary layer (lookup, its gradient,
softmax cross entropy and its gradient) and a float32 one of the AdamW step, in
the order of operations that the formulas give (include/qlora.h).

Test infrastructure only; the library never calls it.
"""

from __future__ import annotations

import numpy as np

F32, F64 = np.float32, np.float64
GROUP = 32


# ---- lookup -----------------------------------------------------------------
def lookup(W, ids, vocab, scale, s=0.0, A=None, B=None):
    """x [M, K] float64; W [K, N] the dequantized weight."""
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < vocab)
    at = np.where(ok, ids, 0)
    x = W[:, at].T.astype(F64)
    if A is not None:
        x = x + s * (B.astype(F64)[:, at].T @ A.astype(F64).T)
    return np.where(ok[:, None], scale * x, 0.0)


def lookup_bwd(ids, vocab, N, dy, scale, s, A, B):
    """(dA [K, r], dB [r, N]) in float64; rows without a token are left out."""
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < vocab)
    dy, at = dy.astype(F64)[ok], ids[ok]
    u = scale * s * (dy @ A.astype(F64))
    dB = np.zeros((N, A.shape[1]))
    np.add.at(dB, at, u)
    return scale * s * (dy.T @ B.astype(F64)[:, at].T), dB.T


# ---- loss -------------------------------------------------------------------
def logits(xh, W, vocab, s=0.0, t=None, B=None):
    """xh: the rows as their codes stand for them."""
    l = xh.astype(F64) @ W[:, :vocab].astype(F64)
    if t is not None:
        l = l + s * (t.astype(F64) @ B[:, :vocab].astype(F64))
    return l


def loss_of(l, targets):
    """(loss, lse) of logits l [M, vocab]."""
    targets = np.asarray(targets, np.int64)
    ok = (targets >= 0) & (targets < l.shape[1])
    top = l.max(1)
    lse = top + np.log(np.exp(l - top[:, None]).sum(1))
    at = np.where(ok, targets, 0)
    return np.where(ok, lse - l[np.arange(len(l)), at], 0.0), lse


def dlogits(l, lse, targets, dloss):
    targets = np.asarray(targets, np.int64)
    ok = (targets >= 0) & (targets < l.shape[1])
    d = np.exp(l - np.asarray(lse, F64)[:, None])
    rows = np.flatnonzero(ok)
    d[rows, targets[rows]] -= 1.0
    return np.where(ok[:, None], d * np.where(ok, dloss, 0.0)[:, None], 0.0)


def loss_bwd(dl, x, W, vocab, s=0.0, t=None, A=None, B=None):
    """(dx, dA, dB) of dl [M, vocab]; dA and dB None without an adapter."""
    dx = dl @ W[:, :vocab].astype(F64).T
    if A is None:
        return dx, None, None
    u = dl @ B[:, :vocab].astype(F64).T
    dB = np.zeros(B.shape)
    dB[:, :vocab] = s * (t.astype(F64).T @ dl)
    return dx + s * (u @ A.astype(F64).T), s * (x.astype(F64).T @ u), dB


# ---- AdamW ------------------------------------------------------------------
def hash32(element, item, k, seed):
    """The 32 bits of one element's rounding."""
    with np.errstate(over="ignore"):
        u = np.uint32
        x = (np.asarray(element).astype(u) * u(0x9E3779B1) + u(item) * u(0x3C6EF373) + u(k) * u(0xBB67AE85) + u(seed))
        x ^= x >> u(16)
        x *= u(0x6A09E667)
        x ^= x >> u(15)
        x *= u(0xBB67AE85)
        return x ^ (x >> u(16))


def s8_write(v, bits, rnd):
    """(codes of |v|, scale bytes); bits of mantissa, rnd 16 bits per element."""
    v = np.abs(np.asarray(v, F32))
    n = len(v)
    pad = -n % GROUP
    g = np.concatenate((v, np.zeros(pad, F32))).reshape(-1, GROUP)
    top = g.max(1)
    bad = ~(top < np.inf)
    safe = np.where(bad, 0, top).astype(F64)
    largest = 2 - 2.0 ** -bits
    e = np.full(len(top), -126)
    nz = safe > 0
    e[nz] = np.ceil(np.log2(safe[nz] / largest)).astype(int)
    e += (safe > largest * np.exp2(e.astype(F64))).astype(int)          # (the logarithm's own rounding)
    e -= ((safe > 0) & (safe <= largest * np.exp2(e - 1.0))).astype(int)
    e = np.clip(e, -126, 127)
    # in units of a subnormal code's step, 2^-(6 + bits) of the scale
    y = np.where(bad[:, None], 0, g).astype(F64) / np.exp2(e.astype(F64))[:, None]
    ex = np.clip(np.floor(np.log2(np.where(y > 0, y, 1e-300))), -6, 0)
    step = np.exp2(ex - bits)
    # the value in units of a float32's last bit after 2^-120 (rounded there, which
    # only values under the least normal code can be), the hash added below the code
    width = 23 - bits
    total = np.rint(y / step * 2.0 ** width) + rnd_pad(rnd, pad).reshape(-1, GROUP) * 2.0 ** (width - 16)
    code = np.where(ex > -6, (ex + 6) * 2 ** bits, 0) + np.floor(total / 2.0 ** width)
    code = np.minimum(code, 8 * 2 ** bits - 1).astype(np.int64)
    code[bad] = 0
    return code.reshape(-1)[:n], np.where(bad, 255, e + 127).astype(np.uint8)


def rnd_pad(rnd, pad):
    return np.concatenate((np.asarray(rnd, F64), np.zeros(pad)))


def s8_read(codes, scales, bits):
    """The magnitudes, float32."""
    codes = np.asarray(codes, np.int64)
    ex, man = codes >> bits, codes & ((1 << bits) - 1)
    f = np.where(ex > 0, 1 + man / 2.0 ** bits, man / 2.0 ** bits) * np.exp2(np.maximum(ex, 1) - 7.0)
    sc = np.repeat(np.asarray(scales, np.int64), GROUP)[:len(codes)]
    return np.where(sc == 255, np.nan, f * np.exp2(sc - 127.0)).astype(F32)


def m_write(m, rnd):
    c, sc = s8_write(m, 4, rnd)
    bad = np.repeat(sc == 255, GROUP)[:len(c)]
    return np.where(bad, 0, c + 128 * (np.asarray(m) < 0)).astype(np.uint8), sc


def root_write(root, rnd):
    c, sc = s8_write(root, 5, rnd)
    bad = np.repeat(sc == 255, GROUP)[:len(c)]
    return np.where((c == 0) & (np.asarray(root) > 0) & ~bad, 1, c).astype(np.uint8), sc


def m_read(codes, sc):
    codes = np.asarray(codes, np.int64)
    v = s8_read(codes & 127, sc, 4)
    return np.where(codes & 128, -v, v)


def root_read(codes, sc):
    return s8_read(codes, sc, 5)


def norm_of(grads):
    return F32(np.sqrt(sum(float((g.astype(F64) ** 2).sum()) for g in grads)))


def adamw(p, g, m, v, k, lr, beta1, beta2, eps, decay, coef=None):
    """One tensor's step in float32, every operation rounded: (p, m, v, root)."""
    one = F32(1)
    c1, c2 = F32(1 - beta1 ** k), F32(1 - beta2 ** k)
    g = g if coef is None else g * F32(coef)
    m = F32(beta1) * m + F32(1 - beta1) * g
    v = F32(beta2) * v + F32(1 - beta2) * (g * g)
    root = np.sqrt(v)
    keep, rate = one - F32(lr) * F32(decay), F32(lr) / c1
    p = p * keep - rate * (m / (root / np.sqrt(c2) + F32(eps)))
    return p, m, v, root
