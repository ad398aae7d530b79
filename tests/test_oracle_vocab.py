"""The vocabulary and AdamW oracle: gradients against differences, the 8-bit
form against its definition by enumeration, the rounding's average."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab_oracle as V

F64 = np.float64


def problem(seed, M=7, K=12, N=16, vocab=13, r=3):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    ids = rng.integers(-2, vocab + 2, M)
    return n((K, N)), n((K, r)), n((r, N)), n((M, K)), ids, vocab, 0.7


def slopes(f, a, h=1e-5):
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        p, q = a.copy(), a.copy()
        p[i] += h
        q[i] -= h
        out[i] = (f(p) - f(q)) / (2 * h)
    return out


@pytest.mark.parametrize("seed", [0, 1])
def test_lookup_gradient_against_differences(seed):
    W, A, B, dy, ids, vocab, s = problem(seed)
    f = lambda A, B: (V.lookup(W, ids, vocab, 1.7, s, A, B) * dy).sum()  # noqa: E731
    dA, dB = V.lookup_bwd(ids, vocab, W.shape[1], dy, 1.7, s, A, B)
    assert np.allclose(dA, slopes(lambda a: f(a, B), A), atol=1e-8)
    assert np.allclose(dB, slopes(lambda b: f(A, b), B), atol=1e-8)
    assert not dB[:, vocab:].any()


@pytest.mark.parametrize("seed", [2, 3])
def test_loss_gradient_against_differences(seed):
    W, A, B, x, ids, vocab, s = problem(seed)
    g = np.random.default_rng(9).standard_normal(len(x))

    def f(x, A, B):
        loss, _ = V.loss_of(V.logits(x, W, vocab, s, x @ A, B), ids)
        return (loss * g).sum()

    t = x @ A
    l = V.logits(x, W, vocab, s, t, B)
    _, lse = V.loss_of(l, ids)
    dl = V.dlogits(l, lse, ids, g)
    assert np.allclose(dl.sum(1), 0, atol=1e-12)
    dx, dA, dB = V.loss_bwd(dl, x, W, vocab, s, t, A, B)
    assert np.allclose(dx, slopes(lambda a: f(a, A, B), x), atol=1e-7)
    assert np.allclose(dA, slopes(lambda a: f(x, a, B), A), atol=1e-7)
    assert np.allclose(dB, slopes(lambda b: f(x, A, b), B), atol=1e-7)


@pytest.mark.parametrize("bits", [4, 5])
def test_codes_are_a_grid_and_read_back(bits):
    codes = np.arange(8 << bits)
    scales = np.full(len(codes) // 32, 130, np.uint8)
    v = V.s8_read(codes, scales, bits)
    assert (np.diff(v) > 0).all() and v[0] == 0 and v[-1] == (2 - 2.0 ** -bits) * 8
    assert (np.diff(v) >= 8 * 2.0 ** -(6 + bits)).all()
    # a value of the grid keeps its code whatever the hash; the scale is the group's own
    for rnd in (0, 0xffff):
        c, s = V.s8_write(v, bits, np.full(len(v), rnd))
        assert np.array_equal(V.s8_read(c, s, bits), v)


@pytest.mark.parametrize("bits", [4, 5])
def test_roundings_average_to_the_value(bits):
    rng = np.random.default_rng(1)
    v = np.repeat(rng.uniform(0.01, 1.9, 8).astype(np.float32), 4)
    total, runs = np.zeros(32), 4000
    for k in range(runs):
        h = V.hash32(np.arange(32), 3, k, 77)
        rnd = (h & 0xffff) if bits == 4 else h >> 16
        total += V.s8_read(*V.s8_write(v, bits, rnd), bits)
    step = np.exp2(np.maximum(np.floor(np.log2(v)), -6) - bits)
    # a step's standard deviation is at most half of it: five of the mean's
    assert (np.abs(total / runs - v) <= 5 * 0.5 * step / np.sqrt(runs)).all()


def test_hash_bits_are_even():
    h = V.hash32(np.arange(1 << 16), 5, 11, 3)
    for b in range(32):
        share = ((h >> np.uint32(b)) & 1).mean()
        assert abs(share - 0.5) < 5 * 0.5 / 256, b
    assert len(np.unique(h)) > 0.99 * len(h)


def test_groups_with_infinities_or_nan_read_as_nan():
    v = np.ones(96, np.float32)
    v[3], v[40] = np.inf, np.nan
    c, s = V.m_write(v, np.zeros(96))
    assert list(s[:2]) == [255, 255] and not c[:64].any()
    back = V.m_read(c, s)
    assert np.isnan(back[:64]).all() and (back[64:] == 1).all()


def test_adamw_follows_the_textbook_for_a_few_steps():
    rng = np.random.default_rng(4)
    p = rng.standard_normal(50).astype(np.float32)
    m = v = np.zeros(50, np.float32)
    q, m64, v64 = p.astype(F64), np.zeros(50), np.zeros(50)
    for k in range(1, 6):
        g = rng.standard_normal(50).astype(np.float32)
        p, m, v, _ = V.adamw(p, g, m, v, k, 1e-2, 0.9, 0.999, 1e-6, 0.1)
        m64, v64 = 0.9 * m64 + 0.1 * g, 0.999 * v64 + 0.001 * g.astype(F64) ** 2
        q = q - 1e-2 * (m64 / (1 - 0.9 ** k) / (np.sqrt(v64 / (1 - 0.999 ** k)) + 1e-6) + 0.1 * q)
    assert np.allclose(p, q, rtol=1e-5, atol=1e-6)
