"""The loss's gradient of 4-bit layers over the range of their scales, on the
GPU against the float64 oracle: dx as accurate for weights far from one as for
ordinary ones."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import qlora_oracle as O
from oracle import vocab_oracle as V
from quantized_frozen_weight_amd import binding as Q
from quantized_frozen_weight_amd import workloads as WL
from tests.helpers import to_numpy
from tests.test_gpu_vocab import F64, H16, U16, U32, Case, dev, say, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    Q.lib()   # raises if libqlora.so is missing: no silent fallback


def dx_bound(c, l, tol, lse, tol_lse):
    """(dx, its bound) of a 4-bit layer without adapter.

    dl travels in float16 in units of dloss 2^-14: half a step relative, and half
    of 2^-24 of the unit where it is small. A weight is code times scale in
    float16 under a power of two that puts the layer's largest scale S in [2^12,
    2^13): half a step relative, and half of 2^-24 where it is small, which is at
    most 2^-25 2^-12 S of the weight; a scale itself stays whole from 2^-26 of S
    on (2^-14 over 2^12), or is off by half of 2^-24 for each unit of the code."""
    g = np.abs(c.dloss)
    dl = V.dlogits(l, lse, c.ids, c.dloss)
    ok = (c.ids >= 0) & (c.ids < c.vocab)
    p = np.exp(l - lse[:, None])
    ep = tol + tol_lse[:, None] + U32 * (3 * np.abs(l) + 3 * np.abs(lse)[:, None] + 4)
    tdl = np.where(ok[:, None], g[:, None] * (p * np.expm1(ep) + 2 * U32 * (p + 1)), 0.0)
    W = np.abs(c.W[:, :c.vocab]).T.astype(F64)
    scales = to_numpy(c.lin.scales)[:c.vocab].astype(F64)
    top = scales.max()
    floor = 2.0 ** -25 * 2.0 ** -12 * top
    wtiny = np.full_like(W, floor) + np.where(np.repeat(scales, 128, 1) < 2.0 ** -26 * top, 7 * floor, 0.0)
    rel = 2 * H16 + H16 * H16
    tdx = (tdl + rel * np.abs(dl) + 2.0 ** -39 * g[:, None]) @ W + (np.abs(dl) + tdl) @ wtiny
    tdx = tdx + (c.vocab + 8) * U32 * ((np.abs(dl) + tdl) @ W)
    dx = dl @ c.W[:, :c.vocab].astype(F64).T
    return dx, U16 * (np.abs(dx) + tdx) + tdx


def check(c):
    l, tol, _, _ = c.logits()
    _, wlse = V.loss_of(l, c.ids)
    tol_lse = c.lse_tol(l, tol)
    _, lse, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=c.vocab)
    got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), vocab=c.vocab)[0]
    torch.cuda.synchronize()
    within(to_numpy(lse), wlse, tol_lse, "lse")
    dx, bound = dx_bound(c, l, tol, wlse, tol_lse)
    within(to_numpy(got), dx, bound + 1e-37, "dx")
    return to_numpy(got)


# 1e-6: scales of one step of float16 and of none; 1e6: scales of 2^14
@pytest.mark.parametrize("M,K,vocab", [(20, 256, 300), (90, 128, 500), (300, 384, 260)])
@pytest.mark.parametrize("scale", [1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 1.0, 1e3, 1e5, 4e5])
def test_gradient_of_4_bit_weights_far_from_one(M, K, vocab, scale):
    """Every weight times `scale`, the rows of x divided by it."""
    c = Case(M, K, vocab, 0, "w4g128", "bf16", wstd=0.05 * scale)
    c.x_t, c.x = WL.as_compute_dtype((c.x / scale).astype(np.float32), "bf16")
    c.x_t = c.x_t.cuda()
    say("4-bit weights times", scale, M, K, vocab)
    got = check(c)
    if np.abs(c.W[:, :vocab]).max() > 0:
        assert np.abs(got).max() > 0


def test_gradient_of_4_bit_weights_of_many_sizes():
    """Entries from 1e-6 to 30 times the ordinary ones, and one group far above."""
    c = Case(70, 256, 96, 0, "w4g128", "bf16")
    f = np.exp(np.linspace(np.log(1e-6), np.log(30.0), 96))
    for high in (1.0, 1e6):
        W = (0.05 * np.random.default_rng(5).standard_normal((256, 96)) * f).astype(np.float32)
        W[128:, 40] *= high
        codes, scales = Q.qlora_quantize(dev(W), "w4g128")
        c.lin.codes, c.lin.scales = codes, scales
        c.W = O.dequant_w4(*O.quantize_w4(W))
        say("4-bit weights of many sizes", high)
        check(c)


def test_scales_of_padding_and_of_zero_take_no_part():
    """The power of two is of the scales of entries that exist."""
    c = Case(50, 256, 100, 0, "w4g128", "bf16", N=128, wstd=5e-6)
    c.x_t, c.x = WL.as_compute_dtype((c.x * 1e4).astype(np.float32), "bf16")
    c.x_t = c.x_t.cuda()
    say("scales of padding")
    got = check(c)
    for value in (65504.0, float("inf"), float("nan")):
        c.lin.scales[100:] = value
        assert np.array_equal(check(c), got)
    # no weight at all: dx is 0
    c.lin.scales.zero_()
    c.W = np.zeros_like(c.W)
    assert not check(c).any()


@pytest.mark.parametrize("k", [-12, -6, 5, 12])
def test_dx_scales_with_the_layer(k):
    """A layer whose scales are 2^k times another's, at rows of x 2^-k times: the
    same logits, and dx 2^k times, bit for bit (nothing is rounded another way)."""
    c = Case(130, 256, 400, 0, "w4g128", "bf16", wstd=4.0)
    c.x_t = c.x_t / 16
    dloss = dev(c.dloss)
    say("powers of two", k)

    def run(lin, x):
        loss, lse, _ = Q.qlora_xent_fwd(lin, x, c.ids_t, vocab=400)
        return loss, Q.qlora_xent_bwd(lin, x, c.ids_t, lse, dloss, vocab=400)[0]

    loss, dx = run(c.lin, c.x_t)
    lin = Q.QLinear(256, c.N, 0, 16.0, "w4g128", c.lin.codes, (c.lin.scales.float() * 2.0 ** k).half(), None, None)
    assert torch.equal(lin.scales.float() * 2.0 ** -k, c.lin.scales.float())
    loss2, dx2 = run(lin, (c.x_t.float() * 2.0 ** -k).bfloat16())
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2)
    assert torch.equal(dx2.float() * 2.0 ** -k, dx.float())
