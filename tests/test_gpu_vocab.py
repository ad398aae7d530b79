"""The vocabulary layer on the GPU against the float64 oracle: lookup and its
gradient, the loss without logits and its gradient; and one training step
through both ends of a model."""

from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import epilogue_oracle as E
from oracle import qlora_oracle as O
from oracle import vocab_oracle as V
from quantized_frozen_weight_amd import binding as Q
from quantized_frozen_weight_amd import workloads as WL
from tests.helpers import to_numpy

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F64 = np.float64
U32 = 2.0 ** -24          # half a step of float32, relative
U16 = 2.0 ** -8           # of bfloat16 (one part of a value: relative to it)
H16 = 2.0 ** -11          # of float16
# A product of two values in three bf16 parts each (8 bits a part, each rounded: what
# is left of a value is 2^-27 of it), without the products of parts 2^-27 and smaller
# (second times third, both ways, third times third): 2 2^-27 + 2 2^-27 and a little
THREE = 2.0 ** -24


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    Q.lib()   # raises if libqlora.so is missing: no silent fallback


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


def within(got, want, tol, what):
    got, want = np.asarray(got, F64), np.asarray(want, F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN pattern"
    ok = ~np.isnan(want)
    inf = ok & np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities"
    ok &= ~inf
    over = np.abs(got - want)[ok] - np.broadcast_to(tol, want.shape)[ok]
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.size} past the bound, worst by {over.max():.3e}"


def padded(vocab):
    return -(-vocab // 16) * 16


class Case:
    """A vocabulary layer, its oracle operands, and rows for it."""

    def __init__(self, M, K, vocab, r, fmt="w8", dtype="bf16", itype="i64", N=None, seed=0, alpha=16.0, wstd=0.05,
                 tokens=None):
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.M, self.K, self.vocab, self.r, self.fmt, self.dtype = M, K, vocab, r, fmt, dtype
        self.N = N = padded(vocab) if N is None else N
        W = wstd * n(K, N)
        codes, scales = Q.qlora_quantize(dev(W), fmt)
        if fmt == "w8":
            self.W = O.dequant_w8(*O.quantize_w8(W))
            self.logit_rel = 4 * U32
        else:
            self.W = O.dequant_w4(*O.quantize_w4(W))
            self.logit_rel = (K // 128 + 4) * U32
        self.A, self.B = (0.05 * n(K, r), 0.05 * n(r, N)) if r else (None, None)
        self.s = float(O.lora_scale(alpha, r)) if r else 0.0
        self.lin = Q.QLinear(K, N, r, alpha, fmt, codes, scales, dev(self.A) if r else None, dev(self.B) if r else None)
        self.x_t, self.x = WL.as_compute_dtype(n(M, K), dtype)
        self.dy_t, self.dy = WL.as_compute_dtype(n(M, K), dtype)
        self.x_t, self.dy_t = self.x_t.cuda(), self.dy_t.cuda()
        # tokens as frequent as in text; one in ten stands for none
        ids = np.minimum(np.exp(rng.uniform(0, np.log(vocab + 1.0), M)) - 1, vocab - 1).astype(np.int64)
        ids = np.where(rng.uniform(size=M) < 0.1, -100, ids) if tokens is None else np.asarray(tokens, np.int64)
        self.ids = ids
        self.ids_t = dev(ids.astype(np.int32 if itype == "i32" else np.int64))
        self.dloss = (rng.uniform(0.5, 1.5, M) / M).astype(np.float32)
        self.u = U16 if dtype == "bf16" else U32
        self.td = self.x_t.dtype
        self.A64 = self.A.astype(F64) if r else None
        self.B64 = self.B.astype(F64) if r else None

    # ---- the loss in float64, with bounds ----
    def rows(self):
        return E.read_rows(*O.quantize_rows(self.x))

    def logits(self):
        """(l, bound of each, t, bound of t)."""
        xh = self.rows()
        l = V.logits(xh, self.W, self.vocab)
        tol = self.logit_rel * (np.abs(xh) @ np.abs(self.W[:, :self.vocab]))
        t = tol_t = None
        if self.r:
            x64 = self.x.astype(F64)
            t = x64 @ self.A64
            tol_t = self.K * U32 * (np.abs(x64) @ np.abs(self.A64))
            B = np.abs(self.B64[:, :self.vocab])
            l = V.logits(xh, self.W, self.vocab, self.s, t, self.B64)
            tol = tol + self.s * (tol_t @ B + (self.r + 2) * U32 * (np.abs(t) @ B))
        return l, tol + 2 * U32 * np.abs(l), t, tol_t

    def lse_tol(self, l, tol):
        """What float32 exponentials and sums add to the logits' own bound."""
        top = np.abs(l).max(1)
        sums = self.vocab / 128 + 64                       # roundings one term passes
        return tol.max(1) + U32 * (8 * top + sums + 4 * (top + np.log(self.vocab)) + 4)

    def grads(self, l, tol, lse, tol_lse, t, tol_t, dloss=None):
        """((dx, dA, dB), bounds)."""
        g = self.dloss if dloss is None else dloss
        dl = V.dlogits(l, lse, self.ids, g)
        ok = (self.ids >= 0) & (self.ids < self.vocab)
        p = np.exp(l - lse[:, None])
        ep = tol + tol_lse[:, None] + U32 * (3 * np.abs(l) + 3 * np.abs(lse)[:, None] + 4)
        tdl = np.where(ok[:, None], np.abs(g)[:, None] * (p * np.expm1(ep) + 2 * U32 * (p + 1)), 0.0)
        W = np.abs(self.W[:, :self.vocab]).T
        sums = (self.vocab + 8) * U32
        if self.fmt == "w4g128":                           # both operands in float16
            rel = 2 * H16 + H16 * H16
            tiny = 2.0 ** -38 * np.abs(g)[:, None] * np.ones_like(dl)
            # a weight is fl16(q fl16(scale / 8)): near 0 each is off by half of 2^-24,
            # the scale's error times |q| <= 7; times 8
            wtiny = 8 * 2.0 ** -22
            tdx = (tdl + rel * np.abs(dl) + tiny) @ W + (np.abs(dl) + tdl) @ np.full_like(W, wtiny)
        elif self.dtype == "bf16":
            # dl times the scale in float16, 2^-24 the smallest step of it: off by half of
            # that where it is small, in units of dloss 2^(E - 14), 2^E at most twice the
            # largest scale; times a code of at most 127, over the vocabulary
            top = float(to_numpy(self.lin.scales)[:self.vocab].max())
            tiny = 2.0 ** -25 * 2.0 ** -14 * 2 * top * 127 * self.vocab
            tdx = (tdl + (H16 + 2 * U32) * np.abs(dl)) @ W + tiny * np.abs(g)[:, None]
        else:
            tdx = (tdl + 4 * U32 * np.abs(dl)) @ W
        tdx = tdx + sums * ((np.abs(dl) + tdl) @ W)
        x64 = self.x.astype(F64)
        dx, dA, dB = V.loss_bwd(dl, x64, self.W, self.vocab, self.s, t, self.A64, self.B64)
        if not self.r:
            return (dx, None, None), (self.u * (np.abs(dx) + tdx) + tdx, None, None)
        B = np.abs(self.B64[:, :self.vocab]).T
        u = dl @ self.B64[:, :self.vocab].T
        tu = (tdl + (THREE + 2 * sums) * np.abs(dl)) @ B
        A = np.abs(self.A64)
        low = np.abs(u) @ A.T
        tdx = tdx + self.s * (tu @ A.T + (self.r + 2) * U32 * low) + 2 * U32 * (np.abs(dx) + self.s * low)
        rows = (self.M + 8) * U32
        tdA = self.s * (np.abs(x64).T @ (tu + rows * np.abs(u)) + 2 * U32 * (np.abs(x64).T @ np.abs(u)))
        at = np.abs(t).T
        tdB = np.zeros_like(dB)
        tdB[:, :self.vocab] = self.s * (at @ tdl + tol_t.T @ np.abs(dl) + (THREE + rows) * (at @ (np.abs(dl) + tdl)))
        return (dx, dA, dB), (self.u * (np.abs(dx) + tdx) + tdx, tdA, tdB)


# ---- lookup -------------------------------------------------------------------
LOOKUPS = [
    # M, K, vocab, r, fmt, dtype, itype
    (1, 16, 1, 0, "w8", "f32", "i64"), (1, 2048, 50257, 8, "w8", "bf16", "i32"), (17, 48, 40, 4, "w8", "f32", "i32"),
    (64, 256, 1000, 1, "w8", "bf16", "i64"), (300, 768, 5000, 16, "w8", "bf16", "i64"),
    (33, 272, 77, 32, "w8", "f32", "i64"), (130, 4112, 100, 3, "w8", "bf16", "i32"), (50, 2064, 33, 9, "w8", "bf16", "i32"),
    (5, 128, 16, 0, "w4g128", "bf16", "i64"), (257, 2048, 3000, 8, "w4g128", "bf16", "i32"),
    (31, 4096, 50, 32, "w4g128", "bf16", "i64"), (2, 16384, 20, 5, "w4g128", "bf16", "i64"),
]


@pytest.mark.parametrize("M,K,vocab,r,fmt,dtype,itype", LOOKUPS)
def test_lookup(M, K, vocab, r, fmt, dtype, itype):
    say("lookup", M, K, vocab, r, fmt, dtype, itype)
    c = Case(M, K, vocab, r, fmt, dtype, itype)
    x = Q.qlora_embed(c.lin, c.ids_t, vocab=vocab, scale=1.7, dtype=c.td)
    torch.cuda.synchronize()
    want = V.lookup(c.W, c.ids, vocab, np.float32(1.7).astype(F64), c.s, c.A64, c.B64)
    size = V.lookup(np.abs(c.W), c.ids, vocab, 1.7, c.s, None if c.A is None else np.abs(c.A64),
                    None if c.B is None else np.abs(c.B64))
    tol = (r + 5) * U32 * size
    within(to_numpy(x), want, c.u * (np.abs(want) + tol) + tol, "x")


def test_lookup_of_ids_that_are_none():
    c = Case(9, 64, 30, 4, tokens=[0, 29, 30, 31, -1, 2 ** 31, -2 ** 63, 2 ** 40 + 3, 5])
    say("ids outside the vocabulary")
    x = to_numpy(Q.qlora_embed(c.lin, c.ids_t, vocab=30, scale=1.0, dtype=torch.float32))
    live = np.array([1, 1, 0, 0, 0, 0, 0, 0, 1], bool)
    assert not x[~live].any() and (np.abs(x[live]).max(1) > 0).all()
    # the whole layer where vocab is not given: 30 and 31 are entries then
    y = to_numpy(Q.qlora_embed(c.lin, c.ids_t, scale=1.0, dtype=torch.float32))
    assert np.array_equal(y[live], x[live]) and not y[4:8].any()
    i32 = dev(np.array([0, 29, 30, -1, -2 ** 31, 2 ** 31 - 1], np.int32))
    z = to_numpy(Q.qlora_embed(c.lin, i32, vocab=30, dtype=torch.float32))
    assert np.array_equal(z[:2], x[:2]) and not z[2:].any()


def run_lookup_bwd(c, **kw):
    dA, dB = Q.qlora_embed_bwd(c.lin, c.ids_t, c.dy_t, vocab=c.vocab, scale=1.7, **kw)
    torch.cuda.synchronize()
    return dA, dB


def check_lookup_bwd(c, dA, dB, dy=None):
    dy = c.dy if dy is None else dy
    scale = F64(np.float32(1.7))
    wA, wB = V.lookup_bwd(c.ids, c.vocab, c.N, dy, scale, c.s, c.A64, c.B64)
    sA, sB = V.lookup_bwd(c.ids, c.vocab, c.N, np.abs(dy), scale, c.s, np.abs(c.A64), np.abs(c.B64))
    count = np.bincount(c.ids[(c.ids >= 0) & (c.ids < c.vocab)], minlength=c.N)
    within(to_numpy(dA), wA, (c.M + 6) * U32 * sA, "dA")
    within(to_numpy(dB), wB, (c.K + count + 6) * U32 * sB, "dB")


LOOKUP_BWDS = [
    # M, K, vocab, r, dtype, itype, tokens
    (1, 16, 1, 1, "f32", "i64", "text"), (15, 48, 40, 4, "bf16", "i32", "text"), (255, 256, 1000, 8, "bf16", "i64", "text"),
    (256, 272, 7, 3, "f32", "i32", "text"), (257, 128, 5000, 16, "bf16", "i64", "text"),
    (1001, 768, 50257, 4, "bf16", "i64", "text"), (2048, 64, 300, 32, "f32", "i64", "text"),
    (2049, 80, 300, 17, "bf16", "i32", "text"), (8193, 144, 20000, 8, "bf16", "i64", "text"),
    (20000, 16, 33, 5, "f32", "i32", "text"), (3000, 32, 64, 8, "bf16", "i64", "one"), (700, 32, 64, 2, "f32", "i64", "one"),
    (512, 48, 512, 8, "bf16", "i64", "each"), (5000, 16, 5008, 1, "f32", "i32", "reversed"),
    (600, 48, 64, 8, "bf16", "i64", "none"), (4096, 32, 64, 4, "bf16", "i64", "blocks"), (16500, 16, 3, 8, "bf16", "i64", "text"),
]


@pytest.mark.parametrize("M,K,vocab,r,dtype,itype,kind", LOOKUP_BWDS)
def test_lookup_gradient(M, K, vocab, r, dtype, itype, kind):
    say("lookup gradient", M, K, vocab, r, dtype, itype, kind)
    tokens = {"text": None, "one": np.full(M, vocab // 2), "each": np.arange(M) % vocab,
              "reversed": (vocab - 1 - np.arange(M)) % vocab, "none": np.full(M, -1),
              "blocks": np.arange(M) // 256 % vocab}[kind]        # runs that end where blocks do
    c = Case(M, K, vocab, r, "w8", dtype, itype, tokens=tokens)
    dA, dB = run_lookup_bwd(c)
    check_lookup_bwd(c, dA, dB)
    again = run_lookup_bwd(c)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip((dA, dB), again))


def test_lookup_gradient_accumulates_and_leaves_rows_without_a_token_out():
    c = Case(1500, 96, 700, 8, "w8", "bf16")
    say("lookup gradient accumulated")
    dA, dB = run_lookup_bwd(c)
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    a1, b1 = a0.clone(), b0.clone()
    run_lookup_bwd(c, dA=a1, dB=b1, accumulate=True)
    # dA = fl(c S) of a float32 sum S, and the added one fl(a0 + c S) or fl(a0 + fl(c S)):
    # |a0 + dA - result| <= U32 |dA| (dA's own rounding, which a fused add does not
    # have) + U32 |result|
    for got, base, grad, what in ((a1, a0, dA, "dA added"), (b1, b0, dB, "dB added")):
        got, base, grad = (to_numpy(v).astype(F64) for v in (got, base, grad))
        within(got, base + grad, 1.01 * U32 * (np.abs(got) + np.abs(grad)), what)
    # entries that no row names keep their bytes
    unseen = np.setdiff1d(np.arange(c.N), c.ids)
    assert torch.equal(b1[:, unseen], b0[:, unseen])
    # whatever stands in a row without a token
    c.dy_t[torch.from_numpy(c.ids < 0).cuda()] = float("nan")
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip((dA, dB), run_lookup_bwd(c)))
    # a NaN in a row with one reaches its own entry and dA, no other entry
    row = int(np.flatnonzero(c.ids >= 0)[3])
    c.dy_t[row, 5] = float("nan")
    dA2, dB2 = run_lookup_bwd(c)
    assert torch.isnan(dA2[5]).all() and torch.isnan(dB2[:, c.ids[row]]).all()
    other = np.setdiff1d(np.arange(c.N), c.ids[row])
    assert torch.equal(dB2[:, other], dB[:, other])
    assert torch.equal(dA2[:5], dA[:5]) and torch.equal(dA2[6:], dA[6:])


# ---- loss -----------------------------------------------------------------------
LOSSES = [
    # M, K, vocab, r, fmt, dtype, itype
    (1, 16, 1, 0, "w8", "f32", "i64"), (1, 64, 17, 4, "w8", "bf16", "i32"), (2, 2048, 1000, 0, "w8", "bf16", "i64"),
    (32, 144, 300, 32, "w8", "bf16", "i64"), (33, 144, 300, 9, "w8", "f32", "i64"), (77, 256, 1000, 4, "w8", "f32", "i64"),
    (128, 784, 129, 16, "w8", "bf16", "i32"), (129, 400, 513, 8, "w8", "bf16", "i64"), (300, 768, 2000, 32, "w8", "bf16", "i64"),
    (300, 272, 2000, 3, "w8", "bf16", "i32"), (257, 1024, 255, 0, "w8", "f32", "i64"), (700, 80, 40, 16, "w8", "bf16", "i64"),
    (1, 128, 5, 2, "w4g128", "bf16", "i64"), (31, 256, 400, 0, "w4g128", "bf16", "i64"),
    (200, 512, 700, 8, "w4g128", "bf16", "i32"), (130, 4096, 300, 20, "w4g128", "bf16", "i64"),
    (20, 8192, 150, 4, "w4g128", "bf16", "i64"), (140, 16384, 130, 0, "w4g128", "bf16", "i64"),
    # few rows over many entries: many splits, and tiles between the smallest and the largest
    (40, 256, 9000, 8, "w4g128", "bf16", "i64"), (5, 64, 20000, 4, "w8", "f32", "i32"),
    (1, 32, 30000, 9, "w8", "bf16", "i64"), (256, 512, 16000, 8, "w8", "bf16", "i64"),
    (200, 320, 33000, 16, "w8", "bf16", "i64"), (600, 64, 9001, 2, "w8", "f32", "i64"),
]


@pytest.mark.parametrize("M,K,vocab,r,fmt,dtype,itype", LOSSES)
def test_loss_and_its_gradient(M, K, vocab, r, fmt, dtype, itype):
    say("loss", M, K, vocab, r, fmt, dtype, itype)
    c = Case(M, K, vocab, r, fmt, dtype, itype)
    loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=vocab)
    torch.cuda.synchronize()
    l, tol, t64, tol_t = c.logits()
    wloss, wlse = V.loss_of(l, c.ids)
    tol_lse = c.lse_tol(l, tol)
    within(to_numpy(lse), wlse, tol_lse, "lse")
    within(to_numpy(loss), wloss, np.where(wloss == 0, 0, 2 * tol_lse + 4 * U32 * np.abs(wlse)), "loss")
    if r:
        within(to_numpy(t), t64, tol_t, "t")
    say("its gradient")
    dloss = dev(c.dloss)
    got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dloss, t=t, vocab=vocab)
    torch.cuda.synchronize()
    want, bound = c.grads(l, tol, wlse, tol_lse, t64, tol_t)
    for g, w, b, what in zip(got, want, bound, ("dx", "dA", "dB")):
        assert (g is None) == (w is None)
        if g is not None:
            within(to_numpy(g), w, b + 1e-37, what)
    # again: the same bytes; t formed again where it is not given
    again = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dloss, vocab=vocab)
    assert all(a is None or torch.equal(bits(a), bits(b)) for a, b in zip(again, got))
    if r:
        none, dA, dB = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dloss, t=t, vocab=vocab, need_dx=False)
        assert none is None and torch.equal(dA, got[1]) and torch.equal(dB, got[2])


@pytest.mark.parametrize("M,K,vocab,r,fmt,dtype", [
    (131072, 16, 1100, 3, "w8", "bf16"), (87000, 16, 1100, 0, "w8", "f32"), (262144, 128, 560, 0, "w4g128", "bf16")])
def test_gradient_in_several_pieces(M, K, vocab, r, fmt, dtype):
    """So many rows that the vocabulary is taken in two or three pieces."""
    say("several pieces", M, K, vocab, r, fmt, dtype)
    c = Case(M, K, vocab, r, fmt, dtype)
    l, tol, t64, tol_t = c.logits()
    _, wlse = V.loss_of(l, c.ids)
    _, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=vocab)
    got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), t=t, vocab=vocab)
    torch.cuda.synchronize()
    want, bound = c.grads(l, tol, wlse, c.lse_tol(l, tol), t64, tol_t)
    for g, w, b, what in zip(got, want, bound, ("dx", "dA", "dB")):
        if g is not None:
            within(to_numpy(g), w, b + 1e-37, what)


@pytest.mark.parametrize("fmt", ["w8", "w4g128"])
@pytest.mark.parametrize("M", [5, 200])
def test_padding_rows_and_targets_that_are_none_touch_nothing(M, fmt):
    vocab = 333
    c = Case(M, 256, vocab, 4, fmt, N=384)
    say("padding", M, fmt)
    args = lambda c: (c.lin, c.x_t, c.ids_t)  # noqa: E731
    loss, lse, t = Q.qlora_xent_fwd(*args(c), vocab=vocab)
    g = Q.qlora_xent_bwd(*args(c), lse, dev(c.dloss), t=t, vocab=vocab)
    # garbage in the columns past vocab: codes, scales and B
    c.lin.codes[vocab:] = 0x77
    c.lin.scales[vocab:] = float("nan")
    c.lin.B[:, vocab:] = float("inf")
    loss2, lse2, _ = Q.qlora_xent_fwd(*args(c), vocab=vocab)
    g2 = Q.qlora_xent_bwd(*args(c), lse2, dev(c.dloss), t=t, vocab=vocab)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(g, g2))
    assert not g2[2][:, vocab:].any()
    # a row of NaN without a target (and its dloss): no trace of it but its own lse
    none = torch.from_numpy(c.ids < 0).cuda()
    assert none.any() or M == 5
    c.ids_t[0], none[0] = -100, True
    dl = dev(c.dloss)
    base = Q.qlora_xent_bwd(*args(c), lse2, dl, vocab=vocab)
    c.x_t[0, 3] = float("inf")
    dl[0] = float("nan")
    loss3, lse3, t3 = Q.qlora_xent_fwd(*args(c), vocab=vocab)
    assert torch.isnan(lse3[0]) and loss3[0] == 0 and torch.equal(lse3[1:], lse2[1:])
    dx, dA, dB = Q.qlora_xent_bwd(*args(c), lse3, dl, vocab=vocab)
    torch.cuda.synchronize()
    assert not dx[none].any()
    assert torch.equal(bits(dx), bits(base[0]))
    assert torch.equal(dA, base[1]) and torch.equal(dB, base[2])


@pytest.mark.parametrize("fmt,dtype", [("w8", "bf16"), ("w8", "f32"), ("w4g128", "bf16")])
@pytest.mark.parametrize("M", [3, 150, 400])
def test_rows_with_nan_or_infinity_touch_no_other_row(M, fmt, dtype):
    c = Case(M, 256, 500, 0, fmt, dtype, tokens=np.arange(M) % 500)
    say("odd rows", M, fmt, dtype)
    dl = dev(c.dloss)
    loss, lse, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=500)
    dx, _, _ = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dl, vocab=500)
    c.x_t[0, 7], c.x_t[M - 1, 200] = float("nan"), float("-inf")
    loss2, lse2, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=500)
    dx2, _, _ = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse2, dl, vocab=500)
    torch.cuda.synchronize()
    odd = torch.zeros(M, dtype=torch.bool, device="cuda")
    odd[0] = odd[M - 1] = True
    for a, b in ((loss, loss2), (lse, lse2)):
        assert torch.isnan(b[odd]).all() and torch.equal(a[~odd], b[~odd])
    assert torch.isnan(dx2[odd]).all() and torch.equal(bits(dx2[~odd]), bits(dx[~odd]))


@pytest.mark.parametrize("fmt,dtype", [("w8", "bf16"), ("w8", "f32"), ("w4g128", "bf16")])
def test_confident_and_far_logits(fmt, dtype):
    """Logits in the hundreds: the target's probability next to 1 or to 0."""
    c = Case(96, 128, 200, 0, fmt, dtype, wstd=3.0, tokens=np.arange(96))
    l, tol, _, _ = c.logits()
    best = l.argmax(1)
    c.ids = np.where(np.arange(96) % 2 == 0, best, c.ids)
    c.ids_t = dev(c.ids)
    say("far logits", fmt, dtype, float(np.abs(l).max()))
    loss, lse, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=200)
    got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), vocab=200)[0]
    torch.cuda.synchronize()
    wloss, wlse = V.loss_of(l, c.ids)
    tol_lse = c.lse_tol(l, tol)
    within(to_numpy(lse), wlse, tol_lse, "lse")
    within(to_numpy(loss), wloss, 2 * tol_lse + 4 * U32 * np.abs(wlse), "loss")
    assert (to_numpy(loss) > -1e-3).all()
    (dx, _, _), (tdx, _, _) = c.grads(l, tol, wlse, tol_lse, None, None)
    within(to_numpy(got), dx, tdx + 1e-37, "dx")


def test_gradient_of_large_and_tiny_weights():
    """Scales of the entries far apart: 1e-6 to 1e4."""
    for fmt, dtype in (("w8", "bf16"), ("w8", "f32"), ("w4g128", "bf16")):
        c = Case(70, 128, 96, 0, fmt, dtype)
        f = np.exp(np.linspace(np.log(1e-6), np.log(30.0 if fmt == "w4g128" else 1e4), 96))
        W = (0.05 * np.random.default_rng(5).standard_normal((128, 96)) * f).astype(np.float32)
        codes, scales = Q.qlora_quantize(dev(W), fmt)
        c.lin.codes, c.lin.scales = codes, scales
        c.W = O.dequant_w8(*O.quantize_w8(W)) if fmt == "w8" else O.dequant_w4(*O.quantize_w4(W))
        say("weights of many sizes", fmt, dtype)
        l, tol, _, _ = c.logits()
        _, wlse = V.loss_of(l, c.ids)
        _, lse, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=96)
        got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), vocab=96)[0]
        torch.cuda.synchronize()
        tol_lse = c.lse_tol(l, tol)
        within(to_numpy(lse), wlse, tol_lse, "lse")
        (dx, _, _), (tdx, _, _) = c.grads(l, tol, wlse, tol_lse, None, None)
        within(to_numpy(got), dx, tdx + 1e-37, "dx")


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12])
def test_gradient_of_weights_far_from_one(scale):
    """Every weight times `scale` (the rows of x divided by it where that is large):
    dx is as far from 0."""
    c = Case(150, 64, 300, 0, "w8", "bf16", wstd=0.05 * scale)
    if scale > 1:
        c.x_t, c.x = WL.as_compute_dtype((c.x / scale).astype(np.float32), "bf16")
        c.x_t = c.x_t.cuda()
    say("weights times", scale)
    l, tol, _, _ = c.logits()
    _, wlse = V.loss_of(l, c.ids)
    _, lse, _ = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=300)
    got = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), vocab=300)[0]
    torch.cuda.synchronize()
    tol_lse = c.lse_tol(l, tol)
    within(to_numpy(lse), wlse, tol_lse, "lse")
    (dx, _, _), (tdx, _, _) = c.grads(l, tol, wlse, tol_lse, None, None)
    within(to_numpy(got), dx, tdx + 1e-37, "dx")


@pytest.mark.parametrize("fmt,dtype", [("w8", "bf16"), ("w8", "f32"), ("w4g128", "bf16")])
def test_rows_without_a_target_beside_weights_that_are_no_numbers(fmt, dtype):
    """No row has a target: every gradient is 0, whatever the weights hold."""
    c = Case(70, 128, 300, 4, fmt, dtype, tokens=np.full(70, -1))
    B = c.B.copy()
    B[1, 7], B[2, 9] = np.inf, np.nan
    c.lin.B = dev(B)
    c.lin.scales[5] = float("nan")
    c.lin.scales[6] = float("inf")
    say("no numbers, no targets", fmt, dtype)
    loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=300)
    dx, dA, dB = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev(c.dloss), t=t, vocab=300)
    torch.cuda.synchronize()
    assert not to_numpy(loss).any()
    for g in (dx, dA, dB):
        assert not to_numpy(g).any()


@pytest.mark.parametrize("itype", ["i32", "i64"])
def test_tokens_that_begin_anywhere(itype):
    """Slices of a longer tensor of ids give what their copies give."""
    c = Case(40, 64, 100, 4, "w8", "bf16", itype=itype)
    say("slices", itype)
    dloss = dev(c.dloss)
    for off in (1, 2, 3):
        long = torch.cat([c.ids_t.new_full((off,), 3), c.ids_t])
        for ids in (long[off:],):
            assert ids.data_ptr() % 16 == off * ids.element_size() % 16

            def run(ids):
                x = Q.qlora_embed(c.lin, ids, vocab=100, dtype=torch.bfloat16)
                loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, ids, vocab=100)
                return [x, loss, lse, *Q.qlora_xent_bwd(c.lin, c.x_t, ids, lse, dloss, t=t, vocab=100),
                        *Q.qlora_embed_bwd(c.lin, ids, c.dy_t, vocab=100)]

            for a, b in zip(run(ids), run(c.ids_t)):
                assert torch.equal(bits(a), bits(b))


def test_adapter_gradients_against_differences_of_the_loss():
    c = Case(200, 256, 700, 4, "w8", "bf16")
    say("differences")
    rng = np.random.default_rng(3)
    dA_dir, dB_dir = rng.standard_normal(c.A.shape), rng.standard_normal(c.B.shape)
    dB_dir[:, 700:] = 0
    dloss = dev(c.dloss)

    def f(h, which):
        A = c.A64 + (h * dA_dir if which == "A" else 0)
        B = c.B64 + (h * dB_dir if which == "B" else 0)
        lin = Q.QLinear(256, c.N, 4, 16.0, "w8", c.lin.codes, c.lin.scales, dev(A.astype(np.float32)),
                        dev(B.astype(np.float32)))
        loss, _, _ = Q.qlora_xent_fwd(lin, c.x_t, c.ids_t, vocab=700)
        return float((loss.double() * dloss.double()).sum())

    _, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=700)
    _, dA, dB = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dloss, t=t, vocab=700)
    for which, g, d in (("A", dA, dA_dir), ("B", dB, dB_dir)):
        h = 1e-3
        slope = (f(h, which) - f(-h, which)) / (2 * h)
        want = float((to_numpy(g).astype(F64) * d).sum())
        # float32 losses of about 7 averaged over the rows: 200 roundings of
        # 2^-24 * 8 each in quadrature at most, twice, over 2 h; and h^2 of curvature
        noise = 2 * 8 * U32 * 4 / (2 * h)
        assert abs(slope - want) <= noise + 0.02 * abs(want), (which, slope, want)


# ---- as programs use it -------------------------------------------------------------
def test_captured_calls_replay_their_bytes():
    c = Case(300, 256, 1000, 8, "w8", "bf16")
    say("graph")
    dloss = dev(c.dloss)

    def step():
        x = Q.qlora_embed(c.lin, c.ids_t, vocab=1000, scale=16.0, dtype=torch.bfloat16)
        loss, lse, t = Q.qlora_xent_fwd(c.lin, x, c.ids_t, vocab=1000)
        dx, dA, dB = Q.qlora_xent_bwd(c.lin, x, c.ids_t, lse, dloss, t=t, vocab=1000)
        Q.qlora_embed_bwd(c.lin, c.ids_t, dx, vocab=1000, scale=16.0, dA=dA, dB=dB, accumulate=True)
        return loss, dx, dA, dB

    eager = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(4):
        for o in out:
            o.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        step()                                            # eager work between the replays
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, eager))
    # other tokens in the same buffers
    c.ids_t.copy_(torch.flip(c.ids_t, (0,)))
    want = [t.clone() for t in step()]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want))


def test_two_streams_at_once():
    cases = [Case(500, 256, 900, 4, "w8", "bf16", seed=1), Case(260, 256, 1200, 0, "w4g128", "bf16", seed=2)]
    say("two streams")

    def run(c):
        x = Q.qlora_embed(c.lin, c.ids_t, vocab=c.vocab, dtype=torch.bfloat16)
        loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=c.vocab)
        g = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dev_loss[id(c)], t=t, vocab=c.vocab)
        return [x, loss, lse] + [o for o in g if o is not None]

    dev_loss = {id(c): dev(c.dloss) for c in cases}
    want = [[t.clone() for t in run(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i] = run(c)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt,state", [("w8", "f32"), ("w4g128", "s8")])
def test_a_training_step_of_a_tied_model(fmt, state):
    """Tokens, lookup, one adapted layer with its residual, loss; backward
    through all of them into the tied vocabulary's adapter and the layer's; one
    AdamW step of the four. Against float64 of the same formulas, with the
    roundings between the calls as the calls have them."""
    M, K, vocab, r = 256, 256, 777, 4
    c = Case(M, K, vocab, r, fmt, "bf16", seed=8)
    rng = np.random.default_rng(12)
    n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    Wm, Am, Bm = 0.03 * n(K, K), 0.05 * n(K, r), 0.05 * n(r, K)
    codes, scales = Q.qlora_quantize(dev(Wm), "w8")
    mid = Q.QLinear(K, K, r, 16.0, "w8", codes, scales, dev(Am), dev(Bm))
    targets = np.roll(c.ids, -1)
    tg, dloss = dev(targets), dev(c.dloss)
    params = [c.lin.A, c.lin.B, mid.A, mid.B]
    opt = Q.AdamW(params, state=state, decay=[0.01, 0.01, 0.01, 0.0])
    say("training step", fmt, state)

    x0 = Q.qlora_embed(c.lin, c.ids_t, vocab=vocab, scale=16.0, dtype=torch.bfloat16)
    x1, t1, _, _ = Q.qlora_fwd_epi(mid, x0, residual=x0)
    loss, lse, t2 = Q.qlora_xent_fwd(c.lin, x1, tg, vocab=vocab)
    dx1, dA, dB = Q.qlora_xent_bwd(c.lin, x1, tg, lse, dloss, t=t2, vocab=vocab)
    dx0, dAm, dBm = Q.qlora_bwd_epi(mid, x0, dx1, t=t1, add=dx1)
    dA_head, dB_head = dA.clone(), dB.clone()
    Q.qlora_embed_bwd(c.lin, c.ids_t, dx0, vocab=vocab, scale=16.0, dA=dA, dB=dB, accumulate=True)
    grads = [dA, dB, dAm, dBm]
    before = [to_numpy(p).copy() for p in params]
    norm = Q.qlora_adamw(opt, grads, lr=1e-2, clip_norm=0.5, need_norm=True)
    torch.cuda.synchronize()

    # each call against the oracle on what it was given
    X = to_numpy(x1)
    c2 = c
    c2.x, c2.x_t, c2.ids, c2.A64, c2.B64 = X, x1, targets, before[0].astype(F64), before[1].astype(F64)
    l, tol, t64, tol_t = c2.logits()
    wloss, wlse = V.loss_of(l, targets)
    within(to_numpy(loss), wloss, np.where(wloss == 0, 0, 2 * c2.lse_tol(l, tol) + 4 * U32 * np.abs(wlse)), "loss")
    want, bound = c2.grads(l, tol, wlse, c2.lse_tol(l, tol), t64, tol_t)
    for g, w, b, what in zip((dx1, dA_head, dB_head), want, bound, ("dx", "dA", "dB")):
        within(to_numpy(g), w, b, what)
    eA, eB = V.lookup_bwd(to_numpy(c.ids_t), vocab, c.N, to_numpy(dx0), 16.0, c.s, c2.A64, c2.B64)
    within(to_numpy(dA), to_numpy(dA_head).astype(F64) + eA, 1e-5 * (np.abs(eA).max() + np.abs(to_numpy(dA))), "dA tied")
    within(to_numpy(dB), to_numpy(dB_head).astype(F64) + eB, 1e-5 * (np.abs(eB).max() + np.abs(to_numpy(dB))), "dB tied")
    G = [to_numpy(g) for g in grads]
    wnorm = V.norm_of([g.ravel() for g in G])
    assert abs(float(norm) - wnorm) <= 2 * U32 * wnorm
    coef = np.float32(0.5) / max(np.float32(norm.item()), np.float32(0.5))
    for p, b, g, d in zip(params, before, G, (0.01, 0.01, 0.01, 0.0)):
        z = np.zeros(g.size, np.float32)
        wp, _, _, _ = V.adamw(b.ravel(), g.ravel(), z, z, 1, 1e-2, 0.9, 0.999, 1e-6, d, coef)
        within(to_numpy(p).ravel(), wp, 4 * U32 * (np.abs(wp) + 1e-2), "parameter")
    assert int(opt.step) == 1
