"""The loss's gradient at the largest sizes that its calls take."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab_oracle as V
from quantized_frozen_weight_amd import binding as Q
from tests.helpers import to_numpy
from tests.test_gpu_vocab import F64, U32, Case, bits, dev, say, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("too little memory")
    Q.lib()   # raises if libqlora.so is missing: no silent fallback


def test_rows_at_the_limit_with_the_largest_rank():
    """2^24 rows at rank 32: 64 rows again and again, so that every repetition has
    the same loss and dx, and dA and dB are 2^18 times those of the 64."""
    n, times, vocab, r = 64, 1 << 18, 16, 32
    c = Case(n, 16, vocab, r, "w8", "bf16", seed=4)
    say("2^24 rows, rank 32")
    x, ids, dloss = c.x_t.repeat(times, 1), c.ids_t.repeat(times), dev(c.dloss).repeat(times)
    loss, lse, t = Q.qlora_xent_fwd(c.lin, x, ids, vocab=vocab)
    dx, dA, dB = Q.qlora_xent_bwd(c.lin, x, ids, lse, dloss, t=t, vocab=vocab)
    torch.cuda.synchronize()
    l, tol, t64, tol_t = c.logits()
    wloss, wlse = V.loss_of(l, c.ids)
    tol_lse = c.lse_tol(l, tol)
    (wx, wA, wB), (tx, tA, tB) = c.grads(l, tol, wlse, tol_lse, t64, tol_t)
    for got, want, bound, what in ((loss, wloss, np.where(wloss == 0, 0, 2 * tol_lse + 4 * U32 * np.abs(wlse)), "loss"),
                                   (dx, wx, tx, "dx")):
        per = got.view(times, n, -1)
        assert all(torch.equal(bits(per[i:i + 1024]), bits(per[:1].expand_as(per[i:i + 1024]).contiguous()))
                   for i in range(0, times, 1024)), what
        within(to_numpy(per[0]).reshape(want.shape), want, bound + 1e-37, what)
    # the sums of `times` equal parts: a float32 sum in a chain of at most 2^17 tiles of 128
    # rows (dA: 2^14 of 1024), each off by at most half a step of what is summed so far
    chain = ((1 << 17) + 2048) * U32
    dl = V.dlogits(l, wlse, c.ids, c.dloss)
    aB = c.s * (np.abs(t64).T @ np.abs(dl))
    aA = c.s * (np.abs(c.x.astype(F64)).T @ (np.abs(dl) @ np.abs(c.B64[:, :vocab]).T))
    within(to_numpy(dA) / times, wA, tA + chain * (aA + tA), "dA")
    within(to_numpy(dB)[:, :vocab] / times, wB[:, :vocab], tB[:, :vocab] + chain * (aB + tB[:, :vocab]), "dB")


def test_entries_at_the_limit_with_the_largest_rank():
    """A layer of 2^27 - 16 columns at rank 32 whose vocabulary is the first few:
    those as a layer of them alone has them, the padding cleared."""
    N, vocab, r, M = (1 << 27) - 16, 1000, 32, 5
    c = Case(M, 16, vocab, r, "w8", "bf16", seed=4, N=1008)
    say("2^27 - 16 columns, rank 32")
    codes = torch.zeros((N, 16), dtype=torch.int8, device="cuda")
    scales = torch.zeros((N,), device="cuda")
    B = torch.zeros((r, N), device="cuda")
    codes[:1008], scales[:1008], B[:, :1008] = c.lin.codes, c.lin.scales, c.lin.B
    wide = Q.QLinear(16, N, r, 16.0, "w8", codes, scales, c.lin.A, B)
    dloss = dev(c.dloss)
    loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=vocab)
    want = Q.qlora_xent_bwd(c.lin, c.x_t, c.ids_t, lse, dloss, t=t, vocab=vocab)
    dB = torch.full((r, N), 7.0, device="cuda")
    got = Q.qlora_xent_bwd(wide, c.x_t, c.ids_t, lse, dloss, t=t, vocab=vocab, dB=dB)
    torch.cuda.synchronize()
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])
    assert torch.equal(dB[:, :1008].contiguous(), want[2])
    assert not any(row.any().item() for row in dB[:, 1008:])
