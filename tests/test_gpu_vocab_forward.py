"""Which forward the loss is that of: int8 layers' qlora_fwd, 4-bit layers'
qlora_fwd_a8w4 (rows of x in 8 bits), not the 4-bit qlora_fwd."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab_oracle as V
from quantized_frozen_weight_amd import binding as Q
from quantized_frozen_weight_amd import workloads as WL
from tests.helpers import to_numpy
from tests.test_gpu_vocab import F64, U16, U32, Case, say, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    Q.lib()   # raises if libqlora.so is missing: no silent fallback


@pytest.mark.parametrize("fmt,dtype", [("w8", "f32"), ("w8", "bf16"), ("w4g128", "bf16")])
@pytest.mark.parametrize("M", [3, 40, 200])
def test_loss_is_that_of_the_integer_forwards_logits(M, fmt, dtype):
    c = Case(M, 512, 700, 4, fmt, dtype, tokens=np.arange(M) * 3 % 700)
    x = c.x.copy()
    x[:, 3::64] *= 60                                     # a few features far above the others
    c.x_t, c.x = WL.as_compute_dtype(x.astype(np.float32), dtype)
    c.x_t = c.x_t.cuda()
    say("forward of the loss", M, fmt, dtype)
    loss, lse, t = Q.qlora_xent_fwd(c.lin, c.x_t, c.ids_t, vocab=700)
    integer = Q.qlora_fwd if fmt == "w8" else Q.qlora_fwd_a8w4
    y, ty = integer(c.lin, c.x_t)
    torch.cuda.synchronize()
    l = to_numpy(y).astype(F64)[:, :700]
    wloss, wlse = V.loss_of(l, c.ids)
    # both form their logits within c.logits()'s bound of the same value; y is then rounded
    _, tol, _, tol_t = c.logits()
    tol_lse = (2 * tol + 1.01 * c.u * np.abs(l)).max(1) + c.lse_tol(l, tol)
    within(to_numpy(lse), wlse, tol_lse, "lse")
    within(to_numpy(loss), wloss, 2 * tol_lse + 4 * U32 * np.abs(wlse), "loss")
    within(to_numpy(t), to_numpy(ty).astype(F64), 2 * tol_t, "t")
    if fmt == "w4g128":
        # x as it is gives other logits: an eight-bit step of these rows is about 1, so each
        # logit is another by some 0.3 x 0.05 x sqrt(512) = 0.3, where the bound is about U16 x 30
        plain = to_numpy(Q.qlora_fwd(c.lin, c.x_t)[0]).astype(F64)[:, :700]
        other, _ = V.loss_of(plain, c.ids)
        assert U16 * np.abs(plain).max() < 0.3
        assert (np.abs(other - to_numpy(loss)) > 2 * tol_lse).mean() > 1 / 3
