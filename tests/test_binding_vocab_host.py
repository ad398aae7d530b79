"""Host-side checks of the binding's vocabulary and optimizer calls (no GPU
needed): what the tensors have to be."""

from __future__ import annotations

import pytest

from quantized_frozen_weight_amd import binding as Q

torch = pytest.importorskip("torch")

K, N, r = 256, 384, 4
CPU = torch.device("cpu")


def layer(rank=r, **kw):
    z = torch.zeros
    t = dict(codes=z(N, K, dtype=torch.int8), scales=z(N), A=z(K, rank) if rank else None,
             B=z(rank, N) if rank else None)
    t.update(kw)
    return Q.QLinear(K, N, rank, 8.0, "w8", t["codes"], t["scales"], t["A"], t["B"])


def test_a_layer_without_adapter():
    cs, vocab = Q._vocab_on(layer(0), None, CPU)
    assert cs.r == 0 and not cs.A and not cs.B and vocab == N
    assert Q._vocab_on(layer(), 300, CPU)[1] == 300
    with pytest.raises(ValueError, match="rank 0"):
        Q._vocab_on(layer(0, A=torch.zeros(K, 1)), None, CPU)
    with pytest.raises(ValueError):
        Q._vocab_on(layer(0, codes=torch.zeros(K, N, dtype=torch.int8)), None, CPU)
    with pytest.raises(TypeError):
        Q._vocab_on(layer(0, scales=torch.zeros(N, dtype=torch.float64)), None, CPU)


def test_ids_are_checked():
    for dt in (torch.int16, torch.uint8, torch.float32, torch.bool):
        with pytest.raises(TypeError, match="int32 or torch.int64"):
            Q._ids(torch.zeros(5, dtype=dt), "tokens")
    with pytest.raises(ValueError, match="GPU"):
        Q._ids(torch.zeros(5, dtype=torch.int64), "tokens")


def test_calls_refuse_tensors_off_the_gpu():
    x, ids, f = torch.zeros(5, K), torch.zeros(5, dtype=torch.int64), torch.zeros(5)
    for call in (lambda: Q.qlora_embed(layer(), ids), lambda: Q.qlora_embed_bwd(layer(), ids, x),
                 lambda: Q.qlora_xent_fwd(layer(), x, ids), lambda: Q.qlora_xent_bwd(layer(), x, ids, f, f),
                 lambda: Q.AdamW([x]), lambda: Q.qlora_moment_read(ids.to(torch.uint8), ids.to(torch.uint8), "m"),
                 lambda: Q.qlora_moment_write(f, "m")):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_names_are_checked():
    f = torch.zeros(5)
    with pytest.raises(ValueError, match="at least one"):
        Q.AdamW([])
    with pytest.raises(ValueError, match="state form"):
        Q.AdamW([f], state="s4")
    for call in (lambda: Q.qlora_moment_read(f, f, "v"), lambda: Q.qlora_moment_write(f, "v")):
        with pytest.raises(ValueError, match="unknown moment"):
            call()
