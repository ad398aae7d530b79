"""Host-side checks of the binding's epilogue calls (no GPU needed): what the
layer's tensors have to be."""

from __future__ import annotations

import pytest

from quantized_frozen_weight_amd import binding as Q

torch = pytest.importorskip("torch")

K, N, r = 256, 384, 4
CPU = torch.device("cpu")


def layer(fmt, heads=1, **kw):
    z = torch.zeros
    t = dict(A=z(K, r), B=z(heads, r, N // heads) if heads > 1 else z(r, N))
    if fmt == "w4g128":
        t.update(codes=z(N, K // 2, dtype=torch.uint8), scales=z(N, K // 128, dtype=torch.float16))
    else:
        t.update(codes=z(N, K, dtype=torch.int8))
        t.update(scales=z(N) if fmt == "w8" else z(Q.qlora_weight_bytes(K, N, fmt)[1], dtype=torch.uint8))
    t.update(kw)
    return Q.QLinear(K, N, r, 8.0, fmt, t["codes"], t["scales"], t["A"], t["B"], heads)


@pytest.mark.parametrize("fmt", ["w8", "w4g128", "w8o"])
def test_tensors_of_a_layer_are_checked(fmt):
    z = torch.zeros
    good = layer(fmt)
    assert Q._layer_on(good, CPU).K == K
    cw = good.codes.shape[1]
    value = [dict(codes=z(N, cw - 16, dtype=good.codes.dtype)),             # short
             dict(codes=z(N - 16, cw, dtype=good.codes.dtype)),
             dict(codes=z(cw, N, dtype=good.codes.dtype)),                   # the weight the other way round
             dict(codes=z(cw, N, dtype=good.codes.dtype).t()),               # its transposed view
             dict(codes=z(N, 2 * cw, dtype=good.codes.dtype)[:, ::2]),
             dict(scales=good.scales[:-1]), dict(scales=good.scales[::2]),
             dict(codes=good.codes.to("meta")), dict(scales=good.scales.to("meta")),
             dict(A=z(r, K)), dict(A=z(r, K).t()), dict(B=z(N, r)), dict(B=z(1, r, N)), dict(B=z(r, N).to("meta"))]
    kind = [dict(codes=good.codes.short()), dict(scales=good.scales.double()), dict(A=z(K, r).half()),
            dict(B=z(r, N).double())]
    for kws, err in ((value, ValueError), (kind, TypeError)):
        for kw in kws:
            with pytest.raises(err):
                Q._layer_on(layer(fmt, **kw), CPU)
    if fmt != "w8o":
        assert Q._layer_on(layer(fmt, heads=3), CPU).heads == 3
    with pytest.raises(ValueError):
        Q._layer_on(Q.QLinear(K, N, r, 8.0, "w2", good.codes, good.scales, good.A, good.B), CPU)


def test_unknown_checkpoint_forms_are_refused():
    codes, scales = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="unknown checkpoint form"):
        Q.qlora_ckpt_read(Q.Checkpoint(codes, scales, "c8"), torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        Q.qlora_ckpt_read(Q.Checkpoint(codes, scales, "c8g32"), torch.float32)      # not on a GPU
