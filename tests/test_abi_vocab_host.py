"""Host-side checks of the vocabulary layer's and the optimizer's calls (no GPU
needed, nothing is launched): sizes, and the statuses of arguments that must be
refused before any launch."""

from __future__ import annotations

import ctypes

import pytest

from quantized_frozen_weight_amd import binding as Q

BF, F32 = Q.QLORA_BF16, Q.QLORA_F32
OK, EINVAL, EUNSUP, EWS, ERANGE = Q.QLORA_OK, Q.QLORA_EINVAL, Q.QLORA_EUNSUPPORTED, Q.QLORA_EWORKSPACE, Q.QLORA_ERANGE

# Stand-ins for device buffers, far apart, aligned and never dereferenced.
STEP = 1 << 28
NAMES = ("codes", "scales", "A", "B", "ids", "x", "dy", "dx", "dA", "dB", "loss", "lse", "dloss", "t", "ws",
         "p", "g", "m", "v", "ms", "vs", "step", "lr", "norm")
P = {n: 0x10000000000 + i * STEP for i, n in enumerate(NAMES)}
M, K, N, R, VOCAB = 64, 256, 384, 4, 377
BIG = 1 << 27


@pytest.fixture(scope="module")
def lib():
    return Q.lib()


def layer(fmt=Q.QLORA_W8, heads=0, **kw):
    d = dict(K=K, N=N, r=R, codes=P["codes"], scales=P["scales"], A=P["A"], B=P["B"])
    d.update(kw)
    if d["r"] == 0 and "A" not in kw and "B" not in kw:
        d["A"] = d["B"] = None
    return Q.qlora_linear(d["K"], d["N"], d["r"], 8.0, fmt, d["codes"], d["scales"], d["A"], d["B"], heads)


def ref(L):
    return None if L is None else ctypes.byref(L)


def embed(lib, L=layer(), vocab=VOCAB, m=M, dt=BF, ids=P["ids"], it=1, x=P["x"]):
    return lib.qlora_embed(ref(L), vocab, m, dt, ids, it, 1.0, x, None)


def embed_bwd(lib, L=layer(), vocab=VOCAB, m=M, dt=BF, ids=P["ids"], it=1, x=P["dy"], dA=P["dA"], dB=P["dB"],
              ws=P["ws"], n=BIG):
    return lib.qlora_embed_bwd(ref(L), vocab, m, dt, ids, it, 1.0, x, 0, dA, dB, ws, n, None)


def fwd(lib, L=layer(), vocab=VOCAB, m=M, dt=BF, x=P["x"], ids=P["ids"], it=1, loss=P["loss"], lse=P["lse"], t=P["t"],
        ws=P["ws"], n=BIG):
    return lib.qlora_xent_fwd(ref(L), vocab, m, dt, x, ids, it, loss, lse, t, ws, n, None)


def bwd(lib, L=layer(), vocab=VOCAB, m=M, dt=BF, x=P["x"], ids=P["ids"], it=1, lse=P["lse"], dloss=P["dloss"],
        t=P["t"], dx=P["dx"], dA=P["dA"], dB=P["dB"], ws=P["ws"], n=BIG):
    return lib.qlora_xent_bwd(ref(L), vocab, m, dt, x, ids, it, lse, dloss, t, dx, dA, dB, ws, n, None)


CALLS = (embed, embed_bwd, fwd, bwd)


def size(lib, what, L, vocab=VOCAB, m=M, dt=BF):
    n = ctypes.c_size_t()
    st = getattr(lib, f"qlora_{what}_workspace")(ref(L), vocab, m, dt, ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_layers_that_are_refused(lib, call):
    assert call(lib, L=None) == EINVAL
    for kw in (dict(K=250), dict(K=0), dict(N=8), dict(N=390), dict(r=-1), dict(r=33), dict(fmt=7), dict(heads=-1),
               dict(codes=None), dict(codes=P["codes"] + 8), dict(scales=None), dict(scales=P["scales"] + 4),
               dict(A=None), dict(B=None), dict(A=P["A"] + 4), dict(B=P["B"] + 8),
               dict(r=0, A=P["A"], B=P["B"]), dict(r=0, A=None, B=P["B"]),
               dict(fmt=Q.QLORA_W4G128, K=272)):
        assert call(lib, L=layer(**kw)) == EINVAL, kw
    for kw in (dict(fmt=Q.QLORA_W8O), dict(heads=3), dict(fmt=Q.QLORA_W4G128, K=16384 + 128)):
        assert call(lib, L=layer(**kw)) == EUNSUP, kw
    assert call(lib, L=layer(fmt=Q.QLORA_W4G128), dt=F32) == EUNSUP
    for kw in (dict(vocab=0), dict(vocab=-1), dict(vocab=N + 1), dict(m=0), dict(m=-5), dict(dt=7), dict(ids=None),
               dict(ids=P["ids"] + 4), dict(ids=P["ids"] + 2, it=0), dict(it=2), dict(it=-1)):
        assert call(lib, **kw) == EINVAL, kw
    assert call(lib, m=1 << 24) == ERANGE                         # M K
    assert call(lib, L=layer(K=1 << 16, N=1 << 16), vocab=1) == ERANGE


def test_embed_refusals(lib):
    for kw in (dict(x=None), dict(x=P["x"] + 2), dict(x=P["codes"] + 32), dict(x=P["scales"]), dict(x=P["A"]),
               dict(x=P["B"] + 64), dict(x=P["ids"] + 16)):
        assert embed(lib, **kw) == EINVAL, kw


def test_embed_gradient_refusals(lib):
    for kw in (dict(x=None), dict(x=P["dy"] + 2), dict(dA=None), dict(dB=None), dict(dA=P["dA"] + 4),
               dict(dB=P["dB"] + 8), dict(dA=P["dy"]), dict(dA=P["dB"] + 16), dict(dB=P["B"]), dict(dA=P["A"]),
               dict(dA=P["ws"]), dict(dB=P["ids"]), dict(L=layer(r=0))):
        assert embed_bwd(lib, **kw) == EINVAL, kw
    for kw in (dict(n=100), dict(ws=None), dict(ws=P["ws"] + 8)):
        assert embed_bwd(lib, **kw) == EWS, kw
    small = layer(K=16)
    assert size(lib, "embed_bwd", small, m=1 << 20)[0] == OK
    assert size(lib, "embed_bwd", small, m=(1 << 20) + 1)[0] == ERANGE
    assert size(lib, "embed_bwd", layer(r=0))[0] == EINVAL
    # a row's place, u and the partial sums of dA at least
    st, n = size(lib, "embed_bwd", layer())
    assert st == OK and n >= M * (R + 2) * 4 + 2 * K * R * 4


def test_loss_refusals(lib):
    for kw in (dict(x=None), dict(x=P["x"] + 2), dict(loss=None), dict(loss=P["loss"] + 4), dict(lse=None),
               dict(lse=P["lse"] + 4), dict(t=P["t"] + 4), dict(loss=P["lse"] + 16), dict(t=P["x"]), dict(lse=P["ids"]),
               dict(loss=P["ws"] + 256), dict(L=layer(r=0))):                    # (t where r = 0)
        assert fwd(lib, **kw) == EINVAL, kw
    for kw in (dict(n=64), dict(ws=None), dict(ws=P["ws"] + 4)):
        assert fwd(lib, **kw) == EWS, kw
    for what in ("xent_fwd", "xent_bwd"):
        f = getattr(lib, f"qlora_{what}_workspace")
        assert f(ref(layer()), VOCAB, M, BF, None) == EINVAL
        assert size(lib, what, layer(K=132096, N=16), vocab=9, m=1)[0] == OK
        assert size(lib, what, layer(K=132112, N=16), vocab=9, m=1)[0] == EUNSUP
        assert size(lib, what, layer(fmt=Q.QLORA_W4G128, K=16384))[0] == OK
        # rows, and rows times entries, of one launch
        assert size(lib, what, layer(K=16, N=16), vocab=16, m=1 << 24)[0] == OK
        assert size(lib, what, layer(K=16, N=16), vocab=16, m=(1 << 24) + 1)[0] == ERANGE
        assert size(lib, what, layer(K=16, N=1 << 20), vocab=1 << 20, m=1 << 17)[0] == OK
        assert size(lib, what, layer(K=16, N=1 << 20), vocab=1 << 20, m=(1 << 17) + 1)[0] == ERANGE


def test_loss_gradient_refusals(lib):
    for kw in (dict(x=None), dict(x=P["x"] + 2), dict(lse=None), dict(lse=P["lse"] + 8), dict(dloss=None),
               dict(dloss=P["dloss"] + 4), dict(t=P["t"] + 4), dict(dx=P["dx"] + 2), dict(dA=None), dict(dB=None),
               dict(dA=P["dA"] + 4), dict(dB=P["dB"] + 4), dict(dx=P["x"]), dict(dx=P["lse"]), dict(dA=P["t"]),
               dict(dB=P["dloss"]), dict(dA=P["dB"]), dict(dx=P["ws"]), dict(dB=P["codes"]),
               # no adapter: no t, dA or dB, and dx is all there is
               dict(L=layer(r=0)), dict(L=layer(r=0), t=None), dict(L=layer(r=0), t=None, dA=None),
               dict(L=layer(r=0), t=None, dA=None, dB=None, dx=None)):
        assert bwd(lib, **kw) == EINVAL, kw
    for kw in (dict(n=64), dict(ws=None), dict(ws=P["ws"] + 4)):
        assert bwd(lib, **kw) == EWS, kw
        assert bwd(lib, L=layer(r=0), t=None, dA=None, dB=None, **kw) == EWS, kw


def test_workspaces_grow_with_what_they_hold(lib):
    for what in ("xent_fwd", "xent_bwd", "embed_bwd"):
        last = 0
        for m in (1, 32, 33, 256, 4096, 9000):
            st, n = size(lib, what, layer(), m=m)
            assert st == OK and n >= last
            last = n
    # 50257 entries of 4096 rows: the loss keeps 8 bytes a row and 256 entries and the
    # rows' codes, not the logits
    big = layer(K=768, N=50272, r=8)
    st, n = size(lib, "xent_fwd", big, vocab=50257, m=4096)
    assert st == OK and n < 4096 * (768 + 4 * 8 + 2 * 8 * 393 + 4096) < 2 * 4096 * 50257 // 8


def item(**kw):
    d = dict(p=P["p"], g=P["g"], m=P["m"], v=P["v"], ms=None, vs=None, n=1000, decay=0.01)
    d.update(kw)
    return Q.qlora_adamw_item(d["p"], d["g"], d["m"], d["v"], d["ms"], d["vs"], d["n"], d["decay"])


def config(**kw):
    c = Q.qlora_adamw_config(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-6, clip_norm=1.0, step=P["step"], seed=1, sfmt=0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def adamw(lib, c=config(), items=(item(),), count=None, ws=P["ws"], n=BIG):
    a = (Q.qlora_adamw_item * max(len(items), 1))(*items)
    return lib.qlora_adamw(ref(c), a if items else None, len(items) if count is None else count, ws, n, None)


def test_adamw_refusals(lib):
    nan, inf = float("nan"), float("inf")
    assert adamw(lib, c=None) == EINVAL and adamw(lib, items=()) == EINVAL and adamw(lib, count=0) == EINVAL
    for kw in (dict(step=None), dict(step=P["step"] + 2), dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(eps=0.0),
               dict(eps=1e-60), dict(eps=nan), dict(eps=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=nan),
               dict(beta2=1.0), dict(beta2=nan), dict(clip_norm=-1.0), dict(clip_norm=nan), dict(clip_norm=inf),
               dict(clip_norm=1e-60), dict(sfmt=2), dict(lr_dev=P["lr"] + 1), dict(norm=P["norm"] + 2),
               dict(norm=P["p"]), dict(norm=P["step"]), dict(step=P["m"]), dict(lr_dev=P["step"])):
        assert adamw(lib, c=config(**kw)) == EINVAL, kw
    for kw in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=P["p"] + 4), dict(g=P["g"] + 8),
               dict(m=P["m"] + 4), dict(v=P["v"] + 4), dict(n=0), dict(n=-3), dict(decay=-0.1), dict(decay=nan),
               dict(decay=inf), dict(ms=P["ms"]), dict(ms=P["ms"], vs=P["vs"]), dict(g=P["p"]), dict(m=P["g"] + 16),
               dict(v=P["m"] + 3984), dict(p=P["ws"])):
        assert adamw(lib, items=(item(), item(**kw))) == EINVAL, kw
    s8 = config(sfmt=Q._SFMT["s8"])
    for kw in (dict(), dict(ms=P["ms"]), dict(vs=P["vs"]), dict(ms=P["m"] + 992, vs=P["vs"]),
               dict(ms=P["ms"], vs=P["ms"] + 31)):
        assert adamw(lib, c=s8, items=(item(**kw),)) == EINVAL, kw
    assert adamw(lib, items=(item(n=(1 << 30) + 1),)) == ERANGE
    for kw in (dict(n=16), dict(ws=None), dict(ws=P["ws"] + 8)):
        assert adamw(lib, **kw) == EWS, kw
    n = ctypes.c_size_t()
    a = (Q.qlora_adamw_item * 3)(item(), item(n=1 << 30), item(n=7))
    assert lib.qlora_adamw_workspace(a, 3, ctypes.byref(n)) == OK and 0 < n.value < 1 << 16
    assert lib.qlora_adamw_workspace(a, 3, None) == EINVAL and lib.qlora_adamw_workspace(None, 3, ctypes.byref(n)) == EINVAL


def test_moment_refusals(lib):
    r = lambda c=P["m"], s=P["ms"], n=100, w=0, dt=F32, x=P["x"]: lib.qlora_moment_read(c, s, n, w, dt, x, None)  # noqa: E731
    w = lambda c=P["m"], s=P["ms"], n=100, w=0, dt=F32, x=P["x"]: lib.qlora_moment_write(x, n, w, dt, c, s, None)  # noqa: E731
    for call in (r, w):
        for kw in (dict(c=None), dict(s=None), dict(x=None), dict(c=P["m"] + 8), dict(x=P["x"] + 4), dict(n=0),
                   dict(n=-1), dict(w=2), dict(w=-1), dict(dt=5), dict(c=P["x"] + 16), dict(s=P["x"])):
            assert call(**kw) == EINVAL, kw
        assert call(n=(1 << 30) + 1) == ERANGE
    assert w(s=P["m"] + 99) == EINVAL                             # (both are written)
