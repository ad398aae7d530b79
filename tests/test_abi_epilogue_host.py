"""Host-side checks of the epilogue and checkpoint calls (no GPU needed,
nothing is launched): sizes, and the statuses of arguments that must be
refused before any launch."""

from __future__ import annotations

import ctypes

import pytest

from quantized_frozen_weight_amd import binding as Q

BF, F32 = Q.QLORA_BF16, Q.QLORA_F32
OK, EINVAL, EUNSUP, EWS, ERANGE = Q.QLORA_OK, Q.QLORA_EINVAL, Q.QLORA_EUNSUPPORTED, Q.QLORA_EWORKSPACE, Q.QLORA_ERANGE

# Stand-ins for device buffers, far apart, aligned and never dereferenced.
STEP = 1 << 28
NAMES = ("codes", "scales", "A", "B", "x", "y", "t", "ws", "res", "z", "zc", "zs", "xc", "xs", "bias", "dy", "dx",
         "dA", "dB", "add", "dz", "db")
P = {n: 0x10000000000 + i * STEP for i, n in enumerate(NAMES)}
M, K, N, R = 64, 256, 384, 4
BIG = 1 << 27


@pytest.fixture(scope="module")
def lib():
    return Q.lib()


def layer(fmt=Q.QLORA_W8, heads=0, **kw):
    d = dict(K=K, N=N, r=R)
    d.update(kw)
    return Q.qlora_linear(d["K"], d["N"], d["r"], 8.0, fmt, P["codes"], P["scales"], P["A"], P["B"], heads)


def epi(act=0, **kw):
    e = Q.qlora_epilogue(act=act)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def grad(act=0, **kw):
    g = Q.qlora_grad_epilogue(act=act)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def fwd(lib, L=None, m=M, dt=BF, x=P["x"], e=None, y=P["y"], t=P["t"], ws=P["ws"], n=BIG):
    L = layer() if L is None else L
    ep = ctypes.byref(e) if e is not None else None
    return lib.qlora_fwd_epi(ctypes.byref(L), m, dt, x, ep, y, t, ws, n, None)


def refwd(lib, L=None, m=M, dt=BF, xc=P["xc"], xs=P["xs"], t=P["t"], e=None, y=P["y"], ws=P["ws"], n=BIG):
    L = layer() if L is None else L
    ep = ctypes.byref(e) if e is not None else None
    return lib.qlora_fwd_ckpt(ctypes.byref(L), m, dt, xc, xs, t, ep, y, ws, n, None)


def bwd(lib, L=None, m=M, dt=BF, x=None, xc=P["xc"], xs=P["xs"], dy=P["dy"], t=P["t"], g=None, dx=P["dx"],
        dA=P["dA"], dB=P["dB"], ws=P["ws"], n=BIG):
    L = layer() if L is None else L
    gp = ctypes.byref(g) if g is not None else None
    half = lib.qlora_bwd_epi_partial(ctypes.byref(L), m, dt, x, xc, xs, dy, t, gp, dx, ws, n, None) \
        if dA == P["dA"] and dB == P["dB"] else None
    whole = lib.qlora_bwd_epi(ctypes.byref(L), m, dt, x, xc, xs, dy, t, gp, dx, dA, dB, ws, n, None)
    assert half in (None, whole)
    return whole


def act(lib, a=2, m=M, n=N, dt=BF, dy=P["dy"], z=P["z"], zc=None, zs=None, dz=P["dz"], db=P["db"], ws=P["ws"],
        nb=BIG):
    return lib.qlora_act_bwd(a, m, n, dt, dy, z, zc, zs, dz, db, ws, nb, None)


@pytest.mark.parametrize("M_,C,fmt,want", [
    (1, 16, 0, (16, 4)), (1, 16, 1, (16, 1)), (7, 80, 0, (560, 28)), (7, 80, 1, (560, 21)),
    (4096, 2304, 1, (4096 * 2304, 4096 * 72)), (512, 16384, 0, (512 * 16384, 2048))])
def test_checkpoint_sizes(lib, M_, C, fmt, want):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.qlora_ckpt_bytes(M_, C, fmt, ctypes.byref(a), ctypes.byref(b)) == OK
    assert (a.value, b.value) == want


def test_checkpoint_refusals(lib):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = lambda *k: lib.qlora_ckpt_bytes(*k, ctypes.byref(a), ctypes.byref(b))  # noqa: E731
    assert size(0, 16, 0) == EINVAL and size(1, 8, 0) == EINVAL and size(1, 24, 1) == EINVAL
    assert size(1, 16, 2) == EINVAL and size(1 << 16, 1 << 15, 0) == ERANGE
    assert lib.qlora_ckpt_bytes(1, 16, 0, None, ctypes.byref(b)) == EINVAL
    w = lambda x=P["x"], m=4, c=64, dt=BF, f=1, q=P["zc"], s=P["zs"]: lib.qlora_ckpt_write(x, m, c, dt, f, q, s, None)  # noqa: E731
    r = lambda q=P["zc"], s=P["zs"], m=4, c=64, f=1, dt=BF, x=P["x"]: lib.qlora_ckpt_read(q, s, m, c, f, dt, x, None)  # noqa: E731
    for call in (w, r):
        for kw in (dict(x=None), dict(q=None), dict(s=None), dict(x=P["x"] + 4), dict(q=P["zc"] + 1),
                   dict(s=P["zs"] + 8), dict(m=0), dict(c=40), dict(f=5), dict(dt=9),
                   dict(q=P["x"] + 256), dict(s=P["x"])):
            assert call(**kw) == EINVAL, kw
        assert call(m=1 << 20, c=1 << 12) == ERANGE


def test_forward_refusals(lib):
    assert fwd(lib) == EINVAL                                     # no epilogue
    for call in (fwd, refwd):
        ok = epi(1, bias=P["bias"], residual=P["res"])
        assert call(lib, e=ok, n=100) == EWS and call(lib, e=ok, ws=None) == EWS
        assert call(lib, e=ok, ws=P["ws"] + 4) == EWS
        for a in (-1, 5):
            assert call(lib, e=epi(a)) == EINVAL
        for kw in (dict(bias=P["bias"] + 4), dict(residual=P["res"] + 8), dict(z=P["z"] + 2), dict(z_codes=P["zc"]),
                   dict(z_scales=P["zs"]), dict(z_codes=P["zc"] + 8, z_scales=P["zs"]),
                   # overlaps: outputs over inputs and over each other
                   dict(z=P["y"]), dict(z=P["codes"]), dict(residual=P["y"] + 16), dict(bias=P["y"] + 64),
                   dict(z_codes=P["y"], z_scales=P["zs"]), dict(z_codes=P["zc"], z_scales=P["zc"] + 16),
                   dict(z=P["z"], z_codes=P["z"] + 32, z_scales=P["zs"]), dict(z=P["ws"])):
            assert call(lib, e=epi(2, **kw)) == EINVAL, kw
        for kw in (dict(y=None), dict(y=P["y"] + 2), dict(t=P["t"] + 4), dict(y=P["A"]), dict(m=0),
                   dict(dt=4), dict(L=layer(r=0)), dict(L=layer(K=200))):
            assert call(lib, e=ok, **kw) == EINVAL, kw
        assert call(lib, e=ok, L=layer(fmt=Q.QLORA_W4G128), dt=F32) == EUNSUP
        assert call(lib, e=ok, L=layer(fmt=Q.QLORA_W8O), dt=F32) == EUNSUP
        assert call(lib, e=ok, m=1 << 24) == ERANGE
    for kw in (dict(x=None), dict(x=P["x"] + 2), dict(y=P["x"])):
        assert fwd(lib, e=epi(1), **kw) == EINVAL, kw
    for kw in (dict(x_codes=P["xc"]), dict(x_scales=P["xs"]), dict(x_codes=P["x"], x_scales=P["xs"]),
               dict(x_codes=P["xc"], x_scales=P["t"])):
        assert fwd(lib, e=epi(1, **kw)) == EINVAL, kw
    # from a checkpoint: codes, scales and t are needed, and x is not saved again
    for kw in (dict(xc=None), dict(xs=None), dict(t=None), dict(xc=P["xc"] + 4), dict(y=P["xc"]), dict(y=P["t"])):
        assert refwd(lib, e=epi(1), **kw) == EINVAL, kw
    assert refwd(lib, e=epi(1, x_codes=P["x"], x_scales=P["z"])) == EINVAL


def test_backward_refusals(lib):
    assert bwd(lib, n=100) == EWS and bwd(lib, ws=None) == EWS
    for kw in (dict(x=P["x"]),                                    # both forms of x
               dict(xc=None), dict(xs=None), dict(xc=None, xs=None),
               dict(t=None), dict(t=P["t"] + 4), dict(dy=None), dict(dy=P["dy"] + 2), dict(dx=P["dx"] + 2),
               dict(dx=P["dy"]), dict(dx=P["xc"]), dict(dx=P["ws"] + 64), dict(dx=P["codes"]),
               dict(m=0), dict(dt=3), dict(dA=None), dict(dB=None), dict(dA=P["dB"]), dict(dA=P["A"]),
               dict(dB=P["dx"]), dict(dA=P["dA"] + 4)):
        assert bwd(lib, **kw) == EINVAL, kw
    for kw in (dict(act=7), dict(act=2), dict(act=0, z=P["z"]), dict(act=0, z_codes=P["zc"], z_scales=P["zs"]),
               dict(act=2, z=P["z"], z_codes=P["zc"], z_scales=P["zs"]), dict(act=2, z_codes=P["zc"]),
               dict(act=2, z=P["z"] + 2), dict(act=0, add=P["add"] + 2), dict(act=0, add=P["dx"] + 16),
               dict(act=2, z=P["dx"]), dict(act=2, z_codes=P["dx"], z_scales=P["zs"])):
        assert bwd(lib, g=grad(**kw)) == EINVAL, kw
    assert bwd(lib, g=grad(act=0, add=P["add"]), dx=None) == EINVAL
    assert bwd(lib, L=layer(fmt=Q.QLORA_W4G128), dt=F32) == EUNSUP


def test_activation_backward_refusals(lib):
    n = ctypes.c_size_t(1)
    assert lib.qlora_act_bwd_workspace(64, 384, ctypes.byref(n)) == OK and n.value == 0
    assert lib.qlora_act_bwd_workspace(4096, 2304, ctypes.byref(n)) == OK and n.value >= 2304 * 4
    for m, c, want in ((0, 64, EINVAL), (1, 8, EINVAL), (1, 40, EINVAL), (1 << 16, 1 << 15, ERANGE)):
        assert lib.qlora_act_bwd_workspace(m, c, ctypes.byref(n)) == want
        assert act(lib, m=m, n=c) == want
    assert lib.qlora_act_bwd_workspace(1, 16, None) == EINVAL
    assert act(lib, m=4096, n=2304, nb=64) == EWS and act(lib, m=4096, n=2304, ws=None) == EWS
    for kw in (dict(a=-1), dict(a=5), dict(a=0), dict(z=None), dict(zc=P["zc"]), dict(zc=P["zc"], zs=P["zs"]),
               dict(dy=None), dict(dy=P["dy"] + 2), dict(dz=P["dz"] + 2), dict(db=P["db"] + 4),
               dict(dz=None, db=None), dict(dz=P["dy"] + 16), dict(dz=P["z"]), dict(db=P["dz"]), dict(db=P["dy"]),
               dict(dt=6)):
        assert act(lib, **kw) == EINVAL, kw
