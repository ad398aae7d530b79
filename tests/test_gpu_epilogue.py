"""The layer with its epilogue, the 8-bit activation checkpoints and the
backward from them, on the GPU against the float64 oracle.

Tolerances are bounds, element by element: half a step of the output's type
(2^-8 of the value in bfloat16, 2^-24 in float32) plus what float32 sums of
the given length and the rounding of dequantized weights to bfloat16 can add
to these very inputs (sums of absolute products, from the oracle's operands).
"""

from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import epilogue_oracle as E
from oracle import qlora_oracle as O
from quantized_frozen_weight_amd import binding as Q
from quantized_frozen_weight_amd import workloads as WL
from tests.helpers import to_numpy

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24          # half a step of float32, relative
U16 = 2.0 ** -8           # of bfloat16
ACT_REL = 2e-5            # float32 activations in their far tails, relative to act(z)
SLOPE_ABS = 4e-6          # float32 slopes
LIPSCHITZ = 1.13          # the steepest act
F64 = np.float64


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
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32) if t.element_size() == 4 else t


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


class Case:
    """A layer with its inputs on the device and its oracle operands."""

    def __init__(self, M, K, N, r, fmt="w8", dtype="bf16", heads=1, seed=0, alpha=16.0):
        rng = np.random.default_rng(seed)
        self.M, self.K, self.N, self.r, self.fmt, self.dtype, self.heads = M, K, N, r, fmt, dtype, heads
        n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        W = (0.05 * rng.standard_t(3, (K, N))).astype(np.float32) if fmt == "w8o" else 0.05 * n(K, N)
        self.A, self.B = 0.05 * n(K, r), 0.05 * n(r, N)
        if heads > 1:
            hd = N // heads
            codes, scales = Q.qlora_quantize(dev(W.reshape(K, heads, hd).transpose(1, 0, 2)), fmt)
            B = dev(O.plain_to_heads(self.B, heads))
        else:
            codes, scales = Q.qlora_quantize(dev(W), fmt)
            B = dev(self.B)
        self.lin = Q.QLinear(K, N, r, alpha, fmt, codes, scales, dev(self.A), B, heads)
        self.s = float(O.lora_scale(alpha, r))
        x = n(M, K)
        self.x_t, self.x = WL.as_compute_dtype(x, dtype)
        self.dy_t, self.dy = WL.as_compute_dtype(n(M, N), dtype)
        self.res_t, self.res = WL.as_compute_dtype(n(M, N), dtype)
        self.add_t, self.add = WL.as_compute_dtype(n(M, K), dtype)
        self.z_t, self.z = WL.as_compute_dtype(n(M, K), dtype)
        for a in ("x_t", "dy_t", "res_t", "add_t", "z_t"):
            setattr(self, a, getattr(self, a).cuda())
        self.bias = n(N)
        self.td = self.x_t.dtype
        self.u = U16 if dtype == "bf16" else U32
        # the weight in float64, and a bound on what a product's float32 work
        # adds, per unit of sum |x| |W|
        if fmt == "w8":
            oc, osc = O.quantize_w8(W)
            self.W = O.dequant_w8(oc, osc)
            self.Wabs = np.abs(self.W)
            self.fwd_rel = 4 * U32                       # exact integer sums, three float32 steps
        elif fmt == "w8o":
            q = O.quantize_w8o(W)
            self.W = O.dequant_w8o(q).astype(F64)
            # the affine form adds c acc, b' sum(xq) and the outliers apart
            self.Wabs = np.abs(self.W) + 2 * (abs(float(q["lo"])) + abs(float(q["hi"])))
            self.fwd_rel = K * U32
        else:
            packed, sc = O.quantize_w4(W)
            self.W = O.dequant_w4(packed, sc)
            self.Wabs = np.abs(self.W)
            self.fwd_rel = U16 + (K + 2) * U32           # weights rounded to bfloat16
            self.int_rel = (K // 128 + 4) * U32          # integer sums per group
        self.bwd_rel = (U16 if dtype == "bf16" else 2 * U32) + (N + 2) * U32
        self.B64, self.A64 = self.B.astype(F64), self.A.astype(F64)

    def forward(self, act, bias, residual, from_ckpt=False):
        """(y, z, t, bounds of each) in float64."""
        x64 = self.x.astype(F64)
        t = x64 @ self.A64
        tol_t = self.K * U32 * (np.abs(x64) @ np.abs(self.A64))
        if self.fmt == "w4g128" and not from_ckpt:
            xh, rel = x64, self.fwd_rel
        else:
            xq, sx = O.quantize_rows(self.x)
            xh = E.read_rows(xq, sx)
            rel = self.int_rel if self.fmt == "w4g128" else self.fwd_rel
        base = xh @ self.W
        low = self.s * (t @ self.B64)
        b = self.bias.astype(F64) if bias else np.zeros(self.N)
        z = base + low + b
        tol_z = (rel * (np.abs(xh) @ self.Wabs) + self.s * (tol_t @ np.abs(self.B64)
                 + (self.r + 2) * U32 * (np.abs(t) @ np.abs(self.B64)))
                 + 2 * U32 * (np.abs(base) + np.abs(low) + np.abs(b)))
        a = E.act(act, z)
        res = self.res.astype(F64) if residual else 0.0
        y = a + res
        tol_y = LIPSCHITZ * tol_z + ACT_REL * np.abs(a) + U32 * (np.abs(a) + np.abs(res)) + 1e-30
        return (y, z, t), (self.u * (np.abs(y) + tol_y) + tol_y, tol_z, tol_t)

    def backward(self, act, z64, add, t64, x64):
        """(dx, dA, dB) in float64 and their bounds."""
        dy = self.dy.astype(F64)
        u = dy @ self.B64.T
        tol_u = (self.N + 8) * U32 * (np.abs(dy) @ np.abs(self.B64).T)
        dB = self.s * (t64.T @ dy)
        dA = self.s * (x64.T @ u)
        tol_dB = self.s * (self.M + 8) * U32 * (np.abs(t64).T @ np.abs(dy)) + 1e-30
        tol_dA = self.s * np.abs(x64).T @ (tol_u + (self.M + 8) * U32 * np.abs(u)) + 1e-30
        dx0 = dy @ self.W.T + self.s * (u @ self.A64.T)
        tol0 = (self.bwd_rel * (np.abs(dy) @ self.Wabs.T)
                + self.s * (tol_u @ np.abs(self.A64).T + (self.r + 2) * U32 * (np.abs(u) @ np.abs(self.A64).T)))
        sl = E.slope(act, z64) if act != "none" else np.ones_like(dx0)
        a = self.add.astype(F64) if add else 0.0
        dx = dx0 * sl + a
        tol = np.abs(sl) * tol0 + SLOPE_ABS * (np.abs(dx0) + tol0) + 3 * U32 * (np.abs(dx0 * sl) + np.abs(a))
        return (dx, dA, dB), (self.u * (np.abs(dx) + tol) + tol + 1e-30, tol_dA, tol_dB)


def check_group_ckpt(ck, z, tol_z, what):
    """A group checkpoint written from a z known to within tol_z."""
    codes, byte = ck.codes.cpu().numpy(), ck.scales.cpu().numpy()
    v = E.read_groups(codes, byte)
    M, C = z.shape
    step = np.repeat(2.0 ** (byte.astype(F64) - 127), 32, 1)[:, :C]
    half = np.where(np.abs(codes) == 1, 1.0, 0.5)
    within(v, z, half * step + tol_z, f"{what}: values")
    sure = np.abs(z) > tol_z
    assert np.array_equal(np.sign(v)[sure], np.sign(z)[sure]), f"{what}: signs"
    g = lambda a: np.pad(a, ((0, 0), (0, -C % 32))).reshape(M, -1, 32).max(2)  # noqa: E731
    top, tol = g(np.abs(z)), g(tol_z)
    unit = 2.0 ** (byte.astype(F64) - 127)
    assert np.all(top - tol <= 127 * unit) and np.all(top + tol > 127 * unit / 2), f"{what}: scales"


# (M, K, N, r, fmt, dtype, heads): one per kernel family and ragged edge
FWD = [
    (64, 256, 256, 4, "w8", "f32", 1),
    (1, 16, 16, 1, "w8", "f32", 1),            # the smallest layer
    (130, 144, 272, 32, "w8", "f32", 1),
    (1, 2048, 1040, 8, "w8", "bf16", 1),       # one token
    (2, 208, 80, 1, "w8", "f32", 1),           # few rows, ranks below the padded ones
    (3, 784, 16400, 3, "w8", "bf16", 1),       # ... wide: 64 columns a block, a ragged one
    (4, 16384, 272, 8, "w8", "bf16", 1),       # ... long rows: codes in two batches
    (4, 4096, 8256, 16, "w8", "bf16", 3),      # ... heads, 32 columns a block
    (4, 16384, 144, 16, "w4g128", "bf16", 1),
    (3, 128, 16, 4, "w4g128", "bf16", 1),
    (4, 256, 144, 32, "w8", "bf16", 1),        # rank 32: the tiled product
    (7, 784, 208, 3, "w8", "bf16", 1),
    (1001, 784, 1024, 8, "w8", "bf16", 1),     # 64 x 64 tiles, ragged rows and k
    (700, 256, 4112, 16, "w8", "bf16", 1),     # ... last group of 16 columns
    (2100, 128, 2304, 4, "w8", "bf16", 1),     # 128 x 64 tiles (128 x 192 without an epilogue)
    (2100, 128, 4096, 32, "w8", "bf16", 1),    # ... at rank 32 (128 x 128 without)
    (2100, 1040, 4112, 32, "w8", "bf16", 1),   # 128 x 128 tiles, rank 32, ragged k and columns
    (4100, 1168, 2064, 3, "w8", "bf16", 1),    # ... at rank 3
    (100, 4096, 272, 8, "w8", "bf16", 1),      # split contraction and its second launch
    (130, 16384, 144, 4, "w8", "bf16", 1),     # split 8 ways, long rows
    (40, 4096, 144, 8, "w8", "f32", 1),        # split, float32 outputs
    (300, 256, 384, 4, "w8", "bf16", 3),       # heads
    (100, 256, 384, 8, "w8o", "bf16", 1),
    (257, 1024, 192, 32, "w8o", "bf16", 1),
    (130, 4096, 80, 4, "w8o", "bf16", 1),      # affine, split
    (1, 512, 144, 16, "w8o", "bf16", 1),
    (77, 256, 272, 8, "w4g128", "bf16", 1),    # 4-bit, 64-row tiles
    (1, 1024, 528, 4, "w4g128", "bf16", 1),
    (600, 256, 8320, 4, "w4g128", "bf16", 1),  # 4-bit, 128-row tiles
    (90, 8192, 144, 32, "w4g128", "bf16", 1),  # 4-bit, split, wide scale slab
    (2100, 4224, 2064, 32, "w4g128", "bf16", 1),  # 4-bit, 128-row tiles over more than 32 groups
]
MIXES = [("gelu", True, True, "c8g32"), ("relu", True, False, "full"), ("silu", False, True, "c8g32"),
         ("gelu_tanh", True, True, "full"), ("none", True, False, "c8g32")]


@pytest.mark.parametrize("spec", FWD, ids=lambda s: "-".join(map(str, s)))
def test_forward(spec):
    c = Case(*spec)
    # every activation on the small cases, two of them on the large
    some = MIXES if c.M * c.K * c.N < 3e8 else MIXES[:2]
    for act, bias, residual, save_z in some:
        say("fwd_epi", spec, act, bias, residual, save_z)
        kw = dict(act=act, bias=dev(c.bias) if bias else None, residual=c.res_t if residual else None, save_z=save_z)
        y, t, z, xc = Q.qlora_fwd_epi(c.lin, c.x_t, save_x=True, **kw)
        torch.cuda.synchronize()
        (wy, wz, wt), (ty, tz, tt) = c.forward(act, bias, residual)
        within(to_numpy(t), wt, tt, "t")
        within(to_numpy(y), wy, ty, "y")
        if save_z == "full":
            within(to_numpy(z), wz, c.u * (np.abs(wz) + tz) + tz, "z")
        else:
            check_group_ckpt(z, wz, tz, "z")
        oq, osx = O.quantize_rows(c.x)
        assert np.array_equal(xc.codes.cpu().numpy(), oq), "x codes"
        assert np.array_equal(xc.scales.cpu().numpy().view(np.uint32), osx.view(np.uint32)), "x scales"
        # again from the checkpoint
        say("fwd_ckpt", spec, act)
        y2, z2 = Q.qlora_fwd_ckpt(c.lin, xc, t, c.td, **kw)
        torch.cuda.synchronize()
        if c.fmt == "w4g128":
            (wy, wz, _), (ty, tz, _) = c.forward(act, bias, residual, from_ckpt=True)
            within(to_numpy(y2), wy, ty, "y from the checkpoint")
        else:
            within(to_numpy(y2), wy, ty, "y from the checkpoint")
            if c.M > 8:   # (few rows take a product of their own the first time)
                assert torch.equal(bits(y), bits(y2)), "y from the checkpoint differs"


@pytest.mark.parametrize("spec", [f for f in FWD if f[0] in (64, 1001, 100, 77, 90, 300, 700, 2100)],
                         ids=lambda s: "-".join(map(str, s)))
def test_empty_epilogue_is_the_plain_forward(spec):
    c = Case(*spec)
    say("empty epilogue", spec)
    y, t = Q.qlora_fwd(c.lin, c.x_t)
    y2, t2, z, xc = Q.qlora_fwd_epi(c.lin, c.x_t)
    y3, _, _, _ = Q.qlora_fwd_epi(c.lin, c.x_t, save_t=False)
    torch.cuda.synchronize()
    assert z is None and xc is None
    for a, b in ((y, y2), (t, t2), (y, y3)):
        assert torch.equal(bits(a), bits(b))


BWD = [
    (64, 256, 256, 4, "w8", "f32", 1),
    (1, 16, 16, 1, "w8", "f32", 1),
    (130, 144, 272, 32, "w8", "f32", 1),
    (1, 256, 144, 3, "w8", "bf16", 1),
    (1024, 256, 1024, 8, "w8", "bf16", 1),     # 64-row tiles, scales and B resident
    (333, 208, 400, 32, "w8", "bf16", 1),      # 64-row tiles, ragged
    (4200, 528, 272, 4, "w8", "bf16", 1),      # 128 x 64 tiles, ragged
    (2100, 2064, 144, 16, "w8", "bf16", 1),    # 128 x 128 tiles
    (2100, 2064, 144, 8, "w8", "bf16", 1),     # ... at rank 8
    (130, 528, 2080, 4, "w8", "bf16", 1),      # split
    (70, 144, 8320, 8, "w8", "bf16", 1),       # split 8 ways
    (300, 256, 384, 4, "w8", "bf16", 3),       # heads
    (100, 256, 384, 8, "w8o", "bf16", 1),
    (2100, 2064, 144, 4, "w8o", "bf16", 1),
    (70, 208, 2080, 4, "w8o", "bf16", 1),      # affine, split
    (77, 256, 272, 8, "w4g128", "bf16", 1),
    (77, 384, 144, 32, "w4g128", "bf16", 1),   # 4-bit, rank 32: 128-row tiles
    (4200, 2176, 80, 16, "w4g128", "bf16", 1),
    (77, 256, 4160, 8, "w4g128", "bf16", 1),   # 4-bit, split
    # with the weight laid out first (from 1024 rows and 2^19 weights)
    (1030, 1040, 528, 8, "w8", "bf16", 1),     # 64 x 64 tiles
    (1024, 1056, 576, 3, "w8", "bf16", 3),     # ... heads, whole row tiles
    (4200, 528, 1040, 1, "w8", "bf16", 1),     # 128 x 64 tiles
    (4200, 1040, 528, 32, "w8", "bf16", 1),    # 128 x 128 tiles, rank 32
    (4200, 1056, 576, 16, "w8", "bf16", 3),    # ... heads
    (1030, 528, 2080, 4, "w8", "bf16", 1),     # split 4 ways
    (1100, 144, 8208, 16, "w8", "bf16", 1),    # split 8 ways, ragged last stage
    (1100, 1152, 528, 4, "w4g128", "bf16", 1),
    (1100, 1152, 528, 32, "w4g128", "bf16", 1),  # 4-bit, rank 32: 128 x 64 tiles
    (4200, 1152, 464, 16, "w4g128", "bf16", 1),  # 4-bit, 128 x 128 tiles
    (1030, 256, 2064, 8, "w4g128", "bf16", 1),   # 4-bit, split
]
GRADS = [("gelu", "c8", False), ("relu", "full", True), ("silu", "c8", True), ("gelu_tanh", "c8", False),
         ("none", None, True), ("none", None, False)]


@pytest.mark.parametrize("spec", BWD, ids=lambda s: "-".join(map(str, s)))
def test_backward(spec):
    c = Case(*spec)
    _, t = Q.qlora_fwd(c.lin, c.x_t)
    torch.cuda.synchronize()
    t64 = to_numpy(t).astype(F64)
    oq, osx = O.quantize_rows(c.x)
    xc = Q.Checkpoint(dev(oq), dev(osx), "c8row")
    zq, zb = E.write_groups(c.z)
    zc = Q.Checkpoint(dev(zq), dev(zb), "c8g32")
    for act, zform, add in GRADS:
        z64 = None if zform is None else E.read_groups(zq, zb) if zform == "c8" else c.z.astype(F64)
        zarg = {None: None, "c8": zc, "full": c.z_t}[zform]
        kw = dict(act=act, z=zarg, add=c.add_t if add else None)
        for x, x64, what in ((xc, E.read_rows(oq, osx), "x in 8 bits"), (c.x_t, c.x.astype(F64), "x dense")):
            say("bwd_epi", spec, act, zform, add, what)
            dx, dA, dB = Q.qlora_bwd_epi(c.lin, x, c.dy_t, t, **kw)
            torch.cuda.synchronize()
            (wx, wA, wB), (tx, tA, tB) = c.backward(act, z64, add, t64, x64)
            within(to_numpy(dx), wx, tx, f"dx ({what})")
            within(to_numpy(dA), wA, tA, f"dA ({what})")
            gB = to_numpy(dB)
            within(O.heads_to_plain(gB) if c.heads > 1 else gB, wB, tB, f"dB ({what})")
    # in two halves, and without dx
    say("bwd_epi halves", spec)
    full = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, act="gelu", z=zc, add=c.add_t)
    dx, ws = Q.qlora_bwd_epi_partial(c.lin, xc, c.dy_t, t, act="gelu", z=zc, add=c.add_t)
    dA, dB = Q.qlora_bwd_finish(c.lin, c.M, c.td, ws)
    none, dA0, dB0 = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, need_dx=False)
    torch.cuda.synchronize()
    for a, b in zip(full, (dx, dA, dB)):
        assert torch.equal(bits(a), bits(b)), "halves differ"
    (_, wA, wB), (_, tA, tB) = c.backward("none", None, False, t64, E.read_rows(oq, osx))
    assert none is None
    within(to_numpy(dA0), wA, tA, "dA without dx")
    gB = to_numpy(dB0)
    within(O.heads_to_plain(gB) if c.heads > 1 else gB, wB, tB, "dB without dx")


@pytest.mark.parametrize("spec", [BWD[0], BWD[4], BWD[7], BWD[9], BWD[12], BWD[15]],
                         ids=lambda s: "-".join(map(str, s)))
def test_empty_gradient_epilogue_is_the_plain_backward(spec):
    c = Case(*spec)
    say("plain backward", spec)
    _, t = Q.qlora_fwd(c.lin, c.x_t)
    want = Q.qlora_bwd(c.lin, c.x_t, c.dy_t, t=t)
    same = Q.qlora_bwd_epi(c.lin, c.x_t, c.dy_t, t)
    notx = Q.qlora_bwd_epi(c.lin, c.x_t, c.dy_t)                  # t recomputed from x
    xc = Q.qlora_ckpt_write(c.x_t)
    ck = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t)
    torch.cuda.synchronize()
    for a, b in zip(want, same):
        assert torch.equal(bits(a), bits(b))
    assert torch.equal(bits(want[0]), bits(notx[0])) and torch.equal(bits(want[1]), bits(notx[1]))
    # x enters dA alone: dx and dB are the same bytes from a checkpoint
    assert torch.equal(bits(want[0]), bits(ck[0])) and torch.equal(bits(want[2]), bits(ck[2]))


def test_gradients_are_differences_of_the_forward():
    """dA and dB of the whole chain act(z) + residual against differences of
    the float32 forward (the base product is piecewise constant in x, so the
    adapter is what is differentiated)."""
    c = Case(48, 64, 80, 4, "w8", "f32", seed=3)
    say("differences")
    bias = dev(c.bias)
    act = "gelu"
    # a forward whose x dependence is only through the adapter's parameters
    y, t, z, xc = Q.qlora_fwd_epi(c.lin, c.x_t, act=act, bias=bias, residual=c.res_t, save_z="full", save_x=True)
    dz, dbias = Q.qlora_act_bwd(act, c.dy_t, z)
    _, dA, dB = Q.qlora_bwd_epi(c.lin, c.x_t, dz, t)
    A0, B0 = c.lin.A.clone(), c.lin.B.clone()
    b0 = bias.clone()

    def loss():
        # in float64 from the float32 outputs
        out = Q.qlora_fwd_epi(c.lin, c.x_t, act=act, bias=bias, residual=c.res_t)[0]
        return float((out.double() * c.dy_t.double()).sum())

    rng = np.random.default_rng(1)
    h = 2.0 ** -6
    for name, param, grad, base in (("A", c.lin.A, dA, A0), ("B", c.lin.B, dB, B0), ("bias", bias, dbias, b0)):
        d = dev(rng.standard_normal(tuple(param.shape)).astype(np.float32))
        param.copy_(base + h * d)
        up = loss()
        param.copy_(base - h * d)
        down = loss()
        param.copy_(base)
        got = float((grad.double() * d.double()).sum())
        # rounding of 48 * 80 float32 outputs and their sums, over 2 h; and the
        # third derivative (|gelu'''| < 1.2) of z along d: h^2 / 6 sum |dy| |dz/dh|^3
        t64 = c.x.astype(F64) @ A0.cpu().numpy().astype(F64)
        dn = d.cpu().numpy().astype(F64)
        zdot = (c.s * (c.x.astype(F64) @ dn @ c.B64) if name == "A"
                else c.s * (t64 @ dn) if name == "B" else np.broadcast_to(dn, (48, 80)))
        ysz = float((np.abs(to_numpy(y)) * np.abs(c.dy)).sum())
        bound = 80 * U32 * ysz / h + h * h / 6 * 1.2 * float((np.abs(c.dy) * np.abs(zdot) ** 3).sum()) \
            + 1e-5 * float(np.abs(grad.cpu().numpy().astype(F64) * dn).sum())
        assert abs((up - down) / (2 * h) - got) <= bound, (name, up, down, got, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", [(1, 16), (3, 48), (5, 80), (130, 1040), (1000, 16384), (4096, 2304), (1, 65536), (6, 16400),
                                 (7, 40016)])
def test_checkpoints_bit_exact(M, C, dtype):
    rng = np.random.default_rng(M * C)
    x = rng.standard_normal((M, C)).astype(np.float32) * (10.0 ** rng.integers(-6, 6, (M, 1))).astype(np.float32)
    x[0, 3] = 1e-30                                # far below its row: a sign, no more
    if M > 4:
        x[1] = 0
        x[2, 7], x[3, 9], x[4, 11] = np.inf, np.nan, -3e38
    x_t, x = WL.as_compute_dtype(x, dtype)
    x_t = x_t.cuda()
    say("checkpoints", M, C, dtype)
    g = Q.qlora_ckpt_write(x_t, "c8g32")
    rw = Q.qlora_ckpt_write(x_t, "c8row")
    gv, rv = Q.qlora_ckpt_read(g, x_t.dtype), Q.qlora_ckpt_read(rw, x_t.dtype)
    torch.cuda.synchronize()
    q, b = E.write_groups(x)
    assert np.array_equal(g.scales.cpu().numpy(), b), "group scales"
    assert np.array_equal(g.codes.cpu().numpy(), q), "group codes"
    want = E.read_groups(q, b)
    assert np.array_equal(to_numpy(gv), want, equal_nan=True), "group values"
    oq, osx = O.quantize_rows(x)
    assert np.array_equal(rw.codes.cpu().numpy(), oq), "row codes"
    s = rw.scales.cpu().numpy()
    assert np.array_equal(s, osx, equal_nan=True), "row scales"
    with np.errstate(over="ignore", invalid="ignore"):
        want = O.round_to(E.read_rows(oq, osx), dtype)
    assert np.array_equal(to_numpy(rv), want, equal_nan=True), "row values"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 16), (77, 1040), (128, 48), (129, 272), (1000, 4112), (2500, 272), (5000, 144)])
def test_activation_backward(M, N, dtype):
    rng = np.random.default_rng(M + N)
    dy_t, dy = WL.as_compute_dtype(rng.standard_normal((M, N)).astype(np.float32), dtype)
    z_t, z = WL.as_compute_dtype(3 * rng.standard_normal((M, N)).astype(np.float32), dtype)
    dy_t, z_t = dy_t.cuda(), z_t.cuda()
    q, b = E.write_groups(z)
    u = U16 if dtype == "bf16" else U32
    for act in E.ACTS:
        for zarg, z64 in ((Q.Checkpoint(dev(q), dev(b), "c8g32"), E.read_groups(q, b)), (z_t, z.astype(F64))):
            say("act_bwd", M, N, dtype, act)
            if act == "none":
                zarg = None
            dz, db = Q.qlora_act_bwd(act, dy_t, zarg)
            sl = E.slope(act, z64)
            w = dy.astype(F64) * sl
            tol = (SLOPE_ABS * (act != "none") + U32) * np.abs(dy) + U32 * np.abs(w)
            within(to_numpy(dz), w, u * (np.abs(w) + tol) + tol, "dz")
            within(to_numpy(db), w.sum(0), tol.sum(0) + M * U32 * np.abs(w).sum(0) + 1e-30, "dbias")
            only, none = Q.qlora_act_bwd(act, dy_t, zarg, need_dz=False)
            assert only is None and torch.equal(none, db)
            mine = dy_t.clone()
            dz2, db2 = Q.qlora_act_bwd(act, mine, zarg, need_dbias=False, dz=mine)
            assert dz2 is mine and db2 is None and torch.equal(bits(mine), bits(dz))


def test_activations_at_the_ends_of_the_range():
    """Zeros, denormals, huge values, infinities and NaN through every
    activation and slope, dense and from checkpoints."""
    vals = np.array([0.0, -0.0, 1e-45, -1e-45, 1e-20, -1e-20, 0.5, -0.5, 3, -3, 8, -8, 20, -20, 90, -90, 200, -200,
                     1e9, -1e9, 1e20, -1e20, 3e38, -3e38, np.inf, -np.inf, np.nan, 5, -5, 1, -1, 2], np.float32)
    z = np.tile(vals, (4, 1))
    dy = np.full(z.shape, 1.0, np.float32)
    for dtype in ("f32", "bf16"):
        z_t, zz = WL.as_compute_dtype(z, dtype)
        dy_t, _ = WL.as_compute_dtype(dy, dtype)
        for act in E.ACTS[1:]:
            say("range", dtype, act)
            dz, _ = Q.qlora_act_bwd(act, dy_t.cuda(), z_t.cuda())
            w = E.slope(act, zz)
            u = U16 if dtype == "bf16" else U32
            within(to_numpy(dz), w, u * np.abs(w) + SLOPE_ABS, f"{act} slope")
    # forward: a layer of zero weight and adapter, so z = bias
    K, N = 16, 32
    lin = Q.QLinear(K, N, 1, 1.0, "w8", torch.zeros((N, K), dtype=torch.int8, device="cuda"),
                    torch.zeros((N,), device="cuda"), torch.zeros((K, 1), device="cuda"),
                    torch.zeros((1, N), device="cuda"))
    x = torch.ones((3, K), device="cuda")
    for act in E.ACTS:
        for dt in (torch.float32, torch.bfloat16):
            say("range forward", act, dt)
            y, _, zc, _ = Q.qlora_fwd_epi(lin, x.to(dt), act=act, bias=dev(vals), save_z="full")
            w = np.tile(E.act(act, vals), (3, 1))
            tol = (U32 + ACT_REL) * np.abs(w) + (U16 * np.abs(w) if dt == torch.bfloat16 else 0) + 1e-30
            got = to_numpy(y)
            if dt == torch.bfloat16:   # 3e38 stays finite, 1e-45 may flush
                w = np.where(np.abs(w) < 1e-37, got, w)
            within(got, w, tol, f"{act} values")


@pytest.mark.parametrize("what", ["nan", "inf", "zero"])
@pytest.mark.parametrize("spec", [(70, 256, 272, 8, "w8", "bf16", 1), (2100, 2064, 144, 8, "w8", "bf16", 1),
                                  (130, 528, 2080, 4, "w8", "bf16", 1), (70, 64, 80, 4, "w8", "f32", 1),
                                  (1030, 1040, 528, 8, "w8", "bf16", 1), (4200, 528, 1040, 4, "w8", "bf16", 1),
                                  (1030, 528, 2080, 4, "w8", "bf16", 1)],
                         ids=lambda s: "-".join(map(str, s)) if isinstance(s, tuple) else s)
def test_non_finite_and_empty_rows(spec, what):
    """A row of x that is NaN, infinite or all zero: its checkpoint carries it,
    the other rows are as without it."""
    c = Case(*spec)
    x = c.x_t.clone()
    x[5] = {"nan": float("nan"), "inf": float("inf"), "zero": 0.0}[what]
    say("odd row", spec, what)
    y0 = Q.qlora_fwd_epi(c.lin, c.x_t, act="gelu", residual=c.res_t)[0]
    y, t, z, xc = Q.qlora_fwd_epi(c.lin, x, act="gelu", residual=c.res_t, save_z="c8g32", save_x=True)
    keep = torch.ones(c.M, dtype=torch.bool, device="cuda")
    keep[5] = False
    assert torch.equal(bits(y[keep]), bits(y0[keep])), "other rows"
    if what == "zero":
        assert torch.equal(y[5], c.res_t[5]) and not xc.codes[5].any() and float(xc.scales[5]) == 0
    else:
        assert torch.isnan(y[5]).all() and bool((z.scales[5] == 255).all()) and bool(torch.isnan(xc.scales[5]))
    dx, dA, dB = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, add=c.add_t)
    dx0 = Q.qlora_bwd_epi(c.lin, c.x_t, c.dy_t, t, add=c.add_t)[0]
    torch.cuda.synchronize()
    assert torch.equal(bits(dx), bits(dx0)), "dx does not depend on x"
    assert bool(torch.isnan(dA).all()) == (what != "zero") and bool(torch.isfinite(dA).all()) == (what == "zero")


def test_in_place_operands():
    """y over the residual, dx over add, on every output tile of a ragged
    layer, split and not."""
    for spec in ((333, 784, 272, 8, "w8", "bf16", 1), (100, 4096, 272, 8, "w8", "bf16", 1),
                 (130, 528, 2080, 4, "w8", "bf16", 1), (64, 256, 256, 4, "w8", "f32", 1),
                 (77, 256, 272, 8, "w4g128", "bf16", 1), (1030, 1040, 528, 8, "w8", "bf16", 1),
                 (4200, 528, 1040, 4, "w8", "bf16", 1), (1030, 528, 2080, 4, "w8", "bf16", 1),
                 (4, 784, 272, 8, "w8", "bf16", 1), (3, 256, 272, 8, "w4g128", "bf16", 1)):
        c = Case(*spec)
        say("in place", spec)
        y, t, _, xc = Q.qlora_fwd_epi(c.lin, c.x_t, act="silu", residual=c.res_t, save_x=True)
        r = c.res_t.clone()
        y2 = Q.qlora_fwd_epi(c.lin, c.x_t, act="silu", residual=r, y=r)[0]
        dx = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, act="silu", z=c.z_t, add=c.add_t)[0]
        a = c.add_t.clone()
        dx2 = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, act="silu", z=c.z_t, add=a, dx=a)[0]
        torch.cuda.synchronize()
        assert y2 is r and torch.equal(bits(y), bits(r)) and dx2 is a and torch.equal(bits(dx), bits(a))


def test_nothing_is_written_past_the_outputs():
    """Guard bytes around every output stay, at ragged sizes."""
    c = Case(37, 144, 272, 3)

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        size = torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n * size + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + n * size].view(dtype).view(shape)

    say("guards")
    bufs = {}
    for name, shape, dt in (("y", (37, 272), torch.bfloat16), ("t", (37, 3), torch.float32),
                            ("zc", (37, 272), torch.int8), ("zs", (37, 9), torch.uint8),
                            ("xq", (37, 144), torch.int8), ("sx", (37,), torch.float32),
                            ("dx", (37, 144), torch.bfloat16), ("dz", (37, 272), torch.bfloat16),
                            ("db", (272,), torch.float32), ("rd", (37, 272), torch.bfloat16),
                            ("dA", (144, 3), torch.float32), ("dB", (3, 272), torch.float32)):
        bufs[name] = guarded(shape, dt)
    v = {k: b[1] for k, b in bufs.items()}
    z = Q.Checkpoint(v["zc"], v["zs"], "c8g32")
    xc = Q.Checkpoint(v["xq"], v["sx"], "c8row")
    Q.qlora_fwd_epi(c.lin, c.x_t, act="gelu", y=v["y"], t=v["t"], save_z="c8g32", z=z, save_x=True, xc=xc)
    Q.qlora_ckpt_read(z, torch.bfloat16, out=v["rd"])
    Q.qlora_act_bwd("gelu", c.dy_t, z, dz=v["dz"], dbias=v["db"])
    Q.qlora_bwd_epi(c.lin, xc, c.dy_t, v["t"], act="silu", z=c.z_t, dx=v["dx"], dA=v["dA"], dB=v["dB"])
    Q.qlora_ckpt_write(c.dy_t, "c8g32", out=z)
    torch.cuda.synchronize()
    for name, (buf, view) in bufs.items():
        n = view.numel() * view.element_size()
        # (the last scales share their allocation's tail: bytes past the view)
        assert bool((buf[:256] == 0xAB).all()) and bool((buf[256 + n:] == 0xAB).all()), name


def _block(c1, c2, act, x, dout, b1, b2):
    """One residual feed-forward block, forward and backward, as it is trained:
    everything its backward needs kept in 8 bits. Returns its outputs."""
    h, t1, z1, x8 = Q.qlora_fwd_epi(c1.lin, x, act=act, bias=b1, save_z="c8g32", save_x=True)
    out, t2, _, h8 = Q.qlora_fwd_epi(c2.lin, h, bias=b2, residual=x, save_x=True)
    dz1, dA2, dB2 = Q.qlora_bwd_epi(c2.lin, h8, dout, t2, act=act, z=z1)
    _, db2 = Q.qlora_act_bwd("none", dout, need_dz=False)
    _, db1 = Q.qlora_act_bwd("none", dz1, need_dz=False)
    dx, dA1, dB1 = Q.qlora_bwd_epi(c1.lin, x8, dz1, t1, add=dout)
    h2, _ = Q.qlora_fwd_ckpt(c1.lin, x8, t1, x.dtype, act=act, bias=b1)
    return dict(out=out, dx=dx, dA1=dA1, dB1=dB1, dA2=dA2, dB2=dB2, db1=db1, db2=db2, h=h, h2=h2,
                t1=t1, t2=t2, z1c=z1.codes, z1s=z1.scales, h8c=h8.codes, h8s=h8.scales)


@pytest.mark.parametrize("fmt,dtype,M,D,H", [("w8", "bf16", 333, 256, 1040), ("w8", "f32", 65, 64, 144),
                                             ("w4g128", "bf16", 130, 256, 1024), ("w8o", "bf16", 130, 256, 1040),
                                             ("w8", "bf16", 130, 2048, 4096)])
def test_a_block_as_it_is_trained(fmt, dtype, M, D, H):
    """The operators in a row: each stage's inputs are the stage before's
    outputs as they came, so each is held to its own bound."""
    say("block", fmt, dtype, M, D, H)
    c1, c2 = Case(M, D, H, 8, fmt, dtype, seed=1), Case(M, H, D, 8, fmt, dtype, seed=2)
    b1, b2 = dev(c1.bias), dev(c2.bias)
    o = _block(c1, c2, "gelu", c1.x_t, c2.dy_t, b1, b2)
    torch.cuda.synchronize()
    (wh, wz, _), (th, tz, _) = c1.forward("gelu", True, False)
    within(to_numpy(o["h"]), wh, th, "h")
    z1 = Q.Checkpoint(o["z1c"], o["z1s"], "c8g32")
    check_group_ckpt(z1, wz, tz, "z1")
    if fmt != "w4g128":
        assert torch.equal(bits(o["h"]), bits(o["h2"])), "h again"
    c2.x, c2.res = to_numpy(o["h"]), c1.x                     # the stage's own inputs
    (wo, _, _), (to, _, _) = c2.forward("none", True, True)
    within(to_numpy(o["out"]), wo, to, "out")
    x64 = E.read_rows(o["h8c"].cpu().numpy(), o["h8s"].cpu().numpy())
    z64 = E.read_groups(o["z1c"].cpu().numpy(), o["z1s"].cpu().numpy())
    dz1, dA2, dB2 = Q.qlora_bwd_epi(c2.lin, Q.Checkpoint(o["h8c"], o["h8s"], "c8row"), c2.dy_t, o["t2"],
                                    act="gelu", z=z1)
    (wz1, wA, wB), (tz1, tA, tB) = c2.backward("gelu", z64, False, to_numpy(o["t2"]).astype(F64), x64)
    within(to_numpy(dz1), wz1, tz1, "dz1")
    within(to_numpy(o["dA2"]), wA, tA, "dA2")
    within(to_numpy(o["dB2"]), wB, tB, "dB2")
    dz = to_numpy(dz1)
    within(to_numpy(o["db1"]), dz.astype(F64).sum(0), M * U32 * np.abs(dz).sum(0) + 1e-30, "db1")
    within(to_numpy(o["db2"]), c2.dy.astype(F64).sum(0), M * U32 * np.abs(c2.dy).sum(0) + 1e-30, "db2")
    c1.dy, c1.add = dz, c2.dy
    oq, osx = O.quantize_rows(c1.x)
    (wx, wA, wB), (tx, tA, tB) = c1.backward("none", None, True, to_numpy(o["t1"]).astype(F64),
                                             E.read_rows(oq, osx))
    within(to_numpy(o["dx"]), wx, tx, "dx")
    within(to_numpy(o["dA1"]), wA, tA, "dA1")
    within(to_numpy(o["dB1"]), wB, tB, "dB1")


@pytest.mark.parametrize("fmt,dtype,M,D,H", [("w8", "bf16", 333, 256, 1040), ("w8", "f32", 65, 64, 144),
                                             ("w4g128", "bf16", 130, 256, 1024), ("w8o", "bf16", 130, 256, 1040),
                                             ("w8", "bf16", 1, 2048, 4096), ("w8", "bf16", 130, 2048, 4096),
                                             ("w8", "bf16", 1030, 528, 1040), ("w4g128", "bf16", 4, 256, 1024),
                                             ("w4g128", "bf16", 1030, 512, 1152)])
def test_block_captured_and_replayed(fmt, dtype, M, D, H):
    """The block in a HIP graph: replays between eager calls, on new inputs,
    give the eager bytes; so does a call on another stream."""
    say("graph", fmt, dtype, M, D, H)
    c1, c2 = Case(M, D, H, 8, fmt, dtype, seed=1), Case(M, H, D, 8, fmt, dtype, seed=2)
    b1, b2 = dev(c1.bias), dev(c2.bias)
    x, dout = c1.x_t.clone(), c2.dy_t.clone()
    args = (c1, c2, "gelu_tanh")
    sets = [(c1.x_t, c2.dy_t), (c1.x_t.flip(0).contiguous(), c2.dy_t.flip(1).contiguous())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _block(*args, x, dout, b1, b2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = _block(*args, x, dout, b1, b2)
    for it, k in enumerate([0, 1, 1, 0]):
        x.copy_(sets[k][0])
        dout.copy_(sets[k][1])
        g.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in o.items()}
        want = _block(*args, sets[k][0], sets[k][1], b1, b2)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(bits(got[n]), bits(want[n])), f"replay {it}: {n}"
        if it == 0:
            for n in want:
                assert torch.equal(bits(other[n]), bits(want[n])), f"other stream: {n}"


def test_two_streams_at_once():
    """The same layers used on two streams at a time, each with its own
    workspaces: the bytes of one call after the other."""
    for fmt, M, D, H in (("w8", 1030, 528, 1040), ("w8", 130, 2048, 4096), ("w4g128", 3, 512, 1152)):
        say("two streams", fmt, M, D, H)
        c1, c2 = Case(M, D, H, 8, fmt, seed=1), Case(M, H, D, 8, fmt, seed=2)
        b1, b2 = dev(c1.bias), dev(c2.bias)
        ins = [(c1.x_t, c2.dy_t), (c1.x_t.flip(0).contiguous(), c2.dy_t.flip(1).contiguous())]
        want = [_block(c1, c2, "silu", *i, b1, b2) for i in ins]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [[], []]
        for _ in range(8):
            for st, i, g in zip(streams, ins, got):
                with torch.cuda.stream(st):
                    g.append(_block(c1, c2, "silu", *i, b1, b2))
        torch.cuda.synchronize()
        for w, gs in zip(want, got):
            for g in gs:
                for n in w:
                    assert torch.equal(bits(w[n]), bits(g[n])), n


def test_refusals():
    """What the binding refuses before the library is called."""
    c = Case(8, 64, 80, 4)
    xc = Q.qlora_ckpt_write(c.x_t)
    z = Q.qlora_ckpt_write(c.z_t, "c8g32")
    _, t = Q.qlora_fwd(c.lin, c.x_t)
    bias = dev(c.bias)
    say("refusals")
    val, typ = pytest.raises(ValueError), pytest.raises(TypeError)
    for bad in (c.x_t[:, :48], c.x_t.t(), c.x_t[0], c.x_t.cpu(), torch.cat([c.x_t, c.x_t], 1)[:, ::2]):
        with val:
            Q.qlora_fwd_epi(c.lin, bad)
    # buffers for what is not asked for
    for kw in (dict(t=t, save_t=False), dict(xc=xc), dict(z=c.dy_t)):
        with val:
            Q.qlora_fwd_epi(c.lin, c.x_t, **kw)
    with val:
        Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, need_dx=False, dx=c.add_t.clone())
    for kw in (dict(need_dz=False, dz=c.dy_t.clone()), dict(need_dbias=False, dbias=bias.clone())):
        with val:
            Q.qlora_act_bwd("none", c.dy_t, **kw)
    with typ:
        Q.qlora_fwd_epi(c.lin, c.x_t.half())
    for kw in (dict(bias=bias[:64]), dict(bias=bias.cpu()), dict(residual=c.res_t[:4]), dict(act="tanh"),
               dict(save_z="c8row"), dict(save_x=True, xc=z), dict(y=torch.empty_like(c.x_t))):
        with val:
            Q.qlora_fwd_epi(c.lin, c.x_t, **kw)
    for kw in (dict(bias=bias.bfloat16()), dict(residual=c.res_t.float())):
        with typ:
            Q.qlora_fwd_epi(c.lin, c.x_t, **kw)
    with val:
        Q.qlora_fwd_ckpt(c.lin, z, t, torch.bfloat16)
    with val:
        Q.qlora_bwd_epi(c.lin, xc, c.dy_t)                        # t missing
    with val:
        Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, need_dx=False, add=c.add_t)
    with val:
        Q.qlora_bwd_epi(c.lin, z, c.dy_t, t)                      # x in groups
    for kw in (dict(act="gelu"), dict(z=z), dict(act="none", z=z)):
        with pytest.raises(Q.QloraError):
            Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, **kw)
    with pytest.raises(Q.QloraError):
        Q.qlora_act_bwd("gelu", c.dy_t)
    with pytest.raises(Q.QloraError):
        Q.qlora_act_bwd("none", c.dy_t, need_dz=False, need_dbias=False)
    with pytest.raises(Q.QloraError):
        Q.qlora_fwd_epi(c.lin, c.x_t[:0])                         # no rows
    with pytest.raises(Q.QloraError):                            # y over x's storage
        sq = Case(8, 64, 64, 4)
        Q.qlora_fwd_epi(sq.lin, sq.x_t, y=sq.x_t)
    with pytest.raises(Q.QloraError):
        Q.qlora_ckpt_write(torch.zeros((2, 24), device="cuda"))   # C % 16
    with val:
        Q.qlora_ckpt_write(c.x_t, "c4")
    torch.cuda.synchronize()
