"""Corners of the epilogue and checkpoint calls on the GPU: values far apart in
one group, the ends of the float range, odd rows among few, the largest sizes."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import epilogue_oracle as E
from oracle import qlora_oracle as O
from quantized_frozen_weight_amd import binding as Q
from quantized_frozen_weight_amd import workloads as WL
from tests.helpers import to_numpy
from tests.test_gpu_epilogue import Case, bits, check_group_ckpt, dev, say, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F64 = np.float64
TD = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    Q.lib()


def zero_layer(K, N, fmt):
    """A layer whose product and adapter are zero, so that z is the bias."""
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    if fmt == "w4g128":
        codes, scales = z(N, K // 2, dtype=torch.uint8), z(N, K // 128, dtype=torch.float16)
    elif fmt == "w8o":
        codes, scales = Q.qlora_quantize(z(K, N), "w8o")
    else:
        codes, scales = z(N, K, dtype=torch.int8), z(N)
    return Q.QLinear(K, N, 4, 8.0, fmt, codes, scales, z(K, 4), z(4, N))


# pairs (abs-max of a group, a value in it) whose ratio takes the value under
# the smallest float once the group's scale is divided out
FAR = [(1e30, 1e-20), (1e30, -1e-20), (1e20, -1e-30), (1e10, 1e-38), (3e38, -1e-9), (1e3, 1e-45), (-1e3, -1e-45),
       (2.0, 1e-39)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_codes_keep_the_sign_of_values_far_below_their_group(dtype):
    x = np.zeros((len(FAR), 80), np.float32)
    for i, (top, v) in enumerate(FAR):
        x[i, 5], x[i, 6:30], x[i, 40], x[i, 79] = top, v, v, v
    x_t, x = WL.as_compute_dtype(x, dtype)
    say("far below the group", dtype)
    c = Q.qlora_ckpt_write(x_t.cuda(), "c8g32")
    dz, _ = Q.qlora_act_bwd("relu", torch.ones_like(x_t).cuda(), c, need_dbias=False)
    torch.cuda.synchronize()
    q, b = E.write_groups(x)
    assert np.array_equal(c.scales.cpu().numpy(), b)
    assert np.array_equal(c.codes.cpu().numpy(), q)
    assert np.array_equal(np.sign(q), np.sign(x))
    assert np.array_equal(to_numpy(dz), (x > 0).astype(np.float32))


@pytest.mark.parametrize("M,K,N,fmt,dtype", [
    (1, 64, 272, "w8", "f32"), (3, 64, 272, "w8", "bf16"), (2, 16384, 144, "w8", "bf16"),   # few rows
    (4, 256, 272, "w4g128", "bf16"), (70, 64, 272, "w8", "f32"), (70, 64, 272, "w8", "bf16"),
    (100, 4096, 272, "w8", "bf16"), (70, 256, 272, "w4g128", "bf16"), (90, 8192, 144, "w4g128", "bf16"),
    (70, 256, 272, "w8o", "bf16"), (130, 4096, 80, "w8o", "bf16")])
def test_saved_z_keeps_the_sign_of_values_far_below_their_group(M, K, N, fmt, dtype):
    z = np.zeros(N, np.float32)
    for i in range(N // 16):
        top, v = FAR[i % len(FAR)]
        z[16 * i + 3], z[16 * i + 4: 16 * i + 9] = top, v
    lin = zero_layer(K, N, fmt)
    x = torch.ones((M, K), device="cuda", dtype=TD[dtype])
    say("saved z far below the group", M, K, N, fmt, dtype)
    _, t, c, xc = Q.qlora_fwd_epi(lin, x, bias=dev(z), save_z="c8g32", save_x=True)
    c2 = Q.qlora_fwd_ckpt(lin, xc, t, x.dtype, bias=dev(z), save_z="c8g32")[1]
    torch.cuda.synchronize()
    q, b = E.write_groups(np.tile(z, (M, 1)))
    for got in (c, c2):
        assert np.array_equal(got.scales.cpu().numpy(), b)
        assert np.array_equal(got.codes.cpu().numpy(), q)


@pytest.mark.parametrize("fmt", ["c8row", "c8g32"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_checkpoints_of_the_largest_finite_values_read_back_finite(dtype, fmt):
    top = np.float32(np.finfo(np.float32).max) if dtype == "f32" else np.float32(2.0 ** 128 - 2.0 ** 120)
    x = np.zeros((7, 48), np.float32)
    x[0, 3], x[1, 40], x[2, :] = top, -top, top
    x[3, 0], x[4, 1] = np.float32(3.4e38) if dtype == "f32" else top, 127 / 64 * 2.0 ** 127
    x[5, 7], x[6, 9] = np.inf, np.nan
    x_t, x = WL.as_compute_dtype(x, dtype)
    say("largest values", dtype, fmt)
    c = Q.qlora_ckpt_write(x_t.cuda(), fmt)
    got = {d: to_numpy(Q.qlora_ckpt_read(c, TD[d])) for d in TD}      # in its own dtype and the other
    if fmt == "c8row":
        want = E.read_rows(*O.quantize_rows(x))
    else:
        want = E.read_groups(*E.write_groups(x))
    for d, g in got.items():
        lim = np.finfo(np.float32).max if d == "f32" else 2.0 ** 128 - 2.0 ** 120
        with np.errstate(over="ignore"):
            w = np.clip(O.round_to(want, d).astype(F64), -lim, lim)
        assert np.array_equal(g.astype(F64), w, equal_nan=True), d
        assert np.isfinite(g[:5]).all() and np.array_equal(np.sign(g[:5]), np.sign(x[:5]))


@pytest.mark.parametrize("M,K,N,r", [(1, 256, 272, 4), (3, 4096, 144, 8), (4, 4096, 528, 16), (2, 16384, 80, 1)])
def test_few_4bit_rows_with_huge_inputs(M, K, N, r):
    """Inputs up to the largest finite one, whose products with the weight stay
    finite, give finite outputs within the bounds of any other input; the other
    rows are the bytes they are without them."""
    c = Case(M, K, N, r, "w4g128")
    y0 = Q.qlora_fwd_epi(c.lin, c.x_t)[0]
    for big in (2.0 ** 114, -2.0 ** 126, 2.0 ** 127 * 1.98):
        say("huge few rows", M, K, N, r, big)
        x = c.x.copy()
        x[M - 1, 5::131] = big
        x[M - 1, 7::509] = -big
        c2 = Case(M, K, N, r, "w4g128")
        c2.x_t, c2.x = WL.as_compute_dtype(x, "bf16")
        W = c2.W
        # (finite: every output, and every sum of absolute products on the way)
        low = c2.s * (np.abs(c2.x.astype(F64)) @ np.abs(c2.A64)) @ np.abs(c2.B64)
        scale = (np.abs(c2.x.astype(F64)) @ np.abs(W) + low).max() / 2.0 ** 126
        if scale > 1:
            c2.x_t, c2.x = WL.as_compute_dtype(x * np.float32(2.0 ** -np.ceil(np.log2(scale))), "bf16")
        y, t, _, _ = Q.qlora_fwd_epi(c2.lin, c2.x_t.cuda())
        torch.cuda.synchronize()
        (wy, _, wt), (ty, _, tt) = c2.forward("none", False, False)
        assert np.isfinite(to_numpy(y)).all()
        within(to_numpy(y), wy, ty, "y")
        within(to_numpy(t), wt, tt, "t")
        if scale <= 1 and M > 1:
            assert torch.equal(bits(y[:M - 1]), bits(y0[:M - 1]))


@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("M,K,N,r", [(1, 256, 272, 4), (3, 4096, 144, 8), (4, 16384, 80, 16),
                                     (1, 256, 272, 1), (2, 16384, 80, 3), (4, 384, 80, 11)])
def test_few_4bit_rows_that_are_not_finite(M, K, N, r, what):
    """NaN and infinities sit where the tiled product and the oracle have
    them, and touch no other row."""
    c = Case(M, K, N, r, "w4g128")
    # one sign in the adapter: its term is an infinity then, and no NaN
    c.A64, c.B64 = np.abs(c.A64), np.abs(c.B64)
    c.lin.A, c.lin.B = c.lin.A.abs(), c.lin.B.abs()
    x = c.x_t.clone()
    x[M - 1, 9] = what
    say("few rows not finite", M, K, N, r, what)
    y0, y = (Q.qlora_fwd_epi(c.lin, v)[0] for v in (c.x_t, x))
    tiled = Q.qlora_fwd(c.lin, x)[0]
    torch.cuda.synchronize()
    assert torch.equal(bits(y[:M - 1]), bits(y0[:M - 1]))
    x64 = to_numpy(x).astype(F64)
    with np.errstate(invalid="ignore"):
        want = x64 @ c.W + c.s * ((x64 @ c.A64) @ c.B64)
    for name, g in (("few", to_numpy(y)), ("tiled", to_numpy(tiled))):
        for f in (np.isnan, np.isposinf, np.isneginf):
            assert (f(g) != f(want)).sum() == 0, (name, f.__name__)


@pytest.mark.parametrize("M", [1, 70])
def test_float32_gelu_tail_to_a_millionth(M):
    """Float32 GELU and its slope down to the smallest normal results. y for z
    < 0 is -|z| Phi(-|z|): 1e-6 of the tail (the polynomial's 6e-7 with its own
    roundings, and one step of 2^-23 each for the exponential and the
    reciprocal) and the output's rounding. The slope is Phi + z phi: 1e-6 of
    the first; the exponential's 4e-7 and three roundings of the second; and
    the output's."""
    N = 16384
    z = np.concatenate([-np.linspace(0, 12.6, N - 4096), np.geomspace(1e-6, 12, 4096)]).astype(np.float32)
    lin = zero_layer(16, N, "w8")
    say("gelu tail", M)
    y = Q.qlora_fwd_epi(lin, torch.ones((M, 16), device="cuda"), act="gelu", bias=dev(z))[0]
    zt = dev(np.tile(z, (M, 1)))
    dz, _ = Q.qlora_act_bwd("gelu", torch.ones_like(zt), zt)
    torch.cuda.synchronize()
    u = 2.0 ** -24
    z64 = z.astype(F64)
    w = E.act("gelu", z64)
    tail = np.abs(z64) * E.act("gelu", -np.abs(z64)) / np.minimum(-np.abs(z64), -1e-300)   # |z| Phi(-|z|)
    within(to_numpy(y), np.tile(w, (M, 1)), np.tile(1e-6 * tail + u * np.abs(w) + 2.0 ** -149, (M, 1)), "gelu")
    phi = np.exp(-0.5 * z64 * z64) / np.sqrt(2 * np.pi)
    sl = E.slope("gelu", z64)
    cdf = tail / np.maximum(np.abs(z64), 1e-300)
    tol = 1e-6 * cdf + (4e-7 + 3 * u) * np.abs(z64) * phi + 2 * u * np.abs(sl) + 2.0 ** -149
    within(to_numpy(dz), np.tile(sl, (M, 1)), np.tile(tol, (M, 1)), "gelu slope")


@pytest.mark.parametrize("C", [2 ** 29 + 16, 2 ** 30, 2 ** 31 - 16])
def test_activation_backward_of_the_longest_rows(C):
    """One row up to the longest that the calls take: more threads than a
    launch has at 32 row lanes a block."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dy = torch.empty((1, C), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    say("longest rows", C)
    dz, db = Q.qlora_act_bwd("relu", dy, dy)
    torch.cuda.synchronize()
    want = dy.clamp_min(0)
    assert torch.equal(dz, want)
    assert torch.equal(db, want[0].float())
    del dz, db, want
    torch.cuda.empty_cache()


def test_affine_forward_from_a_checkpoint_of_many_rows():
    """More rows than the code sums have waves: the bytes of the forward that
    wrote the checkpoint, whose row pass sums the codes on the way."""
    c = Case(300001, 32, 16, 1, "w8o")
    say("many affine rows")
    y, t, _, xc = Q.qlora_fwd_epi(c.lin, c.x_t, save_x=True)
    y2, _ = Q.qlora_fwd_ckpt(c.lin, xc, t, torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(y2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", [(1, 16), (130, 1040), (5, 16384), (600, 4112), (3, 40016)])
def test_row_quantizer_and_row_checkpoint_are_one(M, C, dtype):
    rng = np.random.default_rng(M + C)
    x = rng.standard_normal((M, C)).astype(np.float32)
    if M > 2:
        x[0], x[1, 5], x[2, 7] = 0, np.inf, np.nan
    x_t = WL.as_compute_dtype(x, dtype)[0].cuda()
    say("rows", M, C, dtype)
    xq, sx = Q.qlora_quantize_rows(x_t)
    c = Q.qlora_ckpt_write(x_t)
    torch.cuda.synchronize()
    assert torch.equal(xq, c.codes)
    assert torch.equal(bits(sx), bits(c.scales))


@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "zero"])
@pytest.mark.parametrize("spec", [
    (2, 64, 80, 3, "w8", "f32"), (4, 784, 272, 8, "w8", "bf16"),             # few rows, t in the same launch
    (2, 8192, 144, 8, "w8", "f32"), (3, 16384, 80, 4, "w8", "bf16"),         # ... t by the launch before
    (4, 256, 272, 8, "w4g128", "bf16"), (3, 16384, 144, 16, "w4g128", "bf16"),
    (4, 256, 144, 32, "w8", "bf16"), (3, 256, 144, 8, "w8o", "bf16"),        # few rows, tiled product
    (70, 256, 272, 8, "w4g128", "bf16"), (90, 8192, 144, 4, "w4g128", "bf16"),
    (100, 256, 384, 8, "w8o", "bf16"), (130, 4096, 80, 4, "w8o", "bf16")],
    ids=lambda s: "-".join(map(str, s)) if isinstance(s, tuple) else s)
def test_odd_rows_of_every_format(spec, what):
    """A row of x with a NaN or an infinity, or all zero: its checkpoints carry
    it, its outputs show it, and every other row is the bytes it is without."""
    c = Case(*spec)
    row = c.M - 1
    x = c.x_t.clone()
    if what == "zero":
        x[row] = 0
    else:
        x[row, 7] = float(what)
    say("odd row", spec, what)
    kw = dict(act="gelu", residual=c.res_t, save_z="c8g32", save_x=True)
    y0, t0, z0, xc0 = Q.qlora_fwd_epi(c.lin, c.x_t, **kw)
    y, t, z, xc = Q.qlora_fwd_epi(c.lin, x, **kw)
    y2, z2 = Q.qlora_fwd_ckpt(c.lin, xc, t, c.td, act="gelu", residual=c.res_t, save_z="c8g32")
    torch.cuda.synchronize()
    keep = torch.arange(c.M, device="cuda") != row
    for a, b in ((y, y0), (t, t0), (z.codes, z0.codes), (z.scales, z0.scales), (xc.codes, xc0.codes),
                 (xc.scales, xc0.scales)):
        assert torch.equal(bits(a[keep]), bits(b[keep])), "other rows"
    assert not xc.codes[row].any()
    if what == "zero":
        assert float(xc.scales[row]) == 0 and not t[row].any()
        for yy, zz in ((y, z), (y2, z2)):
            assert torch.equal(yy[row], c.res_t[row])
            assert not zz.codes[row].any() and bool((zz.scales[row] == 1).all())
    else:
        assert bool(torch.isnan(xc.scales[row])) and not torch.isfinite(t[row]).any()
        for yy, zz in ((y, z), (y2, z2)):
            assert not zz.codes[row].any() and bool((zz.scales[row] == 255).all())
        assert torch.isnan(y2[row]).all()                    # from a NaN row scale
        if c.fmt != "w4g128" or what == "nan":               # (4-bit: x itself, gelu(-inf) = 0)
            assert torch.isnan(y[row]).all()
    dx, dA, dB = Q.qlora_bwd_epi(c.lin, xc, c.dy_t, t, act="silu", z=c.z_t, add=c.add_t)
    dx0 = Q.qlora_bwd_epi(c.lin, xc0, c.dy_t, t, act="silu", z=c.z_t, add=c.add_t)[0]
    torch.cuda.synchronize()
    assert torch.equal(bits(dx), bits(dx0)), "dx does not depend on x"
    assert bool(torch.isnan(dA).all()) == (what != "zero") and bool(torch.isfinite(dA).all()) == (what == "zero")
    assert bool(torch.isfinite(dB).all()) == (what == "zero")


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations_at_the_ends_of_the_range_absolutely(M, dtype):
    """Every value of the forward activations held to a bound of its own. A
    sigma below 2^-126 may be 0 (the reciprocal instruction flushes denormal
    results): z sigma(w) is then at most 87.4 2^-126 = 1.03e-36 in size, since
    |z| e^-|z| falls past 1 and e^-87.34 = 2^-126 (silu; tanh gelu reaches that
    sigma at a smaller |z|). Elsewhere float32 values within 2e-5 (w rounded
    three times, times |w| < 89), and half a step of the output."""
    vals = np.array([0.0, -0.0, 1e-45, -1e-45, 1e-39, -1e-39, 1e-20, -1e-20, 0.5, -0.5, 3, -3, 8, -8, 12, -12, 20, -20,
                     88, -88, 90, -90, 200, -200, 1e9, -1e9, 1e20, -1e20, 3e38, -3e38, np.inf, -np.inf], np.float32)
    lin = zero_layer(16, 32, "w8")
    x = torch.ones((M, 16), device="cuda", dtype=TD[dtype])
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for act in E.ACTS:
        say("range", M, dtype, act)
        y = Q.qlora_fwd_epi(lin, x, act=act, bias=dev(vals))[0]
        torch.cuda.synchronize()
        w = np.tile(E.act(act, vals), (M, 1))
        with np.errstate(invalid="ignore"):
            tol = (u + (2e-5 if act != "none" else 0)) * np.abs(w) + 1.04e-36
            within(to_numpy(y), w, tol, act)


@pytest.mark.parametrize("spec", [
    (1, 256, 4096, 3, "w8", "bf16"), (4, 272, 4112, 8, "w8", "f32"),          # 16 and 32 columns a block
    (2, 784, 8192, 4, "w8", "bf16"), (3, 784, 8208, 16, "w8", "bf16"),        # 32 and 64
    (4, 256, 12304, 8, "w4g128", "bf16"), (1, 4096, 16400, 8, "w8", "bf16"),  # 64, and a second round
    (4, 4096, 16400, 11, "w8", "bf16"), (3, 128, 16400, 16, "w4g128", "bf16"),
    (2, 256, 16400, 4, "w8", "f32"), (4, 64, 32768, 8, "w8", "bf16")],        # int8 past 16384 outputs: tiles
    ids=lambda s: "-".join(map(str, s)))
def test_few_rows_at_every_block_width(spec):
    c = Case(*spec)
    for act, save_z in (("gelu", "c8g32"), ("silu", "full")):
        say("few rows", spec, act, save_z)
        y, t, z, xc = Q.qlora_fwd_epi(c.lin, c.x_t, act=act, bias=dev(c.bias), residual=c.res_t, save_z=save_z,
                                      save_x=True)
        torch.cuda.synchronize()
        (wy, wz, wt), (ty, tz, tt) = c.forward(act, True, True)
        within(to_numpy(t), wt, tt, "t")
        within(to_numpy(y), wy, ty, "y")
        if save_z == "full":
            within(to_numpy(z), wz, c.u * (np.abs(wz) + tz) + tz, "z")
        else:
            check_group_ckpt(z, wz, tz, "z")
        oq, osx = O.quantize_rows(c.x)
        assert np.array_equal(xc.codes.cpu().numpy(), oq)
        assert np.array_equal(xc.scales.cpu().numpy().view(np.uint32), osx.view(np.uint32))


@pytest.mark.parametrize("M,K,N,r", [(1, 256, 272, 4), (3, 4096, 144, 8), (4, 1024, 528, 16), (2, 16384, 80, 4)])
def test_few_4bit_rows_with_an_outlier_on_zero_weights(M, K, N, r):
    """An input far above the others that meets only zero codes (and zeros of
    A) leaves the sums of the others to float32 accuracy."""
    rng = np.random.default_rng(K + N)
    c = Case(M, K, N, r, "w4g128")
    W = (0.05 * rng.standard_normal((K, N))).astype(np.float32)
    at = [7, 130, K - 1]
    W[at] = 0
    c.A[at] = 0
    c.A64 = c.A.astype(F64)
    packed, sc = O.quantize_w4(W)
    c.W = O.dequant_w4(packed, sc)
    c.Wabs = np.abs(c.W)
    codes, scales = Q.qlora_quantize(dev(W), "w4g128")
    c.lin = Q.QLinear(K, N, r, 16.0, "w4g128", codes, scales, dev(c.A), dev(c.B))
    for big in (1e4, -1e6, 1e9, 1e30):
        say("outlier on zeros", M, K, N, r, big)
        x = c.x.copy()
        x[:, at] = big
        x_t, c.x = WL.as_compute_dtype(x, "bf16")
        y, t, _, _ = Q.qlora_fwd_epi(c.lin, x_t.cuda())
        torch.cuda.synchronize()
        (wy, _, wt), (ty, _, tt) = c.forward("none", False, False)
        within(to_numpy(t), wt, tt, "t")
        within(to_numpy(y), wy, ty, "y")
