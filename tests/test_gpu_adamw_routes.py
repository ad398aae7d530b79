"""What the AdamW step promises beside its formulas, by every way that it takes:
one launch for a few elements, two for more, two for each 64 tensors."""

from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import vocab_oracle as V
from quantized_frozen_weight_amd import binding as Q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24          # half a step of float32, relative

# one launch; two, by the elements and by the tensors; four, six
ROUTES = [(500, 33), (9000, 33), (40, 33, 7), (33, 100000), (70,) * 100, (9,) * 128 + (5000, 33)]
WAYS = pytest.mark.parametrize("sizes", ROUTES, ids=lambda s: f"{len(s)}x{max(s)}")
STATES = pytest.mark.parametrize("state", ["f32", "s8"])


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    Q.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().numpy()


def held(opt):
    """Every tensor that a step writes."""
    t = opt.params + opt.m + opt.v + [opt.step]
    return t + opt.m_scales + opt.v_scales if opt.state == "s8" else t


def tensors(sizes, seed):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(k).astype(np.float32) for k in sizes]


@STATES
@WAYS
def test_a_norm_that_is_not_finite_moves_nothing(sizes, state):
    say("not finite", len(sizes), max(sizes), state)
    opt = Q.AdamW([dev(a) for a in tensors(sizes, 1)], state=state, decay=0.01)
    good = [dev(a) for a in tensors(sizes, 2)]
    Q.qlora_adamw(opt, good, lr=1e-2, clip_norm=1.0)
    torch.cuda.synchronize()
    kept = [t.clone() for t in held(opt)]
    for odd in (float("nan"), float("inf"), float("-inf")):
        # in the first tensor's first element, the last one's last, and one between
        for i, e in ((0, 0), (len(sizes) - 1, sizes[-1] - 1), (len(sizes) // 2, sizes[len(sizes) // 2] // 2)):
            bad = [g.clone() for g in good]
            bad[i][e] = odd
            for need in (False, True):
                norm = Q.qlora_adamw(opt, bad, lr=1e-2, clip_norm=1.0, need_norm=need)
                torch.cuda.synchronize()
                assert norm is None or not np.isfinite(float(norm))
                assert all(torch.equal(a, b) for a, b in zip(held(opt), kept))
    # and the next step is the second
    want = Q.AdamW([t.clone() for t in kept[:len(sizes)]], state=state, decay=0.01, step=kept[3 * len(sizes)].clone(),
                   m=[t.clone() for t in kept[len(sizes):2 * len(sizes)]],
                   v=[t.clone() for t in kept[2 * len(sizes):3 * len(sizes)]],
                   **({} if state == "f32" else
                      dict(m_scales=[t.clone() for t in kept[3 * len(sizes) + 1:4 * len(sizes) + 1]],
                           v_scales=[t.clone() for t in kept[4 * len(sizes) + 1:]])))
    for o in (opt, want):
        Q.qlora_adamw(o, good, lr=1e-2, clip_norm=1.0)
    torch.cuda.synchronize()
    assert int(opt.step) == 2 and all(torch.equal(a, b) for a, b in zip(held(opt), held(want)))


@STATES
@WAYS
def test_without_clipping_only_the_odd_element_is_none(sizes, state):
    say("odd element", len(sizes), max(sizes), state)
    last, e = len(sizes) - 1, sizes[-1] - 1
    for odd in (np.nan, np.inf):
        opt = Q.AdamW([dev(a) for a in tensors(sizes, 1)], state=state)
        g = tensors(sizes, 2)
        g[last][e] = odd
        norm = Q.qlora_adamw(opt, [dev(a) for a in g], lr=1e-2, need_norm=True)
        torch.cuda.synchronize()
        assert not np.isfinite(float(norm)) and int(opt.step) == 1
        for i, p in enumerate(opt.params):
            b = np.isnan(host(p))
            assert b.sum() == (i == last) and (i != last or b[e])
        if state == "s8":
            b = host(opt.m_scales[last]) == 255
            assert b.sum() == 1 and b[e // 32]


@WAYS
def test_gradients_whose_squares_pass_float32(sizes):
    say("large gradients", len(sizes), max(sizes))
    n = sum(sizes)
    opt = Q.AdamW([torch.zeros(k, device="cuda") for k in sizes])
    norm = Q.qlora_adamw(opt, [torch.full((k,), 1e30, device="cuda") for k in sizes], lr=1e-2, clip_norm=float(n) ** 0.5,
                         need_norm=True)
    torch.cuda.synchronize()
    want = float(np.float32(1e30)) * float(n) ** 0.5
    assert abs(float(norm) - want) <= 2 * U32 * want
    # clipped to 1 each: the first step is lr down, over 1 + eps = 1 + 1e-6, and a few roundings
    for p in opt.params:
        assert np.abs(host(p) / -1e-2 - 1).max() <= 1e-6 + 16 * U32


@STATES
@WAYS
def test_captured_steps_count_on(sizes, state):
    """Replays of one captured step, its rate on the device, against eager steps."""
    say("captured", len(sizes), max(sizes), state)
    p, g = tensors(sizes, 3), [dev(a) for a in tensors(sizes, 4)]
    make = lambda: Q.AdamW([dev(a) for a in p], state=state, decay=0.01, seed=5)  # noqa: E731
    eager, opt = make(), make()
    rate = torch.full((1,), 1e-2, device="cuda")
    start = [t.clone() for t in held(opt)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Q.qlora_adamw(opt, g, lr=rate, clip_norm=1.0, need_norm=True)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = Q.qlora_adamw(opt, g, lr=rate, clip_norm=1.0, need_norm=True)
    for t, k in zip(held(opt), start):
        t.copy_(k)
    step = 0
    for k in range(1, 7):
        lr = 1e-2 / k
        rate.fill_(lr)
        odd = k == 4                                      # a norm that is none, between the others
        was = g[-1][0].clone()
        if odd:
            g[-1][0] = float("inf")
        graph.replay()
        torch.cuda.synchronize()
        n = Q.qlora_adamw(eager, g, lr=float(np.float32(lr)), clip_norm=1.0, need_norm=True)
        torch.cuda.synchronize()
        step += not odd
        assert int(opt.step) == int(eager.step) == step
        assert torch.equal(norm, n)
        assert all(torch.equal(a, b) for a, b in zip(held(opt), held(eager)))
        g[-1][0] = was


@STATES
def test_8_bit_and_float32_moments_follow_a_steady_gradient(state):
    """As many steps as it takes the second moment to move, by two launches: it
    arrives where it belongs (8 bits: on average)."""
    n = 4096
    opt = Q.AdamW([torch.zeros(n, device="cuda") for _ in range(3)], state=state, seed=3)
    g = [torch.full((n,), 0.5, device="cuda") for _ in range(3)]
    for t in g:
        t[::32] = 1.0                                     # each group's scale
    say("steady gradient", state)
    steps = 2000
    for _ in range(steps):
        Q.qlora_adamw(opt, g, lr=0.0)
    want = 0.5 * np.sqrt(1 - 0.999 ** steps)
    for i in range(3):
        if state == "s8":
            root = host(Q.qlora_moment_read(opt.v[i], opt.v_scales[i], "root_v"))
            m = host(Q.qlora_moment_read(opt.m[i], opt.m_scales[i], "m"))
        else:
            root, m = np.sqrt(host(opt.v[i])), host(opt.m[i])
        root, m = root.reshape(-1, 32)[:, 1:], m.reshape(-1, 32)[:, 1:]
        # 8 bits: an element's spread is under 0.15 of v, as a step's drift of at most 0.001
        # of it on a grid of 1/32 leaves it, a mean of 3968 of them under 0.003; float32:
        # at most three roundings a step, of which those of the last 1000 count
        tol = 0.03 if state == "s8" else 3 * 1000 * 2 * U32
        assert abs(root.mean() / want - 1) < tol and abs(m.mean() / 0.5 - 1) < tol


@STATES
def test_many_tensors_against_the_oracle(state):
    """More sums of the norm than 512, over several launches: a step of each."""
    sizes = [37] * 700
    say("many tensors", state)
    p, g = tensors(sizes, 6), tensors(sizes, 7)
    opt = Q.AdamW([dev(a) for a in p], state=state, decay=0.01, seed=11)
    norm = Q.qlora_adamw(opt, [dev(a) for a in g], lr=3e-3, clip_norm=0.5, need_norm=True)
    torch.cuda.synchronize()
    want = V.norm_of(g)
    assert abs(float(norm) - want) <= 2 * U32 * want
    n = np.float32(norm.item())
    coef = np.float32(0.5) / max(n, np.float32(0.5))
    for i in range(len(sizes)):
        z = np.zeros(sizes[i], np.float32)
        w, m, v, _ = V.adamw(p[i], g[i], z, z, 1, 3e-3, 0.9, 0.999, 1e-6, 0.01, coef)
        assert np.array_equal(host(opt.params[i]), w), i
        if state == "f32":
            assert np.array_equal(host(opt.m[i]), m) and np.array_equal(host(opt.v[i]), v), i
