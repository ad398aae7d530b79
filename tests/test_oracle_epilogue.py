"""Pins of the epilogue oracle: closed values, differences, and the group
form's defining properties."""

import numpy as np
import pytest

from oracle import epilogue_oracle as E


def test_activation_values():
    assert E.act("gelu", 1.0) == pytest.approx(0.8413447460685429, rel=1e-14)       # Phi(1)
    assert E.act("silu", 1.0) == pytest.approx(1 / (1 + np.exp(-1.0)), rel=1e-14)
    h = np.tanh(np.sqrt(2 / np.pi) * 1.044715)
    assert E.act("gelu_tanh", 1.0) == pytest.approx(0.5 * (1 + h), rel=1e-14)
    assert list(E.act("relu", [-1.0, 0.0, 2.0])) == [0.0, 0.0, 2.0]
    for name in E.ACTS[1:]:
        v = E.act(name, [-np.inf, np.inf, np.nan, 0.0])
        assert v[0] == 0 and v[1] == np.inf and np.isnan(v[2]) and v[3] == 0
        s = E.slope(name, [-np.inf, np.inf, np.nan])
        assert abs(s[0]) < 1e-30 and s[1] == 1 and np.isnan(s[2])


@pytest.mark.parametrize("name", E.ACTS)
def test_slopes_against_differences(name):
    z = np.concatenate([np.linspace(-9, 9, 400), [0.3, -0.7]])    # (no 0: relu has a corner there)
    h = 1e-5
    d = (E.act(name, z + h) - E.act(name, z - h)) / (2 * h)
    # central difference: h^2 / 6 |f'''| (below 4 for each) and rounding 9 2^-52 / h
    assert np.abs(d - E.slope(name, z)).max() < h * h + 9 * 2.0 ** -52 / h * 2
    assert E.slope("relu", 0.0) == 0


def test_group_form():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((7, 80)) * 10.0 ** rng.integers(-30, 30, (7, 1))).astype(np.float32)
    v[0, :32] = 0
    v[1, 3] = 1e-38 * v[1, 4]                     # tiny beside its group: keeps its sign
    q, b = E.write_groups(v)
    r = E.read_groups(q, b)
    assert q.shape == (7, 80) and b.shape == (7, 3) and b[0, 0] == 1
    step = np.repeat(2.0 ** (b.astype(float) - 127), 32, 1)[:, :80]
    small = np.abs(q) == 1
    assert np.all(np.abs(r - v) <= np.where(small, 1.0, 0.5) * step)
    assert np.array_equal(np.sign(r), np.sign(v))
    # the scale is the smallest that holds the group
    g = np.abs(np.pad(v.astype(float), ((0, 0), (0, 16)))).reshape(7, 3, 32).max(2)
    e = b.astype(int) - 127
    assert np.all(g <= 127 * 2.0 ** e) and np.all((g > 127 * 2.0 ** (e - 1.0)) | (e == -126))
    # reading is exact in bfloat16: 7 bits
    assert np.array_equal(r, (r.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32))


def test_group_form_of_non_finite_and_extreme_values():
    v = np.zeros((5, 32), np.float32)
    v[0, 5] = np.inf
    v[1, 5] = np.nan
    v[2, 5] = 3.4e38
    v[3, 5] = 1e-45                                # the smallest denormal
    v[4, :] = 127.0
    q, b = E.write_groups(v)
    assert list(b[:, 0]) == [255, 255, 249, 1, 127]
    assert not q[:2].any() and q[2, 5] == 64 and q[3, 5] == 1 and np.all(q[4] == 127)
    assert np.isnan(E.read_groups(q, b)[:2]).all()
