"""Host-side checks of the epilogue calls' size limits and workspaces (no GPU
needed, nothing is launched)."""

from __future__ import annotations

import ctypes

import pytest

from quantized_frozen_weight_amd import binding as Q
from tests.test_abi_epilogue_host import BF, EUNSUP, EWS, F32, OK, epi, fwd, layer, refwd


@pytest.fixture(scope="module")
def lib():
    return Q.lib()


@pytest.mark.parametrize("fmt,dt", [(Q.QLORA_W8, BF), (Q.QLORA_W8, F32), (Q.QLORA_W8O, BF)])
def test_contractions_whose_code_sums_could_overflow_are_refused(lib, fmt, dt):
    """127 * 128 K < 2^31 (int32 products) and 127 K < 2^24 (float32 sums of
    codes) up to K = 132096, the multiple of 16; not past it."""
    last = 132096
    assert 127 * 128 * last < 2 ** 31 and 127 * last < 2 ** 24 <= 127 * (last + 16)
    for call in (fwd, refwd):
        assert call(lib, L=layer(fmt, K=last, N=16), m=1, dt=dt, e=epi(), n=16) == EWS    # accepted so far
        for k in (last + 16, 1 << 20):
            assert call(lib, L=layer(fmt, K=k, N=16), m=1, dt=dt, e=epi(), n=16) == EUNSUP
    n = ctypes.c_size_t()
    # the plain forward takes what it took
    assert lib.qlora_fwd_workspace(ctypes.byref(layer(fmt, K=last + 16, N=16)), 1, dt, ctypes.byref(n)) == OK


@pytest.mark.parametrize("fmt", [Q.QLORA_W8, Q.QLORA_W8O, Q.QLORA_W4G128])
@pytest.mark.parametrize("m", [1, 4, 5])
def test_forward_workspace_of_few_rows_is_that_of_the_plain_forward(lib, m, fmt):
    """Codes, scales, t and (affine) the rows' code sums, each to 256 bytes; no
    split of so wide an output, and nothing for the few-row kernel."""
    k, n_out, r = 4096, 25600, 8
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    n = ctypes.c_size_t()
    assert lib.qlora_fwd_workspace(ctypes.byref(layer(fmt, K=k, N=n_out, r=r)), m, BF, ctypes.byref(n)) == OK
    assert n.value == up(m * k) + up(4 * m) + up(4 * m * r) + (up(4 * m) if fmt == Q.QLORA_W8O else 0)
