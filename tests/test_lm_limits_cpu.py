"""The limits that the language-model calls state, from both sides, without a
GPU: a call of valid sizes and values gets as far as its misaligned pointer,
one past a limit is refused for its shape or value."""
from __future__ import annotations

import os

import pytest

import sample_gradient_clipping_layer_amd as dpc

FAKE = 0x100000  # aligned, never dereferenced
SHAPE, ALIGN, VALUE = dpc.DP_ERR_SHAPE, dpc.DP_ERR_ALIGN, dpc.DP_ERR_VALUE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dpc.LIB_PATH):
        pytest.fail("libdpclip.so is not built (run __graft_entry__.build())")
    return dpc.lib()


def _matmul(lib, dt, R, E, B, d, p, transpose=0):
    return lib.dp_grouped_matmul(None, FAKE + 8, FAKE, dt, FAKE, R, E, B, d, p, transpose, None, 0, FAKE)


def _norm(lib, dt, R, E, B, d, p):
    return lib.dp_grouped_norm(None, FAKE + 8, FAKE, dt, FAKE, R, E, B, d, p, None, 0, FAKE, 0)


def _sum(lib, dt, R, E, B, d, p):
    return lib.dp_grouped_clipped_sum_noise(None, FAKE + 8, FAKE, dt, FAKE, R, E, B, d, p, FAKE, 1.0, 0.0, 1.0, 0, 0,
                                            0, None, 0, FAKE)


CALLS = [_matmul, lambda *a: _matmul(*a, transpose=1), _norm, _sum]


@pytest.mark.parametrize("dt", [0, 1])
def test_rows_ranges_and_widths(lib, dt):
    for f in CALLS:
        assert f(lib, dt, 1 << 30, 8, 4, 64, 64) == ALIGN
        assert f(lib, dt, (1 << 30) + 1, 8, 4, 64, 64) == SHAPE
        for E, B in ((1 << 4, 1 << 20), (1 << 20, 1 << 4), (1 << 23, 2)):
            assert f(lib, dt, 1000, E // 2, B, 5, 7) == ALIGN
        assert f(lib, dt, 1000, 1, 1 << 24, 5, 7) == ALIGN
        assert f(lib, dt, 1000, 1, (1 << 24) + 1, 5, 7) == SHAPE
        assert f(lib, dt, 100, 1, 2, 1 << 20, 1 << 10) == ALIGN
        assert f(lib, dt, 100, 1, 2, 1 << 10, 1 << 20) == ALIGN
        assert f(lib, dt, 100, 1, 2, (1 << 20) + 1, 8) == f(lib, dt, 100, 1, 2, 8, (1 << 20) + 1) == SHAPE


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("d", [64, 65])
def test_products_tiles(lib, dt, d):
    """(R / 128 + E) * ceil(n / 128) at most 2^24 - 8 for n output columns."""
    for n in (1, 128, 129, 50304, 50305):
        cols = -(-n // 128)
        rows = ((1 << 24) - 8) // cols - 100  # row tiles that fit beside 100 experts
        R = rows * 128
        if R <= 1 << 30:
            assert _matmul(lib, dt, R + 127, 100, 3, d, n) == ALIGN, n
            assert _matmul(lib, dt, R + 128, 100, 3, d, n) == SHAPE, n
            assert _matmul(lib, dt, R + 127, 100, 3, n, d, 1) == ALIGN, n
            assert _matmul(lib, dt, R + 128, 100, 3, n, d, 1) == SHAPE, n
    # a million rows of a vocabulary's width, refused for the 32-row tiles of other sizes before
    assert _matmul(lib, dt, 1000000, 8, 32, 1280, 50304) == ALIGN


@pytest.mark.parametrize("dt", [0, 1])
def test_sums_tiles_and_noise(lib, dt):
    """E * ceil(d / 128) * ceil(p / 128) below 2^23 and ceil(E d / 4) p below 2^32."""
    assert _sum(lib, dt, 1000, (1 << 23) - 1, 1, 1, 1) == ALIGN
    assert _sum(lib, dt, 1000, 1 << 23, 1, 1, 1) == SHAPE
    assert _sum(lib, dt, 1000, 1 << 13, 1, 1 << 10, (1 << 11) - 1) == ALIGN
    assert _sum(lib, dt, 1000, 1 << 13, 1, 1 << 10, 1 << 11) == SHAPE
    # neither is a limit of the other calls
    for f in CALLS[:3]:
        assert f(lib, dt, 1000, 1 << 23, 1, 1, 1) == ALIGN
        assert f(lib, dt, 1000, 64, 1, 1 << 14, 1 << 14) == ALIGN
        assert f(lib, dt, 1000, 1 << 20, 1, 300, 300) == ALIGN
    assert _sum(lib, dt, 1000, 1 << 20, 1, 300, 300) == SHAPE


@pytest.mark.parametrize("dt", [0, 1])
def test_workspace_of_sizes_that_one_call_refuses(lib, dt):
    """The largest workspace of the calls that take the sizes."""
    both = lib.dp_grouped_workspace_bytes(dt, 1000, (1 << 23) - 1, 1, 1, 1)
    assert both > 4 * 1000
    no_sum = lib.dp_grouped_workspace_bytes(dt, 1000, 1 << 23, 1, 1, 1)
    assert 4 * 1000 < no_sum  # the norm's
    assert lib.dp_grouped_workspace_bytes(dt, (1 << 30) + 1, 8, 4, 64, 64) == 0


def test_temperatures(lib):
    """From 2^-63 to 2^63: outside, the temperature's inverse or its square
    leaves fp32's range (a loss of NaN at 1e-39 and of 0 at 1e-38)."""
    def loss(tau):
        return lib.dp_distill_loss(None, FAKE + 8, FAKE, FAKE, 1, 0, 2, 3, 50, 4, tau, None, None, 0, FAKE, FAKE)

    def back(tau):
        return lib.dp_distill_loss_backward(None, FAKE + 8, FAKE, FAKE, 1, 0, 2, 3, 50, 4, tau, None, None, FAKE, FAKE)

    for f in (loss, back):
        for tau in (2.0 ** -63, 1e-6, 1.0, 1e6, 2.0 ** 63):
            assert f(tau) == ALIGN, tau
        for tau in (1e-39, 1e-38, 2.0 ** -64, 2.0 ** 64, 3e38):
            assert f(tau) == VALUE, tau
