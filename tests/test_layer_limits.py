"""The sizes that the convolution takes are those its header states, and no launch of an
accepted problem has 2^32 threads or more (CPU only: no kernel is launched)."""
import ctypes
import itertools

import pytest

from gated_deltanet_chunked_gdn_amd import _native as nat

LIMIT = (1 << 32) - (1 << 23)


def status(B, T, C, W, io):
    p = nat.ConvProblem(B, T, C, W, B, None, None, io, nat.GDN_ACT_SILU)
    return nat.load().gdn_conv_workspace_size(p, ctypes.c_size_t(0))


def up256(n):
    return (n + 255) // 256 * 256


def launches(B, T, C, W, io):
    """Threads of the launches that count them in one dimension: forward with its kept
    rows, step, last kernel of the backward with dstate0."""
    rows, vec = B * T, 8 if io == nat.GDN_BF16 else 4
    run = 2 if rows * (C // 4) // 8 < 1 << 16 else 8
    forward = up256(-(-rows // run) * (C // 4) + B * (W - 1) * (C // vec))
    return forward, up256(B * (C // vec)), up256(up256((W + 1) * C) + B * (C // vec))


def stated(B, T, C, W, io):
    return B * T * C // 32 + B * (W - 1) * (C // (8 if io == nat.GDN_BF16 else 4)) <= LIMIT and B * T < 1 << 31 and B <= 65535


SIZES = [(1, 4200000), (1, (1 << 31) - 1), (16383, 0), (16384, 0), (65535, 0), (65535, 1), (65535, 3), (4096, 4096), (4095, 1),
         (32, 8000), (31, 4095), (1, 130000), (8191, 1), (5460, 1), (2, 1 << 30)]


@pytest.mark.parametrize("io", [nat.GDN_BF16, nat.GDN_FP32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_accepted_problems_are_the_stated_ones_and_fit_a_launch(W, io):
    for (B, T), C in itertools.product(SIZES, (8, 64, 4096, 8192, 65536, 1 << 18, (1 << 20) - 8, 1 << 20)):
        ok = stated(B, T, C, W, io)
        assert status(B, T, C, W, io) == (nat.GDN_OK if ok else nat.GDN_ERR_UNSUPPORTED), (B, T, C)
        if ok:
            assert max(launches(B, T, C, W, io)) < 1 << 32, (B, T, C)


def test_many_rows_of_wide_layers_are_taken():
    assert status(1, 4200000, 4096, 4, nat.GDN_BF16) == nat.GDN_OK


def test_more_threads_than_a_launch_has_are_refused():
    """Last kernel of the backward: 3 2^20 threads for the sums and 16383 2^18 for dstate0."""
    assert launches(16383, 0, 1 << 20, 2, nat.GDN_FP32)[2] >= 1 << 32
    assert status(16383, 0, 1 << 20, 2, nat.GDN_FP32) == nat.GDN_ERR_UNSUPPORTED
