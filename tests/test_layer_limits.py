"""The sizes that the convolution takes are those its header states, and no launch of an
accepted problem has 2^32 threads or more (CPU only: no kernel is launched)."""
import ctypes
import itertools

import pytest
import torch

from gated_deltanet_chunked_gdn_amd import _native as nat
from gated_deltanet_chunked_gdn_amd import layer

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


def _calls():
    many = (1 << 32) + 1  # one sequence, counted in 32 bits
    z = torch.zeros
    x, w = z(many, 0, 8), z(8, 4)
    u, A, Bm = z(many, 0, 8), z(8, 8), z(many, 0, 1, 8)
    q, v, g, S = z(many, 1, 0, 64), z(many, 1, 0, 16), z(many, 1, 0), z(many, 0, 64, 16)
    return {"conv_fwd": lambda: layer.conv_fwd(x, w), "conv_bwd": lambda: layer.conv_bwd(x, w, x),
            "conv_step": lambda: layer.conv_step(z(many, 1, 0), z(0, 4), z(many, 3, 0)),
            "conv_packed": lambda: layer.conv_fwd(z(1, many, 0), z(0, 4), cu_seqlens=layer_seqs([0, 1])),
            "scan_fwd": lambda: layer.scan_fwd(u, u, A, Bm, Bm), "scan_buffers": lambda: layer.scan_buffers(u, Bm),
            "scan_packed": lambda: layer.scan_buffers(z(1, many, 0), z(1, many, 0, 8), cu_seqlens=layer_seqs([0, 1])),
            "scan_step": lambda: layer.scan_step(z(many, 1, 0), z(many, 1, 0), z(0, 8), z(many, 1, 0, 8), z(many, 1, 0, 8), z(many, 0, 8)),
            "step": lambda: layer.step(q, q, v, g, g, S), "kda_step": lambda: layer.kda_step(q, q, v, q, g, S)}


def layer_seqs(offsets):
    from gated_deltanet_chunked_gdn_amd.ops import SeqLens

    return SeqLens(offsets, "cpu")


@pytest.mark.parametrize("name", sorted(_calls()))
def test_sizes_beyond_32_bits_are_refused(monkeypatch, name):
    """The library's sizes are 32-bit: 2^32 + 1 sequences or tokens must not be taken for one
    (host tensors without elements, on which no call gets past its checks)."""
    monkeypatch.setattr(layer, "_first", lambda t, *_: t.get_device())
    monkeypatch.setattr(layer, "_packed", lambda cu, dev: cu)
    monkeypatch.setattr(layer, "_call", lambda *a: pytest.fail("the library call was reached"))
    with pytest.raises(ValueError, match="4294967297"):
        _calls()[name]()


def _segments(T, D, N, pass_):
    """Slots of segments that the workspace of one sequence has: its end states and sums."""
    p = nat.ScanProblem(1, T, D, N, 1, 1, None, None, nat.GDN_FP32, 1)
    n = ctypes.c_size_t(0)
    assert nat.load().gdn_scan_workspace_size(p, pass_, n) == nat.GDN_OK
    if pass_ == nat.GDN_SCAN_BWD:  # and the partial sums of dB and dC, of dA, dD and ddt_bias
        return (n.value - -(-D // 64) * T * 2 * N * 4) // (D * (2 * N + 3) * 4)
    return n.value // (D * (N + 1) * 4)


@pytest.mark.parametrize("T", [4096, 5000, 8192, 16384, 65536, 262144, 1 << 20])
@pytest.mark.parametrize("D,N", [(64, 8), (64, 16), (256, 16), (64, 32), (64, 64), (1024, 64)])
def test_scan_segments_do_not_outgrow_their_tokens(T, D, N):
    """Every segment composes all the others of its sequence, so their number squared stays
    near the sequence's tokens (times the backward's passes over wide states; a third more
    where lengths are rounded to 16 tokens), and the split is still taken."""
    for pass_, tokens in ((nat.GDN_SCAN_FWD, T), (nat.GDN_SCAN_BWD, T * max(1, N // 16))):
        segs = _segments(T, D, N, pass_)
        assert 16 <= segs <= 4 / 3 * max(64, tokens ** 0.5) + 1, (pass_, segs)
