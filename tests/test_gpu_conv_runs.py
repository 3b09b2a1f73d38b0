"""Short convolution at sizes that take its other instances: runs of eight rows in the
forward (2^21 values and more), eight and more blocks of 512 rows in the backward's last
kernel, against the float64 definition (marked gpu).

Roundings counted per term: 64 in the forward and 128 in a gradient, as test_gpu_conv.py
does; the sums of dweight and dbias have 32 multiply-adds in a run, two additions over the
lanes, two over the waves, and over the blocks of 512 rows one in eight of them, up to seven
for what is left over eight and three that join the eight sums."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
PACKED = [0, 0, 1, 3, 8, 13, 16, 16, 29, 30, 500, 505, 511, 1030, 1030]  # cuts inside, at and between runs of eight


def _inputs(B, T, C, W, io, bias, state, cu, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    return dict(x=r(B, T, C).to(io), weight=0.5 * r(C, W), bias=r(C) if bias else None,
                state0=r(n, W - 1, C).to(io) if state else None), r(B, T, C).to(io), r(n, W - 1, C).to(io)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C,cu,bias,state,silu", [
    (1, 1030, 2048, PACKED, True, True, True),
    (1, 1030, 2048, PACKED, False, False, False),
    (1, 1024, 2048, None, True, True, False),      # exactly 2^21 values
    (3, 701, 1000, None, False, True, True),       # runs that cross from one sequence into the next
    (1, 2105, 1000, [0, 7, 2105], True, False, True),
])
def test_forward_in_runs_of_eight(B, T, C, cu, bias, state, silu, W, io):
    assert B * T * C >= 1 << 21
    a, _, _ = _inputs(B, T, C, W, io, bias, state, cu)
    y_ref, s_ref = ref.conv(*ref._f64(a["x"], a["weight"], a["bias"], a["state0"]), cu, silu)
    size = ref.conv_sizes(a["x"], a["weight"], a["bias"], a["state0"], cu)
    room = torch.full((B + 2, T, C), 7.0, device=DEV, dtype=io)
    y, last = gdn.conv_fwd(**a, cu_seqlens=cu, activation="silu" if silu else None, out=room[1:B + 1])
    torch.cuda.synchronize()
    assert bool((room[0] == 7).all()) and bool((room[B + 1] == 7).all())
    ref.check("y", y, y_ref, size["y"], 64)
    assert torch.equal(last.double().cpu(), s_ref)  # rows of the input, kept exactly


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,C,W,cu", [
    (1, 4096, 24, 4, None),                 # eight blocks
    (1, 4200, 24, 4, [0, 1, 511, 513, 4000, 4000, 4200]),
    (2, 2350, 72, 3, None),                 # ten, sequences that end inside one
    (1, 8200, 16, 2, None),                 # seventeen
    (1, 8110, 40, 4, [0, 4095, 4097, 8110]),
])
def test_backward_over_many_blocks(B, T, C, W, cu, io):
    a, dy, ds = _inputs(B, T, C, W, io, True, True, cu, seed=1)
    want = ref.conv_grads(a["x"], a["weight"], a["bias"], a["state0"], cu, True, dy, ds)
    size = ref.conv_sizes(a["x"], a["weight"], a["bias"], a["state0"], cu, dy, ds)
    blocks = -(-B * T // 512)
    assert blocks >= 8
    got = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds, cu_seqlens=cu)
    for key in ("dx", "dstate0"):
        ref.check(key, got[key], want[key], size[key], 128)
    for key in ("dweight", "dbias"):
        ref.check(key, got[key], want[key], size[key], 128 + 32 + 4 + blocks // 8 + 7 + 3)
