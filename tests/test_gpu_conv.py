"""Short causal convolution on the GPU against its float64 definition: forward,
backward and single-token step (marked gpu).

Roundings counted per term: W + 1 multiply-adds, and about 40 in the sigmoid (its
argument's rounding is scaled by |p|, below 10 here, twice) -- 64; the gradients go
through the sigmoid's derivative as well -- 128; the sums of dweight and dbias over R
rows are 16 in a run, 5 across lanes and waves, one per block of 512."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _inputs(B, T, C, W, io, bias=True, state=True, cu=None, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    return dict(x=r(B, T, C).to(io), weight=0.5 * r(C, W), bias=r(C) if bias else None,
                state0=r(n, W - 1, C).to(io) if state else None), r(B, T, C).to(io), r(n, W - 1, C).to(io)


CASES = [  # B, T, C, W, cu, bias, state, silu
    (2, 37, 64, 4, None, True, True, True),
    (1, 1, 8, 4, None, True, True, True),
    (3, 2, 72, 4, None, False, True, False),
    (1, 515, 264, 4, None, True, False, True),
    (2, 100, 520, 3, None, False, False, True),
    (1, 16, 8, 2, None, True, True, False),
    (1, 64, 128, 4, [0, 0, 1, 3, 6, 6, 22, 38, 64, 64], True, True, True),
    (1, 70, 40, 3, [0, 1, 2, 3, 4, 35, 70], True, True, True),
    (1, 700, 24, 2, [0, 15, 16, 17, 511, 512, 513, 700], False, True, False),
    (1, 33, 16, 4, [0, 33], True, False, True),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,C,W,cu,bias,state,silu", CASES)
def test_forward(B, T, C, W, cu, bias, state, silu, io):
    a, _, _ = _inputs(B, T, C, W, io, bias, state, cu)
    y_ref, s_ref = ref.conv(*ref._f64(a["x"], a["weight"], a["bias"], a["state0"]), cu, silu)
    size = ref.conv_sizes(a["x"], a["weight"], a["bias"], a["state0"], cu)
    room = torch.full((B, T + 2, C), 7.0, device=DEV, dtype=io) if B == 1 else None
    out = room[:, 1:T + 1] if room is not None else None
    y, last = gdn.conv_fwd(**a, cu_seqlens=cu, activation="silu" if silu else None, out=out)
    torch.cuda.synchronize()
    if room is not None:
        assert bool((room[:, 0] == 7).all()) and bool((room[:, T + 1] == 7).all())
    ref.check("y", y, y_ref, size["y"], 64)
    assert torch.equal(last.double().cpu(), s_ref)  # rows of the input, kept exactly


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dlast", [False, True])
@pytest.mark.parametrize("B,T,C,W,cu,bias,state,silu", CASES)
def test_backward(B, T, C, W, cu, bias, state, silu, io, dlast):
    a, dy, ds = _inputs(B, T, C, W, io, bias, state, cu)
    ds = ds if dlast else None
    want = ref.conv_grads(a["x"], a["weight"], a["bias"], a["state0"], cu, silu, dy, ds)
    size = ref.conv_sizes(a["x"], a["weight"], a["bias"], a["state0"], cu, dy, ds)
    got = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds, cu_seqlens=cu,
                       activation="silu" if silu else None)
    again = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds, cu_seqlens=cu,
                         activation="silu" if silu else None)
    torch.cuda.synchronize()
    for key in ("dx", "dweight", "dbias", "dstate0"):
        assert (got[key] is None) == (want[key] is None), key
        if got[key] is not None:
            assert torch.equal(got[key], again[key]), key
            ref.check(key, got[key], want[key], size[key], 128 + (32 if key in ("dweight", "dbias") else 0))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,C,W", [(1, 8, 4), (5, 264, 3), (33, 1032, 2), (2, 64, 4)])
def test_steps_equal_the_prompt(B, C, W, io):
    """T single steps give the prompt's rows and final state bit for bit: the same
    multiply-adds in the same order."""
    T = 6
    a, _, _ = _inputs(B, T, C, W, io)
    y, last = gdn.conv_fwd(**a)
    state = a["state0"].clone()
    for t in range(T):
        yt = gdn.conv_step(a["x"][:, t:t + 1].contiguous(), a["weight"], state, bias=a["bias"])
        assert torch.equal(yt, y[:, t:t + 1]), t
    assert torch.equal(state, last)


def test_a_sequence_of_nan_stays_alone():
    cu = [0, 10, 30, 41]
    a, dy, ds = _inputs(1, 41, 64, 4, F32, True, True, cu)
    clean_y, clean_s = gdn.conv_fwd(**a, cu_seqlens=cu)
    clean = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds, cu_seqlens=cu)
    a["x"][:, 10:30] = float("nan")
    y, s = gdn.conv_fwd(**a, cu_seqlens=cu)
    got = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds, cu_seqlens=cu)
    for rows in (slice(0, 10), slice(30, 41)):
        assert torch.equal(y[:, rows], clean_y[:, rows])
        assert torch.equal(got["dx"][:, rows], clean["dx"][:, rows])
    assert torch.equal(s[[0, 2]], clean_s[[0, 2]])
    assert bool(y[:, 10:30].isnan().all())


def test_large_pre_activations():
    """silu at +-100 and beyond: p and -0 (the sigmoid's exponential over- or underflows)."""
    x = torch.tensor([-3e38, -1e4, -100.0, 100.0, 1e4, 3e38], device=DEV).reshape(1, 6, 1).expand(1, 6, 8).contiguous()
    w = torch.zeros(8, 2, device=DEV)
    w[:, 1] = 1
    y, _ = gdn.conv_fwd(x, w)
    want = x.double() * torch.sigmoid(x.double())
    assert float((y.double() - want).abs()[:, :3].max()) < 1e-37
    assert torch.equal(y[:, 3:], x[:, 3:])


def test_no_tokens():
    a, dy, ds = _inputs(2, 0, 16, 4, F32)
    y, last = gdn.conv_fwd(**a)
    got = gdn.conv_bwd(a["x"], a["weight"], dy, bias=a["bias"], state0=a["state0"], dstate_final=ds)
    assert y.shape == (2, 0, 16) and torch.equal(last, a["state0"])
    assert torch.equal(got["dstate0"], ds) and float(got["dweight"].abs().max()) == 0 and float(got["dbias"].abs().max()) == 0
