"""Gated linear recurrence on the GPU against its float64 definition: forward (whole and
in segments), backward from the kept states, single-token step (marked gpu).  The bounds
are counted in _hybrid_oracle.glr."""
import math

import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, C, io, z=True, state=True, cu=None, seed=0, slow=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    a = dict(x=r(B, T, C).to(io), r=r(B, T, C).to(io), i=r(B, T, C).to(io), lam=(2 * r(C) - (6 if slow else 2)),
             z=r(B, T, C).to(io) if z else None)
    return a, (r(n, C) if state else None), r(B, T, C).to(io), (r(n, C) if state else None)


def compare(a, h0, dy, dl, cu, c=8.0):
    want, err = ref.glr(*a.values(), h0, cu, c=c, dy=dy, dlast=dl)
    B, T, C = a["x"].shape
    room = torch.full((1, T + 2, C), 7.0, device=DEV, dtype=a["x"].dtype) if B == 1 else None
    y, h = gdn.glr_fwd(**a, h0=h0, c=c, cu_seqlens=cu, out=room[:, 1:T + 1] if room is not None else None)
    y2, h2, saved = gdn.glr_fwd_save(**a, h0=h0, c=c, cu_seqlens=cu)
    got = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, c=c, cu_seqlens=cu)
    again = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, c=c, cu_seqlens=cu)
    torch.cuda.synchronize()
    if room is not None:  # rows beside the output are left as they were
        assert bool((room[:, 0] == 7).all()) and bool((room[:, T + 1] == 7).all())
    assert torch.equal(y, y2) and torch.equal(h, h2)
    got = {"y": y, "state": h, **got}
    assert set(got) - {"dz"} == set(want) - {"dz"} and (got["dz"] is None) == (a["z"] is None)
    for key, value in got.items():
        if value is None:
            continue
        ref.check(key, value, want[key], err[key])
        if key in again:
            assert torch.equal(value, again[key]), key


CASES = [  # B, T, C, cu, z, state
    (2, 33, 64, None, True, True),
    (1, 1, 8, None, True, True),
    (3, 8, 40, None, False, False),
    (2, 257, 72, None, False, True),
    (1, 700, 16, None, True, False),
    (1, 97, 64, [0, 0, 1, 16, 33, 33, 96, 97, 97], True, True),
    (1, 600, 40, [0, 270, 272, 600], True, True),
    (1, 64, 2056, [0, 1, 64], False, True),
    (5, 31, 264, None, True, True),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,C,cu,z,state", CASES)
def test_glr(B, T, C, cu, z, state, io):
    a, h0, dy, dl = inputs(B, T, C, io, z, state, cu)
    compare(a, h0, dy, dl, cu)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T,C,cu", [(3000, 8, None), (2049, 64, None), (4100, 32, [0, 3000, 3003, 3003, 4100])])
def test_in_segments(T, C, cu, io):
    """Few channels and many tokens, decays near one: several segments, whose starts are composed."""
    a, h0, dy, dl = inputs(1, T, C, io, True, True, cu, slow=True)
    assert gdn.glr_buffers(a["x"], cu_seqlens=cu)["forward"] > 0  # the split is taken
    compare(a, h0, dy, dl, cu)


@pytest.mark.parametrize("c", [0.0, 1.0, 30.0])
def test_factor(c):
    a, h0, dy, dl = inputs(2, 40, 24, F32)
    compare(a, h0, dy, dl, None, c=c) if c else None
    y, h = gdn.glr_fwd(**{**a, "z": None}, h0=h0, c=c)
    if c == 0:  # nothing decays and nothing is written
        assert torch.equal(h, h0) and torch.equal(y, h0.unsqueeze(1).expand(2, 40, 24))


def test_extreme_gates():
    """Gates open and shut so far that sigmoids saturate, lam far out on both sides: finite,
    and the limits of the definition."""
    a, h0, dy, dl = inputs(1, 24, 16, F32, z=False)
    a["r"][:, :8] = -200.0
    a["r"][:, 8:16] = 200.0
    a["i"][:, 4:12] = -200.0
    a["lam"][:4] = torch.tensor([-120.0, -60.0, 40.0, 90.0], device=DEV)
    y, h, saved = gdn.glr_fwd_save(**a, h0=h0)
    got = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)
    for t in (y, h, *(v for v in got.values() if v is not None)):
        assert bool(torch.isfinite(t).all())
    assert torch.equal(y[:, :8], h0.unsqueeze(1).expand(1, 8, 16))  # shut: the state stays
    assert float(y[0, 11, 2:4].abs().max()) == 0.0                  # forgotten, nothing written
    assert float(got["dr"][:, :8].abs().max()) == 0.0


def test_nan_and_infinity_reach_later_tokens_of_their_channel_alone():
    cu = [0, 30, 60]
    a, h0, dy, _ = inputs(1, 60, 40, F32, z=False, cu=cu)
    clean, _ = gdn.glr_fwd(**a, h0=h0, cu_seqlens=cu)
    a["x"][0, 12, 5] = math.nan
    a["x"][0, 40, 6] = math.inf
    y, h, saved = gdn.glr_fwd_save(**a, h0=h0, cu_seqlens=cu)
    touched = torch.zeros_like(y, dtype=torch.bool)
    touched[0, 12:30, 5] = True
    touched[0, 40:60, 6] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert not bool(torch.isfinite(y[touched]).any())
    dy[0, 20, 9] = math.nan
    got = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, cu_seqlens=cu)
    bad = ~torch.isfinite(got["di"])
    assert bool(bad[0, :21, 9].all()) and not bool(bad[0, 21:, 9].any()) and not bool(bad[0, 30:, 5].any())
    assert not bool(bad[..., [c for c in range(40) if c not in (5, 6, 9)]].any())


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,C,z", [(1, 8, True), (3, 72, False), (257, 264, True)])
def test_step_is_one_token(B, C, z, io):
    a, h0, _, _ = inputs(B, 1, C, io, z)
    want, err = ref.glr(*a.values(), h0, None)
    state = h0.clone()
    y = gdn.glr_step(**a, state=state)
    ref.check("y", y, want["y"], err["y"])
    ref.check("state", state, want["state"], err["state"])


def test_wants():
    a, h0, dy, dl = inputs(2, 20, 16, BF)
    y, h = gdn.glr_fwd(**a, h0=h0, output_final_state=False)
    assert h is None
    _, _, saved = gdn.glr_fwd_save(**a, h0=h0)
    full = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)
    part = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, want_dh0=False)
    assert part["dh0"] is None and all(torch.equal(part[k], full[k]) for k in full if k != "dh0")


def test_empty():
    for B, T, cu in ((0, 5, None), (2, 0, None), (1, 0, [0]), (1, 0, [0, 0, 0])):
        a, h0, dy, dl = inputs(B, T, 16, F32, cu=cu)
        y, h, saved = gdn.glr_fwd_save(**a, h0=h0, cu_seqlens=cu)
        got = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
        assert y.shape == a["x"].shape and torch.equal(h, h0)
        assert torch.equal(got["dh0"], dl) and float(got["dlam"].abs().max()) == 0.0


def test_gradients_against_differences():
    """The whole chain of a fp32 call against central differences of its own forward: the
    step h leaves h^2 times a third derivative (below 1e-3 here) and roundings of 300 2^-24 / h."""
    a, h0, dy, dl = inputs(1, 12, 8, F32)
    _, _, saved = gdn.glr_fwd_save(**a, h0=h0)
    got = gdn.glr_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)

    def loss(b, s):
        y, h = gdn.glr_fwd(**b, h0=s)
        return float((y.double() * dy).sum() + (h.double() * dl).sum())

    for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("z", "dz"), ("h0", "dh0")):
        for j in (0, 5):
            out = []
            for sign in (1, -1):
                b, s = {k: v.clone() for k, v in a.items()}, h0.clone()
                (s if name == "h0" else b[name]).view(-1)[j] += sign * 2.0 ** -6
                out.append(loss(b, s))
            assert abs((out[0] - out[1]) * 32 - float(got[grad].view(-1)[j])) <= 2e-2, name
