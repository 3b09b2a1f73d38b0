"""Norm and rotation of queries and keys on the GPU against the float64 definition, forward
and backward (marked gpu).  The bounds are counted in _hybrid_oracle.rope."""
import math

import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, Hq, Hk, D, R, io, norm="rms", weights=True, views=True, far=1000, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if views:  # columns of one projection
        rows = r(B, T, (Hq + 2 * Hk) * D).to(io)
        q, k = rows[..., :Hq * D].unflatten(-1, (Hq, D)), rows[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = r(B, T, Hq, D).to(io), r(B, T, Hk, D).to(io)
    freq = 10000.0 ** (-torch.arange(R // 2, device=DEV) * 2.0 / max(R, 1))
    pos = torch.randint(-3, far, (B, T), generator=g, device=DEV, dtype=torch.int32)
    w = (r(D), r(D)) if norm == "rms" and weights else (None, None)
    return q, k, freq, pos, w, r(B, T, Hq, D).to(io), r(B, T, Hk, D).to(io)


def compare(q, k, freq, pos, w, dq, dk, norm, inter, eps=1e-6):
    how = dict(positions=pos, norm=norm, eps=eps, wq=w[0], wk=w[1], interleaved=inter)
    yq, yk = gdn.rope_fwd(q, k, freq, **how)
    got = gdn.rope_bwd(q, k, freq, dq, dk, **how)
    again = gdn.rope_bwd(q, k, freq, dq, dk, **how)
    at = pos if pos is not None else torch.arange(q.shape[1], device=DEV).expand(q.shape[:2])
    for name, x, wx, d, y in (("q", q, w[0], dq, yq), ("k", k, w[1], dk, yk)):
        want, err = ref.rope(x, wx, freq, at, norm, eps, inter, d)
        ref.check(name, y, want["out"], err["out"])
        ref.check("d" + name, got["d" + name], want["dx"], err["dx"])
        assert torch.equal(got["d" + name], again["d" + name])
        if wx is None:
            assert got["dw" + name] is None
        else:
            ref.check("dw" + name, got["dw" + name], want["dw"], err["dw"])
            assert torch.equal(got["dw" + name], again["dw" + name])


CASES = [  # B, T, Hq, Hk, D, R, norm, weights, views
    (2, 5, 4, 2, 128, 128, "rms", True, True),
    (1, 1, 1, 1, 64, 64, "rms", False, True),
    (3, 1, 16, 4, 128, 64, "l2", False, True),
    (1, 77, 6, 6, 64, 16, "l2", False, False),
    (2, 33, 3, 1, 256, 112, "rms", True, True),
    (2, 33, 3, 1, 256, 256, None, False, True),
    (1, 9, 40, 8, 128, 96, "rms", True, False),
    (1, 2, 2, 2, 128, 0, "rms", True, True),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R,norm,weights,views", CASES)
def test_rope(B, T, Hq, Hk, D, R, norm, weights, views, io, inter):
    q, k, freq, pos, w, dq, dk = inputs(B, T, Hq, Hk, D, R, io, norm, weights, views)
    compare(q, k, freq, pos, w, dq, dk, norm, inter)


@pytest.mark.parametrize("T", [4096, 4099, 9001])
def test_many_tokens(T):
    """Four tokens a workgroup, and more than the backward has workgroups for at once."""
    q, k, freq, _, w, dq, dk = inputs(1, T, 3, 1, 64, 64, BF)
    compare(q, k, freq, None, w, dq, dk, "rms", False)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    """An angle of 10^6 and more, of which fp32 would keep no fraction of a turn."""
    q, k, freq, pos, w, dq, dk = inputs(1, 40, 2, 1, 64, 64, F32, far=far)
    pos[0, :2] = torch.tensor([far, -far], dtype=torch.int32)
    compare(q, k, freq, pos, w, dq, dk, "rms", False)


def test_rows_of_zeros_and_of_extremes():
    q, k, freq, pos, w, dq, dk = inputs(1, 6, 2, 1, 64, 64, F32, norm="l2", views=False)
    q[0, 0] = 0
    k[0, 1] = 0
    q[0, 2, 0] *= 1e15
    q[0, 2, 1] *= 1e-15
    compare(q, k, freq, pos, w, dq, dk, "l2", False)
    y, _ = gdn.rope_fwd(q, k, freq, positions=pos, norm="rms", eps=1e-6)
    assert float(y[0, 0].abs().max()) == 0.0


def test_nan_stays_in_its_row():
    q, k, freq, pos, w, dq, dk = inputs(1, 8, 2, 2, 64, 32, BF, norm=None, views=False)
    clean_q, clean_k = gdn.rope_fwd(q, k, freq, positions=pos, norm=None)
    q[0, 3, 1, 2] = math.nan   # pair (2, 18)
    k[0, 5, 0, 40] = math.inf  # behind the rotation
    yq, yk = gdn.rope_fwd(q, k, freq, positions=pos, norm=None)
    bad_q, bad_k = ~torch.isfinite(yq), ~torch.isfinite(yk)
    assert bad_q.nonzero().tolist() == [[0, 3, 1, 2], [0, 3, 1, 18]] and bad_k.nonzero().tolist() == [[0, 5, 0, 40]]
    assert torch.equal(yq[~bad_q], clean_q[~bad_q]) and torch.equal(yk[~bad_k], clean_k[~bad_k])
    got = gdn.rope_bwd(q, k, freq, dq, dk, positions=pos, norm=None)
    assert bool(torch.isfinite(got["dq"]).all()) and bool(torch.isfinite(got["dk"]).all())
    yq, _ = gdn.rope_fwd(q, k, freq, positions=pos, norm="rms")
    assert (~torch.isfinite(yq)).any(-1).nonzero().tolist() == [[0, 3, 1]]


def test_outputs_of_the_caller():
    q, k, freq, pos, w, _, _ = inputs(1, 7, 2, 1, 64, 64, BF)
    room = torch.full((9, 2, 64), 7.0, device=DEV, dtype=BF)
    want = gdn.rope_fwd(q, k, freq, positions=pos, wq=w[0], wk=w[1])
    yq, yk = gdn.rope_fwd(q, k, freq, positions=pos, wq=w[0], wk=w[1], q_out=room[1:8].unsqueeze(0))
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    assert bool((room[0] == 7).all()) and bool((room[8] == 7).all())


def test_empty():
    q, k, freq, pos, w, dq, dk = inputs(2, 0, 2, 1, 64, 64, BF, views=False)
    yq, yk = gdn.rope_fwd(q, k, freq, positions=pos, wq=w[0], wk=w[1])
    got = gdn.rope_bwd(q, k, freq, dq, dk, positions=pos, wq=w[0], wk=w[1])
    assert yq.shape == q.shape and float(got["dwq"].abs().max()) == 0.0 and float(got["dwk"].abs().max()) == 0.0


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("io", [BF, F32])
def test_nan_makes_its_row_nan(io, norm):
    """The norm of a row that holds a NaN is NaN, and so is all of the row and of its gradient."""
    q, k, freq, pos, _, dq, dk = inputs(1, 8, 2, 2, 64, 32, io, norm=norm, views=False)
    clean = gdn.rope_fwd(q, k, freq, positions=pos, norm=norm), gdn.rope_bwd(q, k, freq, dq, dk, positions=pos, norm=norm)
    q[0, 3, 1, 2] = math.nan
    k[0, 5, 0, 40] = math.nan
    y, got = gdn.rope_fwd(q, k, freq, positions=pos, norm=norm), gdn.rope_bwd(q, k, freq, dq, dk, positions=pos, norm=norm)
    for t, was, at in ((y[0], clean[0][0], (3, 1)), (y[1], clean[0][1], (5, 0)), (got["dq"], clean[1]["dq"], (3, 1)), (got["dk"], clean[1]["dk"], (5, 0))):
        assert bool(torch.isnan(t[0, at[0], at[1]]).all())
        rest = torch.ones(t.shape[:3], dtype=torch.bool, device=DEV)
        rest[0, at[0], at[1]] = False
        assert torch.equal(t[rest], was[rest])
