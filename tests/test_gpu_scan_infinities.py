"""Infinities in the selective scan's inputs: values that the definition leaves finite stay
finite, and infinities reach the outputs that the definition gives them to, as infinities
(marked gpu).

All inputs but A are positive, so that no two infinities of opposite signs meet unless they
do in the definition as well; the decays of T tokens stay far above the smallest fp32 value
(A >= -0.4, steps below 1).  Finite values: tolerances as counted in test_gpu_scan.py."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")
GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def _inputs(T, D, N, G, io, z, n=1, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=gen, device=DEV) + 0.1  # noqa: E731
    a = dict(u=r(1, T, D).to(io), dt=r(1, T, D).to(io), A=-0.1 - 0.2 * r(D, N), Bm=r(1, T, G, N).to(io), Cm=r(1, T, G, N).to(io),
             D=r(D), z=r(1, T, D).to(io) if z else None, dt_bias=r(D) - 2)
    return a, r(n, D, N), r(1, T, D).to(io), r(n, D, N)


def _compare(name, got, want, size, roundings):
    x, r = got.detach().double().cpu(), want.double()
    assert torch.equal(x.isnan(), r.isnan()), (name, "NaN", int(x.isnan().sum()), int(r.isnan().sum()))
    for inf in (INF, -INF):
        assert torch.equal(x == inf, r == inf), (name, inf)
    ok = r.isfinite()
    ref.check(name, got.cpu()[ok], r[ok], size[ok], roundings)


def _case(a, h0, dy, dl, cu):
    want, size = (ref.scan(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], a["dt_bias"], h0, cu, True, dy, dl, s)
                  for s in (False, True))
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    T, D, N = a["u"].shape[1], a["u"].shape[2], a["A"].shape[1]
    _compare("y", y, want["y"], size["y"], 3 * T + N + 64)
    _compare("state", h, want["state"], size["state"], 3 * T + 64)
    for key in GRADS:
        if got[key] is not None:
            _compare(key, got[key], want[key], size[key], 7 * T + N + D + 128)
    return got


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("name", ["Bm", "Cm"])
@pytest.mark.parametrize("D,N,G,z", [(8, 16, 1, True), (72, 16, 1, False), (80, 8, 2, True), (104, 32, 1, True), (48, 64, 2, False),
                                     (64, 16, 1, True)])
def test_infinite_write_or_read_vector(D, N, G, z, name, io):
    """dC behind an infinite B and dB before an infinite C are infinite, in groups whose
    channels fill no whole tile of 64 too."""
    a, h0, dy, dl = _inputs(32, D, N, G, io, z)
    a[name][0, 21, G - 1, N - 3] = INF
    got = _case(a, h0, dy, dl, None)
    key, rows = ("dC", slice(21, 32)) if name == "Bm" else ("dB", slice(0, 22))
    assert bool((got[key][0, rows, G - 1, N - 3] == INF).all())


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("value", [INF, float("nan")])
@pytest.mark.parametrize("T,D,N,cu", [(37, 64, 16, None), (37, 24, 8, None), (49, 64, 32, None), (31, 72, 64, None),
                                      (60, 64, 16, [0, 21, 32, 60])])
def test_a_last_token_that_is_not_finite(T, D, N, cu, value, io):
    """The last state of a sequence enters dC of the last token and no other gradient: dA
    holds the states before the tokens, so it stays finite, wherever the sequence ends."""
    a, h0, dy, dl = _inputs(T, D, N, 1, io, True, n=len(cu) - 1 if cu else 1)
    for end in (cu or [0, T])[1:]:
        a["u"][0, end - 1] = value
    got = _case(a, h0, dy, dl, cu)
    assert bool(got["dA"].isfinite().all())
    assert bool((got["dC"][0, -1].isnan() if value != value else got["dC"][0, -1] == INF).all())
