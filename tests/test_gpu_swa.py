"""Window attention on the GPU against its float64 definition: forward and backward over
dense and packed sequences (marked gpu).  The bounds are counted in _hybrid_oracle.swa."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
from gated_deltanet_chunked_gdn_amd import _native as nat
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, Hq, Hk, D, io, seed=0, views=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(io)  # noqa: E731
    if views:
        rows = r(B, T, (Hq + 2 * Hk) * D)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in rows.split([Hq * D, Hk * D, Hk * D], dim=-1))
        return q, k, v, r(B, T, Hq, D)
    return r(B, T, Hq, D), r(B, T, Hk, D), r(B, T, Hk, D), r(B, T, Hq, D)


def compare(q, k, v, do, W, S, scale, cu):
    want, err = ref.swa(q, k, v, W, S, scale, cu, do)
    how = dict(sinks=S, scale=scale, cu_seqlens=cu)
    B, T = q.shape[:2]
    room = torch.full((1, T + 2, *q.shape[2:]), 7.0, device=DEV, dtype=q.dtype) if B == 1 else None
    o, lse = gdn.swa_fwd(q, k, v, W, return_lse=True, out=room[:, 1:T + 1] if room is not None else None, **how)
    assert torch.equal(gdn.swa_fwd(q, k, v, W, **how), o)
    got = gdn.swa_bwd(q, k, v, o, lse, do, W, **how)
    again = gdn.swa_bwd(q, k, v, o, lse, do, W, **how)
    torch.cuda.synchronize()
    if room is not None:
        assert bool((room[:, 0] == 7).all()) and bool((room[:, T + 1] == 7).all())
    ref.check("o", o, want["o"], err["o"])
    ref.check("lse", lse, want["lse"], err["lse"])
    for key in ("dq", "dk", "dv"):
        ref.check(key, got[key], want[key], err[key])
        assert torch.equal(got[key], again[key]), key


CASES = [  # B, T, Hq, Hk, D, W, S, cu, views
    (1, 1, 1, 1, 64, 1, 0, None, False),
    (2, 5, 2, 1, 64, 3, 0, None, False),
    (1, 65, 2, 2, 128, 1, 0, None, False),
    (1, 129, 4, 2, 128, 64, 0, None, True),
    (2, 200, 3, 1, 64, 65, 1, None, False),
    (1, 300, 2, 1, 128, 33, 4, None, True),
    (1, 260, 1, 1, 64, 1000, 3, None, False),
    (1, 290, 2, 1, 64, 17, 70, None, False),
    (1, 400, 2, 2, 64, 100, 130, None, False),
    (3, 64, 8, 1, 64, 64, 2, None, False),
    (1, 333, 4, 2, 64, 40, 3, [0, 0, 1, 65, 193, 193, 332, 333, 333], False),
    (1, 350, 2, 1, 128, 129, 2, [0, 130, 350], True),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hk,D,W,S,cu,views", CASES)
def test_swa(B, T, Hq, Hk, D, W, S, cu, views, io):
    q, k, v, do = inputs(B, T, Hq, Hk, D, io, views=views)
    compare(q, k, v, do, W, S, D ** -0.5, cu)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T,W,S,D,cu", [(1100, 60, 5, 64, None), (700, 31, 40, 128, None), (1300, 512, 33, 64, [0, 600, 601, 1300])])
def test_first_tokens_of_long_sequences(T, W, S, D, cu, io):
    """Several runs of queries behind the first tokens' window, more of them than one block of keys."""
    q, k, v, do = inputs(1, T, 2, 1, D, io, seed=1)
    compare(q, k, v, do, W, S, D ** -0.5, cu)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("cu", [[0, 900, 930, 1700, 1710, 1730, 2000], [0, 1300, 1331, 1362], [0, 40, 300, 340, 1700, 1740]])
def test_first_tokens_of_short_sequences_beside_long_ones(cu, io):
    """Sequences of a run of queries or less beside others of several: each has its own sums, and
    nothing is written behind the workspace."""
    T, W, S = cu[-1], 20, 5
    q, k, v, do = inputs(1, T, 2, 1, 64, io, seed=9)
    compare(q, k, v, do, W, S, 0.125, cu)
    o, lse = gdn.swa_fwd(q, k, v, W, sinks=S, scale=0.125, cu_seqlens=cu, return_lse=True)
    offsets = np.asarray(cu, dtype=np.int32)
    prob, size = nat.SwaProblem(1, T, 2, 1, 64, W, S, len(cu) - 1, offsets.ctypes.data, 4096, int(io is BF), 0.125, 0, 0, 0), ctypes.c_size_t()
    assert nat.load().gdn_swa_workspace_size(prob, nat.GDN_SWA_BWD, size) == nat.GDN_OK
    size = size.value
    room = torch.full((size + 65536,), 0x5a, dtype=torch.uint8, device=DEV)
    got = gdn.swa_bwd(q, k, v, o, lse, do, W, sinks=S, scale=0.125, cu_seqlens=cu, workspace=room[:size])
    with pytest.raises(gdn.GdnError):
        gdn.swa_bwd(q, k, v, o, lse, do, W, sinks=S, scale=0.125, cu_seqlens=cu, workspace=room[:size - 1])
    assert bool((room[size:] == 0x5a).all())
    want, err = ref.swa(q, k, v, W, S, 0.125, cu, do)
    for key in ("dq", "dk", "dv"):
        ref.check(key, got[key], want[key], err[key])


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scales(scale):
    """Scores of up to a hundred and more, rising where the maximum moves, and none at all."""
    q, k, v, do = inputs(1, 150, 2, 1, 64, F32, seed=2)
    compare(q, k, v, do, 50, 2, scale, None)


def test_large_scores_first():
    """The largest score comes first, or last: the running maximum falls behind or jumps."""
    for at in (0, 149):
        q, k, v, do = inputs(1, 150, 1, 1, 64, F32, seed=3)
        k[0, at] *= 30
        compare(q, k, v, do, 150, 0, 0.125, None)


def test_dense_rows_are_packed_sequences():
    q, k, v, do = inputs(3, 70, 4, 2, 64, BF, seed=4)
    o, lse = gdn.swa_fwd(q, k, v, 20, sinks=2, scale=0.1, return_lse=True)
    got = gdn.swa_bwd(q, k, v, o, lse, do, 20, sinks=2, scale=0.1)
    flat = lambda t: t.reshape(1, 210, *t.shape[2:])  # noqa: E731
    cu = [0, 70, 140, 210]
    o2, lse2 = gdn.swa_fwd(flat(q), flat(k), flat(v), 20, sinks=2, scale=0.1, cu_seqlens=cu, return_lse=True)
    got2 = gdn.swa_bwd(flat(q), flat(k), flat(v), o2, lse2, flat(do), 20, sinks=2, scale=0.1, cu_seqlens=cu)
    assert torch.equal(flat(o), o2) and torch.equal(flat(lse), lse2)
    for key in got:
        assert torch.equal(flat(got[key]), got2[key]), key


def test_empty():
    for B, T, cu in ((0, 5, None), (2, 0, None), (1, 0, [0]), (1, 0, [0, 0, 0])):
        q, k, v, do = inputs(B, T, 2, 1, 64, BF)
        o, lse = gdn.swa_fwd(q, k, v, 4, sinks=1, cu_seqlens=cu, return_lse=True)
        got = gdn.swa_bwd(q, k, v, o, lse, do, 4, sinks=1, cu_seqlens=cu)
        assert o.shape == q.shape and got["dk"].shape == k.shape


def test_gradients_against_differences():
    """The fp32 chain against central differences of its own forward: step 2^-6, whose square
    times a third derivative stays below 1e-3 here; roundings of 200 2^-24 sum |o do| over the step."""
    q, k, v, do = inputs(1, 20, 2, 1, 64, F32, seed=5)
    how = dict(sinks=2, scale=0.125)
    o, lse = gdn.swa_fwd(q, k, v, 6, return_lse=True, **how)
    got = gdn.swa_bwd(q, k, v, o, lse, do, 6, **how)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        for j in (0, 65, 999):
            vals = []
            for sign in (1, -1):
                w = [x.clone() for x in (q, k, v)]
                w[("dq", "dk", "dv").index(name)].view(-1)[j] += sign * 2.0 ** -6
                vals.append(float((gdn.swa_fwd(*w, 6, **how).double() * do).sum()))
            assert abs((vals[0] - vals[1]) * 32 - float(got[name].view(-1)[j])) <= 5e-3, name


def test_infinite_scores_are_nan_in_their_row_alone():
    q, k, v, _ = inputs(1, 100, 1, 1, 64, F32, seed=6)
    clean = gdn.swa_fwd(q, k, v, 30)
    q[0, 40, 0, 3] = math.inf
    o = gdn.swa_fwd(q, k, v, 30)
    assert (~torch.isfinite(o)).any(-1).nonzero()[:, 1].unique().tolist() == [40]
    assert torch.equal(o[:, :40], clean[:, :40]) and torch.equal(o[:, 41:], clean[:, 41:])


MANY = [(64, 150, 8, 8, 64, 40, 3), (64, 150, 8, 1, 128, 60, 0), (16, 530, 16, 2, 64, 100, 20), (8, 300, 64, 64, 128, 140, 2)]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hk,D,W,S", MANY)
def test_many_sequences_and_heads(B, T, Hq, Hk, D, W, S, io):
    """More blocks than the CUs take at once, of queries and of keys: the wider tiles."""
    q, k, v, do = inputs(B, T, Hq, Hk, D, io, seed=7)
    compare(q, k, v, do, W, S, D ** -0.5, None)


def _seen(B, T, W, S, cu):
    """[rows, rows]: which query sees which key, over the flattened tokens."""
    m = torch.zeros(B * T, B * T, dtype=torch.bool, device=DEV)
    for a, b in ref.spans(B, T, cu):
        m[a:b, a:b] = ref.seen(b - a, W, S).to(DEV)
    return m


ODD = [  # B, T, Hq, Hk, D, W, S, cu
    (1, 300, 2, 1, 64, 100, 3, None),
    (1, 420, 2, 2, 128, 33, 20, None),
    (1, 333, 4, 2, 64, 40, 3, [0, 0, 1, 65, 193, 193, 332, 333, 333]),
    (16, 130, 32, 32, 64, 48, 2, None),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("B,T,Hq,Hk,D,W,S,cu", ODD)
def test_values_that_are_not_finite_stay_where_they_are_seen(B, T, Hq, Hk, D, W, S, cu, bad, io):
    """In one row of q, k, v or do, at several places: who does not see it keeps its result
    (within the bounds of the finite problem), and who sees a NaN has NaN."""
    q, k, v, do = inputs(B, T, Hq, Hk, D, io, seed=8)
    how = dict(sinks=S, scale=D ** -0.5, cu_seqlens=cu)
    want, err = ref.swa(q, k, v, W, S, D ** -0.5, cu, do)
    see, group, rows = _seen(B, T, W, S, cu), Hq // Hk, B * T
    for name in "qkvd":
        for at in (0, 1, 40, rows // 2, rows - 1):
            t = {n: x.clone() for n, x in zip("qkvd", (q, k, v, do))}
            h, d = (Hq if name in "qd" else Hk) - 1, 5
            t[name].view(rows, -1, D)[at, h, d] = bad
            heads = slice(Hq - 1, Hq) if name in "qd" else slice(Hq - group, Hq)
            queries = torch.zeros(rows, Hq, dtype=torch.bool, device=DEV)  # whose probabilities or delta it reaches
            queries[:, heads] = (torch.arange(rows, device=DEV) == at if name in "qd" else see[:, at])[:, None]
            keys = torch.stack([(see & queries[:, i * group:(i + 1) * group].any(1)[:, None]).any(0) for i in range(Hk)], 1)
            one = torch.arange(D, device=DEV) == d
            every = torch.ones_like(one)
            reach = {"o": queries[..., None] & {"q": every, "k": every, "v": one, "d": ~every}[name],
                     "lse": queries if name in "qk" else torch.zeros_like(queries),
                     "dq": queries[..., None] & every, "dk": keys[..., None] & every,
                     "dv": keys[..., None] & {"q": every, "k": every, "v": ~every, "d": one}[name]}
            o, lse = gdn.swa_fwd(t["q"], t["k"], t["v"], W, return_lse=True, **how)
            got = gdn.swa_bwd(t["q"], t["k"], t["v"], o, lse, t["d"], W, **how)
            got.update(o=o, lse=lse)
            torch.cuda.synchronize()
            for key, r in reach.items():
                x, r = got[key], r.view(got[key].shape)
                if math.isnan(bad):
                    assert bool(torch.isnan(x[r]).all()), (name, at, key)
                ref.check(f"{name}[{at}] {key}", torch.where(r, torch.zeros_like(x), x),
                          want[key].masked_fill(r.cpu(), 0), err[key])


@pytest.mark.parametrize("io", [BF, F32])
def test_one_long_sequence_beside_many_short_ones(io):
    """Two thousand sequences of a token or none around one of four thousand tokens: heads that
    share nothing, of which two are looked at."""
    before, long, behind, W, S = 1500, 4096, 600, 100, 3
    lens = [i % 2 for i in range(before)] + [long] + [1] * behind
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v, do = inputs(1, cu[-1], 64, 64, 64, io, seed=10)
    seqs, how = gdn.SeqLens(cu, torch.device(DEV)), dict(sinks=S, scale=0.125)
    o, lse = gdn.swa_fwd(q, k, v, W, cu_seqlens=seqs, return_lse=True, **how)
    got = dict(gdn.swa_bwd(q, k, v, o, lse, do, W, cu_seqlens=seqs, **how), o=o, lse=lse)
    caches = [torch.full((len(lens), S + W, 64, 64), 7.0, device=DEV, dtype=io) for _ in range(2)]
    gdn.swa_fill(k, v, *caches, sinks=S, cu_seqlens=seqs)
    assert torch.equal(caches[0][before, :S], k[0, cu[before]:cu[before] + S]) and torch.equal(caches[1][-1, 0], v[0, -1])
    for h in (0, 63):
        want, err = ref.swa(*(t[:, :, h:h + 1] for t in (q, k, v)), W, S, 0.125, cu, do[:, :, h:h + 1])
        for key in got:
            ref.check(f"{key} of head {h}", got[key][:, :, h:h + 1], want[key], err[key])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("N", [63, 64, 65, 4095, 4097, 5000])
def test_thousands_of_sequences(N, io):
    """Every number of sequences finds its blocks, empty sequences among them."""
    lens = torch.randint(0, 3, (N,), generator=torch.Generator().manual_seed(N))
    lens[::501] = 70
    cu = [0] + lens.cumsum(0).tolist()
    q, k, v, do = inputs(1, cu[-1], 2, 1, 64, io, seed=11)
    compare(q, k, v, do, 9, 2, 0.125, cu)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
@pytest.mark.parametrize("B,T,Hq,Hk,D,W,S,cu", ODD)
def test_infinities_reach_those_that_see_them(B, T, Hq, Hk, D, W, S, cu, bad, io):
    """Where the definition leaves no finite result, there is none: an infinite v gives its column of
    o, an infinite q or a score of plus infinity the row of o and lse, an infinite do its column of dv;
    delta is not finite then, and with it dq, and dk of all keys that are seen.  (Left out: scores of
    minus infinity, whose probability is zero.)"""
    q, k, v, do = inputs(B, T, Hq, Hk, D, io, seed=8)
    how = dict(sinks=S, scale=D ** -0.5, cu_seqlens=cu)
    see, group, rows, d = _seen(B, T, W, S, cu), Hq // Hk, B * T, 5
    for name in "qkvd":
        for at in (0, 1, 40, rows // 2, rows - 1):
            t = {n: x.clone() for n, x in zip("qkvd", (q, k, v, do))}
            h = (Hq if name in "qd" else Hk) - 1
            t[name].view(rows, -1, D)[at, h, d] = bad
            heads = slice(Hq - 1, Hq) if name in "qd" else slice(Hq - group, Hq)
            hit = torch.zeros(rows, Hq, dtype=torch.bool, device=DEV)  # queries whose result is not finite
            hit[:, heads] = (torch.arange(rows, device=DEV) == at if name in "qd" else see[:, at])[:, None]
            if name == "k":
                hit &= q.view(rows, Hq, D)[..., d].float() * bad > 0
            keys = torch.stack([(see & hit[:, i * group:(i + 1) * group].any(1)[:, None]).any(0) for i in range(Hk)], 1)
            o, lse = gdn.swa_fwd(t["q"], t["k"], t["v"], W, return_lse=True, **how)
            got = gdn.swa_bwd(t["q"], t["k"], t["v"], o, lse, t["d"], W, **how)
            fine = {key: torch.isfinite(x.view(rows, *x.shape[2:])) for key, x in dict(got, o=o, lse=lse).items()}
            torch.cuda.synchronize()
            if name in "qk":
                assert not bool(fine["o"][hit].any()) and not bool(fine["lse"][hit].any()), (name, at)
            elif name == "v":
                assert not bool(fine["o"][..., d][hit].any()), (name, at)
            else:
                assert not bool(fine["dv"][..., d][keys].any()), (name, at)
            assert not bool(fine["dq"][hit].any()) and not bool(fine["dk"][keys].any()), (name, at)


@pytest.mark.parametrize("io,D", [(BF, 64), (BF, 128), (F32, 128)])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, -4.0])
def test_scales_of_both_signs(scale, D, io):
    """In both types and widths; a negative scale turns the forward's queries."""
    q, k, v, do = inputs(1, 150, 2, 1, D, io, seed=2)
    compare(q, k, v, do, 50, 2, scale, None)


def test_more_workgroups_than_an_axis_of_the_grid():
    """65535 sequences of one token and 70 heads, 4.6 million blocks: a token that sees itself alone
    has its value for a result, and do for dv, exactly."""
    N, H, D = 65535, 70, 64
    q, k, v, do = inputs(1, N, H, H, D, BF, seed=12)
    seqs = gdn.SeqLens(list(range(N + 1)), torch.device(DEV))
    o, lse = gdn.swa_fwd(q, k, v, 5, sinks=2, scale=0.125, cu_seqlens=seqs, return_lse=True)
    got = gdn.swa_bwd(q, k, v, o, lse, do, 5, sinks=2, scale=0.125, cu_seqlens=seqs)
    assert torch.equal(o, v) and torch.equal(got["dv"], do)
    # D products of absolute terms up to 6^2 and their sum; both sides' roundings
    assert float((lse - (q.float() * k.float()).sum(-1) * 0.125).abs().max()) <= 2 * 64 * 67 * 36 * 0.125 * 2.0 ** -24
    assert bool(torch.isfinite(got["dq"]).all()) and bool(torch.isfinite(got["dk"]).all())
