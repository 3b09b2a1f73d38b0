"""Window attention over a cache on the GPU: the filling from prompts and the single-token
step against their float64 definitions, and both continuing a prompt (marked gpu)."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


CASES = [  # Hq, Hk, D, W, S
    (1, 1, 64, 1, 0),
    (4, 2, 128, 7, 3),
    (3, 1, 64, 64, 0),
    (16, 1, 128, 130, 4),
    (20, 1, 64, 33, 2),
    (34, 2, 64, 40, 0),
    (8, 8, 64, 300, 5),
    (4, 1, 128, 1500, 4),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,D,W,S", CASES)
def test_step(Hq, Hk, D, W, S, io):
    lens = [0, 1, S, max(0, S + W - 2), S + W - 1, S + W, S + W + 1, S + 5 * W + 3, -1, 2 ** 31 - 2]
    B = len(lens)
    g = _gen(W)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(io)  # noqa: E731
    rows = r(B, 1, (Hq + 2 * Hk) * D)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in rows.split([Hq * D, Hk * D, Hk * D], dim=-1))
    kc, vc = r(B, S + W, Hk, D), r(B, S + W, Hk, D)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for n, before in enumerate(lens):  # nothing reads a slot that has not been written
        if before >= 0:
            kc[n, before:] = float("nan")
            vc[n, before:] = float("nan")
    want, err, kw, vw = ref.swa_step(q, k, v, kc, vc, at, S, D ** -0.5)
    kc2, vc2 = kc.clone(), vc.clone()
    o = gdn.swa_step(q, k, v, kc, vc, at, sinks=S, scale=D ** -0.5)
    o2 = gdn.swa_step(q, k, v, kc2, vc2, at, sinks=S, scale=D ** -0.5)
    ref.check("o", o, want, err)
    assert float(o[lens.index(-1)].abs().max()) == 0.0
    assert torch.equal(o, o2)
    for got, expected in ((kc, kw), (vc, vw)):
        assert torch.equal(got.nan_to_num(-9).double().cpu(), expected.nan_to_num(-9))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("W,S,cu", [(5, 2, [0, 0, 1, 3, 6, 7, 15, 16, 40]), (1, 0, [0, 2, 3]), (64, 70, [0, 30, 170, 400])])
def test_fill(W, S, cu, io):
    g = _gen(1)
    T, Hk, D = cu[-1], 2, 64
    rows = torch.randn(1, T, 3 * Hk * D, generator=g, device=DEV).to(io)
    k, v = rows[..., :Hk * D].unflatten(-1, (Hk, D)), rows[..., 2 * Hk * D:].unflatten(-1, (Hk, D))
    n = len(cu) - 1
    kc, vc = (torch.full((n, S + W, Hk, D), 7.0, device=DEV, dtype=io) for _ in range(2))
    gdn.swa_fill(k, v, kc, vc, sinks=S, cu_seqlens=cu)
    for cache, x in ((kc, k), (vc, v)):
        want = torch.full_like(cache, 7.0)
        for i in range(n):
            for t in range(cu[i + 1] - cu[i]):
                want[i, ref.slot_of(t, W, S)] = x[0, cu[i] + t]
        assert torch.equal(cache, want)


@pytest.mark.parametrize("W,S", [(9, 0), (9, 3), (200, 4)])
def test_prompt_then_tokens(W, S):
    """swa_fwd and swa_fill over a prompt, then swa_step, against the longer prompt: both are
    within their bounds of the definition."""
    B, T, n, Hq, Hk, D = 2, 50, 12, 4, 2, 64
    g = _gen(2)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v = r(B, T + n, Hq, D), r(B, T + n, Hk, D), r(B, T + n, Hk, D)
    want, err = ref.swa(q, k, v, W, S, 0.125, None)
    whole = gdn.swa_fwd(q, k, v, W, sinks=S, scale=0.125)
    kc, vc = (torch.full((B, S + W, Hk, D), float("nan"), device=DEV) for _ in range(2))
    head = [t[:, :T].contiguous() for t in (q, k, v)]
    o = gdn.swa_fwd(*head, W, sinks=S, scale=0.125)
    assert torch.equal(o, whole[:, :T])
    gdn.swa_fill(*head[1:], kc, vc, sinks=S)
    lens = torch.full((B,), T, dtype=torch.int32, device=DEV)
    for t in range(T, T + n):
        o = gdn.swa_step(*(x[:, t:t + 1].contiguous() for x in (q, k, v)), kc, vc, lens, sinks=S, scale=0.125)
        ref.check(f"token {t}", o, want["o"][:, t:t + 1], err["o"][:, t:t + 1])
        ref.check(f"row {t}", whole[:, t:t + 1], want["o"][:, t:t + 1], err["o"][:, t:t + 1])
        lens += 1


def test_runs_are_joined_and_workspaces_taken():
    """One sequence with many slots: several runs, a caller's workspace, and the same bits."""
    g = _gen(3)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    q, k, v, kc, vc = r(1, 1, 4, 128), r(1, 1, 1, 128), r(1, 1, 1, 128), r(1, 4100, 1, 128), r(1, 4100, 1, 128)
    for before in (0, 3, 100, 700, 4099, 4100, 100000):
        lens = torch.tensor([before], dtype=torch.int32, device=DEV)
        want, err, _, _ = ref.swa_step(q, k, v, kc, vc, lens, 4, 0.09)
        o = gdn.swa_step(q, k, v, kc, vc, lens, sinks=4, scale=0.09)
        ref.check(f"o {before}", o, want, err)
        space = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
        assert torch.equal(gdn.swa_step(q, k, v, kc, vc, lens, sinks=4, scale=0.09, workspace=space), o)


@pytest.mark.parametrize("Hq,Hk,D,W,S", [(4, 1, 64, 300, 5), (16, 4, 128, 130, 0), (4, 1, 128, 1500, 4)])
def test_probabilities_keep_sixteen_bits(Hq, Hk, D, W, S):
    """In bf16 a probability enters its product as its rounding and the rounding of what that leaves:
    2^-8 of 2^-8, so 2^-16 of each term beside the fp32 bounds and the result's own rounding."""
    lens = [1, W // 2, S + W, S + 3 * W + 1]
    g = _gen(W)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    B = len(lens)
    q, k, v, kc, vc = r(B, 1, Hq, D), r(B, 1, Hk, D), r(B, 1, Hk, D), r(B, S + W, Hk, D), r(B, S + W, Hk, D)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    wide = [t.float() for t in (q, k, v, kc, vc)]
    want, err, _, _ = ref.swa_step(*wide, at, S, D ** -0.5)
    terms, _, _, _ = ref.swa_step(wide[0], wide[1], wide[2].abs(), wide[3], wide[4].abs(), at, S, D ** -0.5)
    o = gdn.swa_step(q, k, v, kc, vc, at, sinks=S, scale=D ** -0.5)
    ref.check("o", o, want, err + 2.0 ** -16 * terms)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.1, -2.0])
@pytest.mark.parametrize("W", [40, 1500])
def test_scales_of_both_signs(W, scale, io):
    """None, and negative ones, in one run of slots and in several."""
    Hq, Hk, D, S, lens = 4, 1, 128, 3, [0, 20, W + 2, 5 * W]
    g = _gen(W)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(io)  # noqa: E731
    B = len(lens)
    q, k, v, kc, vc = r(B, 1, Hq, D), r(B, 1, Hk, D), r(B, 1, Hk, D), r(B, S + W, Hk, D), r(B, S + W, Hk, D)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, err, _, _ = ref.swa_step(q, k, v, kc, vc, at, S, scale)
    ref.check("o", gdn.swa_step(q, k, v, kc, vc, at, sinks=S, scale=scale), want, err)
