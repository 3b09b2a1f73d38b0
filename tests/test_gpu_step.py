"""gdn_step and gdn_kda_step (one token, state in place) against their float64
definition, the token-loop reference, and under graph replay (marked gpu)."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(B, H, Dk, Dv, io, channel, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(io)  # noqa: E731
    g = -torch.nn.functional.softplus(r(B, 1, H, Dk) if channel else r(B, 1, H))
    return dict(q=unit(r(B, 1, H, Dk)), k=unit(r(B, 1, H, Dk)), v=r(B, 1, H, Dv).to(io), g=g,
                beta=2 * torch.sigmoid(r(B, 1, H))), 0.3 * r(B, H, Dk, Dv)


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,Dk,Dv", [(1, 1, 64, 16), (1, 8, 128, 128), (3, 5, 64, 80), (2, 3, 128, 256), (17, 2, 128, 48),
                                       (64, 10, 128, 112), (300, 9, 64, 80)])  # the last two: states past the caches (32 MB)
def test_step(B, H, Dk, Dv, io, channel):
    t, S = _inputs(B, H, Dk, Dv, io, channel)
    o_ref, S_ref = ref.delta_step(**t, S=S, scale=0.7)
    o_size, S_size = ref.delta_step(**t, S=S, scale=0.7, size=True)
    room = torch.full((v_rows := B + 2, 1, H, Dv), 7.0, device=DEV, dtype=io)  # a row on either side of the output
    o = (gdn.kda_step if channel else gdn.step)(**t, state=S, scale=0.7, out=room[1:B + 1])
    torch.cuda.synchronize()
    assert o.data_ptr() == room[1].data_ptr()
    assert bool((room[0] == 7).all()) and bool((room[v_rows - 1] == 7).all())
    # per term: the decay (expf), Dk additions in each sum, the error, the write, the read
    ref.check("o", o, o_ref, o_size, 2 * Dk + 64)
    ref.check("S", S, S_ref, S_size, 2 * Dk + 64)


@pytest.mark.parametrize("channel", [False, True])
def test_steps_follow_the_prompt(channel):
    """Prompt with the chunked forward, then tokens one at a time, in fp32: the same as
    one longer prompt (both within the chunked forward's 3e-4 of the definition)."""
    B, T, H, Dk, Dv = 2, 70, 3, 64, 64
    gen = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(r(B, T, H, Dk)), unit(r(B, T, H, Dk)), r(B, T, H, Dv)
    g = -0.3 * torch.nn.functional.softplus(r(B, T, H, Dk) if channel else r(B, T, H))
    beta = torch.sigmoid(r(B, T, H))
    fwd, step = (gdn.kda_chunk_fwd, gdn.kda_step) if channel else (gdn.chunk_fwd, gdn.step)
    o_all, S_all = fwd(q, k, v, g, beta, scale=0.5)
    cut = 64
    head = [t[:, :cut].contiguous() for t in (q, k, v, g, beta)]
    _, S = fwd(*head, scale=0.5)
    for t in range(cut, T):
        o = step(*(x[:, t:t + 1].contiguous() for x in (q, k, v, g, beta)), state=S, scale=0.5)
        worst = float((o - o_all[:, t:t + 1]).abs().max() / o_all.abs().max())
        assert worst <= 6e-4, (t, worst)
    assert float((S - S_all).abs().max() / S_all.abs().max()) <= 6e-4


def test_extreme_gates():
    t, S = _inputs(2, 2, 64, 64, torch.float32, True)
    t["g"][0] = float("-inf")  # forget everything: S = k e^T alone
    t["g"][1] = 0.0            # forget nothing
    o_ref, S_ref = ref.delta_step(**t, S=S, scale=1.0)
    o_size, S_size = ref.delta_step(**t, S=S, scale=1.0, size=True)
    o = gdn.kda_step(**t, state=S)
    ref.check("o", o, o_ref, o_size, 192)
    ref.check("S", S, S_ref, S_size, 192)


def test_no_sequences():
    t, S = _inputs(0, 2, 64, 64, torch.float32, False)
    assert gdn.step(**t, state=S).shape == (0, 1, 2, 64)


def test_graph_replays_match_eager_calls():
    t, S = _inputs(3, 4, 128, 128, torch.bfloat16, False)
    out = torch.empty_like(t["v"])
    start = S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.step(**t, state=S, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    S.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.step(**t, state=S, out=out)
    eager = start.clone()
    for rep in range(4):
        fresh, _ = _inputs(3, 4, 128, 128, torch.bfloat16, False, seed=50 + rep)
        for key in t:
            t[key].copy_(fresh[key])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        o = gdn.step(**fresh, state=eager)
        assert torch.equal(out, o) and torch.equal(S, eager), rep
