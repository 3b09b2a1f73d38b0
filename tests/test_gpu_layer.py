"""The layer operators together, as a layer uses them (marked gpu): prompt and single
tokens of a delta-rule layer and of a state space layer, a training step through both
operators, graph replays, and calls on other streams."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("channel", [False, True])
def test_delta_rule_layer_prompt_then_tokens(channel):
    """conv -> prologue -> chunked delta rule -> epilogue over a prompt, then conv_step ->
    prologue -> step -> epilogue: the same as the longer prompt (fp32; the chunked
    forward is within 3e-4 of the recurrence, and the epilogue's norm does not enlarge
    it beyond twice that)."""
    B, T, n, H, D = 2, 70, 5, 2, 64
    g = _gen(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    C = 3 * H * D
    x, z = r(B, T + n, C), r(B, T + n, H, D)
    a = r(B, T + n, H, D) if channel else r(B, T + n, H)
    b = r(B, T + n, H)
    w, bias = 0.5 * r(C, 4), 0.1 * r(C)
    A_log, dt_bias = r(H).abs(), r(H, D) if channel else r(H)
    fwd, step = (gdn.kda_chunk_fwd, gdn.kda_step) if channel else (gdn.chunk_fwd, gdn.step)

    def inputs(y, s):
        q, k, v = (t.reshape(B, -1, H, D).contiguous() for t in y.split(H * D, dim=2))
        q, k, gate, beta = gdn.prologue(q, k, a[:, s].contiguous(), b[:, s].contiguous(), A_log=A_log, dt_bias=dt_bias,
                                        gate="gdn_channel" if channel else "gdn")
        return q, k, v, gate, beta

    whole, rows = gdn.conv_fwd(x, w, bias=bias)
    o, S_all = fwd(*inputs(whole, slice(0, T + n)), scale=D ** -0.5)
    y_all = gdn.epilogue(o, z)

    head, state = gdn.conv_fwd(x[:, :T].contiguous(), w, bias=bias)
    _, S = fwd(*inputs(head, slice(0, T)), scale=D ** -0.5)
    for t in range(T, T + n):
        s = slice(t, t + 1)
        yt = gdn.conv_step(x[:, s].contiguous(), w, state, bias=bias)
        assert torch.equal(yt, whole[:, s])
        ot = step(*inputs(yt, s), state=S, scale=D ** -0.5)
        y = gdn.epilogue(ot, z[:, s].contiguous())
        assert float((y - y_all[:, s]).abs().max() / y_all.abs().max()) <= 1.2e-3, t
    assert torch.equal(state, rows)
    assert float((S - S_all).abs().max() / S_all.abs().max()) <= 6e-4


def _ssm_inputs(B, T, D, N, seed, io=torch.float32):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=r(B, T, D).to(io), w=0.5 * r(D, 4), b=0.1 * r(D), dt=r(B, T, D).to(io), A=-(0.1 + torch.rand(D, N, generator=g, device=DEV)),
                Bm=r(B, T, 1, N).to(io), Cm=r(B, T, 1, N).to(io), D=r(D), z=r(B, T, D).to(io), dt_bias=r(D) - 2)


_SCAN = ("dt", "A", "Bm", "Cm", "D", "z", "dt_bias")


def test_state_space_layer_prompt_then_tokens():
    """conv -> scan over a prompt, then conv_step -> scan_step, against the longer prompt
    (fp32: 3 (T + n) + 80 roundings a term, as the scan's own test counts them)."""
    B, T, n, D, N = 2, 40, 6, 72, 16
    a = _ssm_inputs(B, T + n, D, N, 2)
    u_all, rows = gdn.conv_fwd(a["x"], a["w"], bias=a["b"])
    y_all, h_all = gdn.scan_fwd(u_all, **{k: a[k] for k in _SCAN})
    size = ref.scan(u_all, a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], a["dt_bias"], None, None, True, size=True)
    cut = lambda s: {k: (a[k][:, s].contiguous() if a[k].dim() > 2 else a[k]) for k in _SCAN}  # noqa: E731
    u, state = gdn.conv_fwd(a["x"][:, :T].contiguous(), a["w"], bias=a["b"])
    y, h = gdn.scan_fwd(u, **cut(slice(0, T)))
    ref.check("prompt", y, y_all[:, :T].double().cpu(), size["y"][:, :T], 6 * T + 160)
    for t in range(T, T + n):
        s = slice(t, t + 1)
        u = gdn.conv_step(a["x"][:, s].contiguous(), a["w"], state, bias=a["b"])
        y = gdn.scan_step(u, state=h, **cut(s))
        ref.check(f"token {t}", y, y_all[:, s].double().cpu(), size["y"][:, s], 2 * (3 * (T + n) + 80))
    assert torch.equal(state, rows)
    ref.check("state", h, h_all.double().cpu(), size["state"], 2 * (3 * (T + n) + 80))


def test_training_step_through_both_operators():
    """Gradients of <y, dy> of conv -> scan for the convolution's input and parameters
    and the scan's, against reverse mode through the float64 definitions."""
    B, T, D, N = 2, 30, 64, 16
    a = _ssm_inputs(B, T, D, N, 3)
    dy = torch.randn(B, T, D, generator=_gen(4), device=DEV)
    u, _ = gdn.conv_fwd(a["x"], a["w"], bias=a["b"])
    scan = {k: a[k] for k in _SCAN}
    _, _, saved = gdn.scan_fwd_save(u, **scan)
    gs = gdn.scan_bwd_saved(u, dy=dy, saved=saved, **scan)
    gc = gdn.conv_bwd(a["x"], a["w"], gs["du"], bias=a["b"])

    leaf = {k: v.double().cpu().requires_grad_() for k, v in a.items()}
    uu, _ = ref.conv(leaf["x"], leaf["w"], leaf["b"], None, None, True)
    delta = torch.nn.functional.softplus(leaf["dt"] + leaf["dt_bias"], threshold=100)
    h = torch.zeros(B, D, N, dtype=torch.float64)
    loss = 0.0
    for t in range(T):
        d = delta[:, t].unsqueeze(-1)
        h = torch.exp(d * leaf["A"]) * h + d * uu[:, t].unsqueeze(-1) * leaf["Bm"][:, t]
        s = (h * leaf["Cm"][:, t]).sum(-1) + leaf["D"] * uu[:, t]
        loss = loss + (s * torch.nn.functional.silu(leaf["z"][:, t]) * dy[:, t].double().cpu()).sum()
    loss.backward()
    got = dict(x=gc["dx"], w=gc["dweight"], b=gc["dbias"], dt=gs["ddt"], A=gs["dA"], Bm=gs["dB"], Cm=gs["dC"], D=gs["dD"],
               z=gs["dz"], dt_bias=gs["ddt_bias"])
    for k, v in got.items():
        want = leaf[k].grad
        # in the norm: no term cancels to less than a thousandth of its size there
        assert float((v.double().cpu() - want).norm() / want.norm()) <= 1000 * 2 ** -24, k


def test_packed_prompts_are_each_alone():
    cu = [0, 0, 1, 2, 17, 49, 60]
    a = _ssm_inputs(1, 60, 64, 16, 5, torch.bfloat16)
    u, rows = gdn.conv_fwd(a["x"], a["w"], bias=a["b"], cu_seqlens=cu)
    y, h = gdn.scan_fwd(u, **{k: a[k] for k in _SCAN}, cu_seqlens=cu)
    for n in range(6):
        s = slice(cu[n], cu[n + 1])
        part = {k: (v[:, s].contiguous() if v.dim() > 2 else v) for k, v in a.items()}
        u1, r1 = gdn.conv_fwd(part["x"], a["w"], bias=a["b"])
        y1, h1 = gdn.scan_fwd(u1, **{k: part[k] for k in _SCAN})
        assert torch.equal(u1, u[:, s]) and torch.equal(r1[0], rows[n])
        assert torch.equal(y1, y[:, s]) and torch.equal(h1[0], h[n])


def _training(a, dy):
    u, rows = gdn.conv_fwd(a["x"], a["w"], bias=a["b"])
    scan = {k: a[k] for k in _SCAN}
    y, h, saved = gdn.scan_fwd_save(u, **scan)
    gs = gdn.scan_bwd_saved(u, dy=dy, saved=saved, **scan)
    gc = gdn.conv_bwd(a["x"], a["w"], gs["du"], bias=a["b"])
    return {"u": u, "rows": rows, "y": y, "h": h, **gs, **{"conv_" + k: v for k, v in gc.items()}}


@pytest.mark.parametrize("B,T,D", [(2, 100, 64), (1, 700, 72)])
def test_captured_training_step_replays(B, T, D):
    a = _ssm_inputs(B, T, D, 16, 6, torch.bfloat16)
    dy = torch.randn(B, T, D, generator=_gen(7), device=DEV).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _training(a, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _training(a, dy)
    for rep in range(4):
        fresh = _ssm_inputs(B, T, D, 16, 60 + rep, torch.bfloat16)
        for k in a:
            a[k].copy_(fresh[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items() if v is not None}
        want = _training(fresh, dy)
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], want[k]), (rep, k)


def test_captured_decoding_replays():
    """One token of conv -> scan in a graph, states carried from replay to replay."""
    B, D, N = 3, 64, 16
    a = _ssm_inputs(B, 1, D, N, 8, torch.bfloat16)
    rows = torch.zeros(B, 3, D, device=DEV, dtype=torch.bfloat16)
    h = torch.zeros(B, D, N, device=DEV)

    def token(a, rows, h):
        u = gdn.conv_step(a["x"], a["w"], rows, bias=a["b"])
        return gdn.scan_step(u, state=h, **{k: a[k] for k in _SCAN})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(a, rows, h)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    rows.zero_()
    h.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(a, rows, h)
    rows2, h2 = torch.zeros_like(rows), torch.zeros_like(h)
    for rep in range(5):
        fresh = _ssm_inputs(B, 1, D, N, 80 + rep, torch.bfloat16)
        for k in a:
            a[k].copy_(fresh[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = token(fresh, rows2, h2)
        assert torch.equal(out, want) and torch.equal(rows, rows2) and torch.equal(h, h2), rep


def test_calls_on_two_streams_at_once():
    """Each call has its own workspace: two training steps on two streams give what each
    gives alone."""
    a = [_ssm_inputs(1, 700, 72, 16, 20 + i, torch.bfloat16) for i in range(2)]
    dy = torch.randn(1, 700, 72, generator=_gen(9), device=DEV).bfloat16()
    alone = [_training(x, dy) for x in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            both[i] = _training(a[i], dy)
    torch.cuda.synchronize()
    for i in range(2):
        for k, v in alone[i].items():
            assert v is None or torch.equal(v, both[i][k]), (i, k)


def test_wrong_arguments_are_refused():
    a = _ssm_inputs(1, 4, 64, 16, 30)
    x, w = a["x"], a["w"]
    with pytest.raises(ValueError, match="contiguous"):
        gdn.conv_fwd(torch.zeros(1, 64, 4, device=DEV).transpose(1, 2), w)
    with pytest.raises(TypeError, match="weight"):
        gdn.conv_fwd(x, w.half())
    with pytest.raises(ValueError, match="state0"):
        gdn.conv_fwd(x, w, state0=torch.zeros(1, 4, 64, device=DEV))
    with pytest.raises(ValueError, match="activation"):
        gdn.conv_fwd(x, w, activation="gelu")
    with pytest.raises(ValueError, match="x must be"):
        gdn.conv_step(x, w, torch.zeros(1, 3, 64, device=DEV))
    with pytest.raises(gdn.GdnError):
        gdn.conv_fwd(x, torch.zeros(64, 5, device=DEV))
    with pytest.raises(ValueError, match="weight must be on"):
        gdn.conv_fwd(x, w.cpu())
    scan = {k: a[k] for k in _SCAN}
    with pytest.raises(TypeError, match="Cm"):
        gdn.scan_fwd(x, **(scan | dict(Cm=a["Cm"].bfloat16())))
    with pytest.raises(ValueError, match="A must be"):
        gdn.scan_fwd(x, **(scan | dict(A=a["A"][:, :8].contiguous())))
    with pytest.raises(ValueError, match="saved"):
        gdn.scan_bwd_saved(x, dy=x, saved=None, **scan)
    with pytest.raises(gdn.GdnError):
        gdn.scan_bwd_saved(x, dy=x, saved=torch.zeros(16, dtype=torch.uint8, device=DEV), **scan)
    with pytest.raises(gdn.GdnError):  # an output over an input
        gdn.scan_fwd(x, **scan, out=x)
    with pytest.raises(ValueError, match="u must be"):
        gdn.scan_step(x, state=torch.zeros(1, 64, 16, device=DEV), **scan)
    q = torch.zeros(1, 2, 1, 64, device=DEV)
    with pytest.raises(ValueError, match="q and k"):
        gdn.step(q, q, q, torch.zeros(1, 2, 1, device=DEV), torch.zeros(1, 2, 1, device=DEV), torch.zeros(1, 1, 64, 64, device=DEV))
