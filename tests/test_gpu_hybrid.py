"""The hybrid models' operators together, as a layer's training step and as decoding use them,
and captured in graphs and on several streams (marked gpu)."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
HQ, HK, D, W, S, R = 4, 2, 64, 24, 3, 32
C = HQ * D


def rand(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, io=F32: torch.randn(*s, generator=g, device=DEV).to(io)


def weights(r):
    freq = 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=F32) / (R // 2))
    return dict(inv_freq=freq, wq=1 + 0.1 * r(D), wk=1 + 0.1 * r(D)), r(C)


def split(rows):
    q, k, v = rows.split([HQ * D, HK * D, HK * D], dim=-1)
    return tuple(t.unflatten(-1, (-1, D)) for t in (q, k, v))


@pytest.mark.parametrize("io", [BF, F32])
def test_prompts_then_tokens(io):
    """Ragged prompts through rotation, attention and recurrence, then tokens one by one through
    the caches: each step's result is the definition's for the longer sequence."""
    lens, more = [5, 1, 40, 27], 60
    r = rand(1)
    how, lam = weights(r)
    rows = [r(1, n + more, (HQ + 2 * HK) * D, io=io) for n in lens]
    gates = [[r(1, n + more, C, io=io) for _ in range(3)] for n in lens]
    rot = []
    for x in rows:
        q, k, v = split(x)
        rot.append((*gdn.rope_fwd(q, k, **how), v))
    # prompts, packed
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    seqs = gdn.SeqLens(cu, torch.device(DEV))
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV, torch.int32)[None]
    prompt = torch.cat([x[:, :n] for x, n in zip(rows, lens)], 1)
    q, k, v = split(prompt)
    q, k = gdn.rope_fwd(q, k, positions=pos, **how)
    for n, (rq, rk, _) in enumerate(rot):
        assert torch.equal(q[:, cu[n]:cu[n + 1]], rq[:, :lens[n]]) and torch.equal(k[:, cu[n]:cu[n + 1]], rk[:, :lens[n]])
    o = gdn.swa_fwd(q, k, v, W, sinks=S, scale=0.125, cu_seqlens=seqs)
    caches = [torch.full((len(lens), S + W, HK, D), float("nan"), device=DEV, dtype=io) for _ in range(2)]
    gdn.swa_fill(k, v, *caches, sinks=S, cu_seqlens=seqs)
    packed = [torch.cat([g[i][:, :n] for g, n in zip(gates, lens)], 1) for i in range(3)]
    y, state = gdn.glr_fwd(*packed, lam, cu_seqlens=seqs)
    outs, ys = [o], [y]
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for t in range(more):
        now = torch.cat([x[:, n + t:n + t + 1] for x, n in zip(rows, lens)])
        q, k, v = split(now)
        q, k = gdn.rope_fwd(q, k, positions=at[:, None], **how)
        for n, (rq, rk, _) in enumerate(rot):
            assert torch.equal(q[n, 0], rq[0, lens[n] + t]) and torch.equal(k[n, 0], rk[0, lens[n] + t])
        outs.append(gdn.swa_step(q, k, v, *caches, at, sinks=S, scale=0.125))
        g = [torch.cat([g[i][:, n + t:n + t + 1] for g, n in zip(gates, lens)]) for i in range(3)]
        ys.append(gdn.glr_step(*g, lam, state))
        at += 1
    for n, L in enumerate(lens):
        def whole(parts):
            return torch.cat([parts[0][:, cu[n]:cu[n + 1]]] + [p[n:n + 1] for p in parts[1:]], 1)
        want, err = ref.swa(*rot[n], W, S, 0.125, None)
        ref.check(f"o of sequence {n}", whole(outs), want["o"], err["o"])
        want, err = ref.glr(*gates[n], lam, None, None, None)
        ref.check(f"y of sequence {n}", whole(ys), want["y"], err["y"])


def chain64(rows, gates, how, lam):
    """The training chain in float64, for autograd: rotation by RMS norm, attention, recurrence."""
    q, k, v = split(rows)
    T = rows.shape[1]

    def turn(x, w):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a = torch.arange(T, dtype=torch.float64)[:, None] * how["inv_freq"].double().cpu()
        c, s = a.cos()[:, None], a.sin()[:, None]
        x1, x2, rest = x[..., :R // 2], x[..., R // 2:R], x[..., R:]
        return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, rest], -1)

    q, k = turn(q, how["wq64"]), turn(k, how["wk64"])
    k, v = (t.repeat_interleave(HQ // HK, 2) for t in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q, k) * 0.125
    p = s.masked_fill(~ref.seen(T, W, S), -torch.inf).softmax(-1)
    x = torch.einsum("bhij,bjhd->bihd", p, v).flatten(2)
    r, i, z = gates
    la = -8 * torch.nn.functional.softplus(lam) * torch.sigmoid(r)
    u = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
    h, out = torch.zeros_like(x[:, 0]), []
    for t in range(T):
        h = la[:, t].exp() * h + u[:, t]
        out.append(h)
    return torch.stack(out, 1) * z * torch.sigmoid(z)


def test_training_step():
    """Gradients of the whole chain against float64's.  Every operator is within some 300 roundings
    of 2^-24 of sums of absolute terms; three forward and three backward, with those sums up to 30
    times their result: 6 300 30 2^-24 < 4e-3 of the largest gradient."""
    r = rand(2)
    how, lam = weights(r)
    rows, gates, dy = r(2, 70, (HQ + 2 * HK) * D), [r(2, 70, C) for _ in range(3)], r(2, 70, C)
    q, k, v = split(rows)
    rq, rk = gdn.rope_fwd(q, k, **how)
    o, lse = gdn.swa_fwd(rq, rk, v, W, sinks=S, scale=0.125, return_lse=True)
    x = o.flatten(2)
    y, _, saved = gdn.glr_fwd_save(x, gates[0], gates[1], lam, z=gates[2])
    g3 = gdn.glr_bwd_saved(x, gates[0], gates[1], lam, dy, saved, z=gates[2])
    g2 = gdn.swa_bwd(rq, rk, v, o, lse, g3["dx"].unflatten(-1, (HQ, D)), W, sinks=S, scale=0.125)
    g1 = gdn.rope_bwd(q, k, dq_out=g2["dq"], dk_out=g2["dk"], **how)
    got = {"rows": torch.cat([t.flatten(2) for t in (g1["dq"], g1["dk"], g2["dv"])], -1), "lam": g3["dlam"], "r": g3["dr"],
           "i": g3["di"], "z": g3["dz"], "wq": g1["dwq"], "wk": g1["dwk"]}
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    leaves = {"rows": leaf(rows), "lam": leaf(lam), "r": leaf(gates[0]), "i": leaf(gates[1]), "z": leaf(gates[2]),
              "wq": leaf(how["wq"]), "wk": leaf(how["wk"])}
    h64 = dict(how, wq64=leaves["wq"], wk64=leaves["wk"])
    want = chain64(leaves["rows"], [leaves[n] for n in "riz"], h64, leaves["lam"])
    assert float((y.double().cpu() - want.detach()).abs().max()) <= 4e-3 * float(want.detach().abs().max())
    for (name, t), g in zip(leaves.items(), torch.autograd.grad((want * dy.double().cpu()).sum(), list(leaves.values()))):
        assert float((got[name].double().cpu() - g).abs().max()) <= 4e-3 * float(g.abs().max()), name


def capture(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    torch.cuda.synchronize()
    return graph, out


@pytest.mark.parametrize("packed", [False, True])
def test_training_step_in_a_graph(packed):
    """Captured once, replayed on other values with eager work between the replays."""
    T = 700  # several segments of the recurrence, queries behind the first tokens' window
    cu = gdn.SeqLens([0, 0, 1, 300, T], torch.device(DEV)) if packed else None
    r = rand(3)
    how, lam = weights(r)
    t = dict(rows=r(1, T, (HQ + 2 * HK) * D, io=BF), r=r(1, T, C, io=BF), i=r(1, T, C, io=BF), dy=r(1, T, C, io=BF))

    def call():
        q, k, v = split(t["rows"])
        rq, rk = gdn.rope_fwd(q, k, **how)
        o, lse = gdn.swa_fwd(rq, rk, v, W, sinks=S, scale=0.125, cu_seqlens=cu, return_lse=True)
        x = o.flatten(2)
        y, h, saved = gdn.glr_fwd_save(x, t["r"], t["i"], lam, cu_seqlens=cu)
        g3 = gdn.glr_bwd_saved(x, t["r"], t["i"], lam, t["dy"], saved, cu_seqlens=cu)
        g2 = gdn.swa_bwd(rq, rk, v, o, lse, g3["dx"].unflatten(-1, (HQ, D)), W, sinks=S, scale=0.125, cu_seqlens=cu)
        g1 = gdn.rope_bwd(q, k, dq_out=g2["dq"], dk_out=g2["dk"], **how)
        return [y, h, *g3.values(), *g2.values(), *g1.values()]

    graph, out = capture(call)
    for rep in range(5):
        for name, x in t.items():
            x.copy_(rand(10 + rep)(*x.shape, io=BF))
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(out, eager)):
            assert a is b or torch.equal(a, b), (rep, n)


def test_decoding_in_a_graph():
    """A step captured once advances its caches, its state and its lengths by each replay."""
    B, r = 5, rand(4)
    how, lam = weights(r)
    t = dict(rows=r(B, 1, (HQ + 2 * HK) * D, io=BF), r=r(B, 1, C, io=BF), i=r(B, 1, C, io=BF))
    long = 1000  # window of several runs of the cache

    def fresh():
        z = rand(5)
        return dict(kc=z(B, S + long, HK, D, io=BF), vc=z(B, S + long, HK, D, io=BF), state=z(B, C),
                    lens=torch.tensor([0, 1, long + 2, 5000, -1], dtype=torch.int32, device=DEV))

    def step(m):
        q, k, v = split(t["rows"])
        rq, rk = gdn.rope_fwd(q, k, positions=m["lens"].clamp(min=0)[:, None], **how)
        o = gdn.swa_step(rq, rk, v, m["kc"], m["vc"], m["lens"], sinks=S, scale=0.125)
        y = gdn.glr_step(o.flatten(2), t["r"], t["i"], lam, m["state"])
        m["lens"] += (m["lens"] >= 0).int()
        return y

    m, e = fresh(), fresh()
    graph, y = capture(lambda: step(m))
    for name, x in fresh().items():  # as before the capture's first run
        m[name].copy_(x)
    for rep in range(6):
        for name, x in t.items():
            x.copy_(rand(20 + rep)(*x.shape, io=BF))
        want = step(e)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), rep
        for name in m:
            assert torch.equal(m[name], e[name]), (rep, name)


def test_two_streams():
    """The same calls at once on two streams, each with its own workspace, and buffers of a
    caller taken again and again: results as one after the other."""
    r = rand(6)
    _, lam = weights(r)
    x = [r(1, 9000, C, io=BF) for _ in range(4)]
    q, k, v = split(r(1, 600, (HQ + 2 * HK) * D, io=BF))
    size = gdn.glr_buffers(x[0])

    def call(bufs):
        y, h, saved = gdn.glr_fwd_save(*x[:3], lam, saved=bufs[0], workspace=bufs[1])
        g = gdn.glr_bwd_saved(*x[:3], lam, x[3], saved, workspace=bufs[2])
        o, lse = gdn.swa_fwd(q, k, v, W, sinks=S, return_lse=True)
        g2 = gdn.swa_bwd(q, k, v, o, lse, q.contiguous(), W, sinks=S)
        return [y, h, g["dx"], g["dlam"], g["dh0"], o, *g2.values()]

    bufs = [[torch.full((size[n],), 0xff, dtype=torch.uint8, device=DEV) for n in ("saved", "forward", "backward")] for _ in range(2)]
    want = call([None, None, None])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, b in zip(streams, bufs):
            with torch.cuda.stream(s):
                got.append(call(b))
        torch.cuda.synchronize()
        for out in got:
            for n, (a, b) in enumerate(zip(out, want)):
                assert torch.equal(a, b), n


def test_refusals_on_the_gpu():
    r = rand(7)
    how, lam = weights(r)
    x = r(1, 4, C, io=BF)
    q, k, v = split(r(2, 4, (HQ + 2 * HK) * D, io=BF))
    cache = [r(2, S + W, HK, D, io=BF) for _ in range(2)]
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    q1, k1, v1 = (t[:, :1] for t in (q, k, v))
    bad = [
        (ValueError, lambda: gdn.glr_fwd(x, x, x.cpu(), lam)), (TypeError, lambda: gdn.glr_fwd(x, x.float(), x, lam)),
        (TypeError, lambda: gdn.glr_fwd(x, x, x, lam.to(BF))), (ValueError, lambda: gdn.glr_fwd(x, x, x[:, :2], lam)),
        (ValueError, lambda: gdn.glr_step(x, x, x, lam, r(1, C))), (ValueError, lambda: gdn.glr_bwd_saved(x, x, x, lam, x, None)),
        (TypeError, lambda: gdn.glr_fwd(x.half(), x, x, lam)), (ValueError, lambda: gdn.glr_fwd(x, x, x, lam, h0=r(2, C))),
        (TypeError, lambda: gdn.rope_fwd(q, k.float(), **how)), (ValueError, lambda: gdn.rope_fwd(q, k, how["inv_freq"], norm="max")),
        (ValueError, lambda: gdn.rope_fwd(q, k, how["inv_freq"], positions=lens)), (ValueError, lambda: gdn.rope_fwd(q.transpose(1, 2), k, **how)),
        (TypeError, lambda: gdn.rope_fwd(q, k, how["inv_freq"], positions=torch.zeros(2, 4, device=DEV, dtype=torch.int64))),
        (ValueError, lambda: gdn.swa_fwd(q, k, v[:, :2], W)), (ValueError, lambda: gdn.swa_fwd(q[..., :32], k, v, W)),
        (ValueError, lambda: gdn.swa_step(q, k, v, *cache, lens, sinks=S)), (TypeError, lambda: gdn.swa_step(q1, k1, v1, *cache, lens.long(), sinks=S)),
        (ValueError, lambda: gdn.swa_step(q1, k1, v1, cache[0], cache[1][:1], lens, sinks=S)),
        (ValueError, lambda: gdn.swa_fill(k, v, *cache, sinks=S + W)),
    ]
    for n, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {n} was taken")
    for n, call in enumerate((lambda: gdn.swa_fwd(q, k, v, 0), lambda: gdn.swa_fwd(q, k, v, W, sinks=2000),
                              lambda: gdn.rope_fwd(q, k, how["inv_freq"], norm="l2", wq=how["wq"]),
                              lambda: gdn.glr_fwd(x, x, x, lam, c=-1.0), lambda: gdn.swa_fwd(q[..., :2 * D], k, v, W, out=None, scale=1.0, cu_seqlens=[0, 5]),
                              lambda: gdn.swa_step(q1, k1, v1, cache[0], cache[0], lens, sinks=S))):
        with pytest.raises((gdn.GdnError, ValueError)):
            call()
            pytest.fail(f"call {n} was taken")
