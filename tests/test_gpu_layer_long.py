"""The layer operators on tensors of more than 2^31 values: their last rows against the
same rows of a small call (marked gpu)."""
import gc

import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
T, C, TAIL = 530000, 4096, 37  # 2.17e9 values


@pytest.fixture(autouse=True)
def _free():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _r(gen, *s, dtype=BF):
    return torch.randn(*s, generator=gen, device=DEV, dtype=dtype)


def _same(a, b):
    """Bitwise equality without copies of the whole tensors."""
    return bool((a == b).all())


def test_conv_of_many_rows():
    """Every output is formed by the same operations in the same order wherever its row
    stands, so the last rows are those of a call on them alone."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    x, dy, w, b = _r(gen, 1, T, C), _r(gen, 1, T, C), _r(gen, C, 4, dtype=F32), _r(gen, C, dtype=F32)
    assert x.numel() > 2 ** 31
    tail = lambda t: t[:, T - TAIL:].contiguous()  # noqa: E731
    rows = x[:, T - TAIL - 3:T - TAIL].contiguous()
    y, last = gdn.conv_fwd(x, w, bias=b)
    want, want_last = gdn.conv_fwd(tail(x), w, bias=b, state0=rows)
    assert _same(tail(y), want) and _same(last, want_last)
    del y
    got = gdn.conv_bwd(x, w, dy, bias=b)
    want = gdn.conv_bwd(tail(x), w, tail(dy), bias=b, state0=rows)
    torch.cuda.synchronize()
    assert _same(tail(got["dx"]), want["dx"])
    assert bool(torch.isfinite(got["dweight"]).all()) and bool(torch.isfinite(got["dbias"]).all())


def test_scan_of_many_tokens():
    """With decays of at most exp(-0.05) a token, terms older than 416 tokens are below
    2^-30: 3 x 416 roundings of the state and 80 of the sums and the composed segments,
    twice that for the gradient's chain on the states', on each side, and a bf16
    rounding on each side."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    N = 8
    u, dy = _r(gen, 1, T, C), _r(gen, 1, T, C)
    assert u.numel() > 2 ** 31
    dt = torch.empty(1, T, C, device=DEV, dtype=BF).uniform_(0.05, 0.2, generator=gen)
    A = -(1 + 2 * torch.rand(C, N, generator=gen, device=DEV))
    Bm, Cm = _r(gen, 1, T, 1, N), _r(gen, 1, T, 1, N)
    kw = dict(dt_softplus=False)
    tail = lambda t: t[:, T - TAIL:].contiguous()  # noqa: E731
    head = lambda t: t[:, T - TAIL - 1024:T - TAIL].contiguous()  # noqa: E731
    roundings = 3 * 416 + 80

    # the state before the tail, from the 1024 tokens before it (older ones: below 2^-70)
    start = lambda f: gdn.scan_fwd(f(head(u)), head(dt), A, f(head(Bm)), f(head(Cm)), **kw)[1]  # noqa: E731
    same = lambda t: t  # noqa: E731
    parts = {}
    for name, f in (("want", same), ("size", torch.abs)):
        ins = (f(tail(u)), tail(dt), A, f(tail(Bm)), f(tail(Cm)))
        y, h, saved = gdn.scan_fwd_save(*ins, h0=start(f), **kw)
        parts[name] = {"y": y, "h": h, **gdn.scan_bwd_saved(*ins, f(tail(dy)), saved, **kw)}
    y, h, saved = gdn.scan_fwd_save(u, dt, A, Bm, Cm, **kw)
    got = {"y": tail(y), "h": h}
    del y
    grads = gdn.scan_bwd_saved(u, dt, A, Bm, Cm, dy, saved, **kw)
    torch.cuda.synchronize()
    got.update({k: tail(grads[k]) for k in ("du", "ddt", "dB", "dC")})
    assert bool(torch.isfinite(grads["dA"]).all())

    want, size = parts["want"], parts["size"]
    # ddt = u sum_n G B + sum_n A q: its second term is negative where all inputs are positive
    size["ddt"] = 2 * tail(u).float().abs() * size["du"].float() / tail(dt).float() - size["ddt"].float()
    for k in ("y", "h", "du", "ddt", "dB", "dC"):
        n = roundings if k in ("y", "h") else 3 * roundings
        tol = 2 * n * 2.0 ** -24 * 1.02 * size[k].float()  # 1.02: the sizes are rounded to bf16 themselves
        if k != "h":
            tol += torch.finfo(BF).eps * want[k].float().abs() * 1.02
        err = (got[k].float() - want[k].float()).abs()
        assert bool((err <= tol).all()), (k, float((err / tol.clamp_min(1e-30)).max()))


def test_scan_step_of_many_sequences():
    gen = torch.Generator(device=DEV).manual_seed(2)
    B, N = 33000, 16
    u, dt, z = (_r(gen, B, 1, C) for _ in range(3))
    Bm, Cm = _r(gen, B, 1, 1, N), _r(gen, B, 1, 1, N)
    A, h = -torch.rand(C, N, generator=gen, device=DEV), _r(gen, B, C, N, dtype=F32)
    assert h.numel() > 2 ** 31
    last = [t[-2:].clone() for t in (u, dt, Bm, Cm, h, z)]
    y = gdn.scan_step(u, dt, A, Bm, Cm, h, z=z)
    want = gdn.scan_step(last[0], last[1], A, *last[2:5], z=last[5])
    assert _same(y[-2:], want) and _same(h[-2:], last[4])


@pytest.mark.parametrize("channel", [False, True])
def test_delta_step_of_many_heads(channel):
    gen = torch.Generator(device=DEV).manual_seed(3)
    B, H, D = 8300, 16, 128
    q, k, v = (_r(gen, B, 1, H, D) * D ** -0.5 for _ in range(3))
    g = -_r(gen, B, 1, H, *([D] if channel else []), dtype=F32).abs()
    beta, S = torch.rand(B, 1, H, generator=gen, device=DEV), _r(gen, B, H, D, D, dtype=F32)
    assert S.numel() > 2 ** 31
    last = [t[-40:].clone() for t in (q, k, v, g, beta, S)]  # 42 MB of states: the same column tiles
    call = gdn.kda_step if channel else gdn.step
    o = call(q, k, v, g, beta, S)
    want = call(*last)
    assert _same(o[-40:], want) and _same(S[-40:], last[5])
