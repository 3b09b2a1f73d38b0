"""Tensors of more than 2^31 values through the hybrid models' operators: what lies at the far end
is what the same call gives on a piece of it, or the definition (marked gpu)."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _hybrid_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def big(*shape):
    return torch.empty(*shape, device=DEV, dtype=BF).uniform_(-2, 2)


def test_recurrence():
    T, C = 33000, 65536
    x, r, i, dy = (big(1, T, C) for _ in range(4))
    lam = torch.linspace(-6, 2, C, device=DEV)
    y, h, saved = gdn.glr_fwd_save(x, r, i, lam)
    g = gdn.glr_bwd_saved(x, r, i, lam, dy, saved)
    for c in (slice(0, 64), slice(32768, 32832), slice(C - 64, C)):
        part = [t[..., c].contiguous() for t in (x, r, i, dy)]
        y1, h1, saved1 = gdn.glr_fwd_save(*part[:3], lam[c].contiguous())
        g1 = gdn.glr_bwd_saved(*part[:3], lam[c].contiguous(), part[3], saved1)
        assert torch.equal(y[..., c], y1) and torch.equal(h[:, c], h1)
        for name in ("dx", "dr", "di", "dlam", "dh0"):
            assert torch.equal(g[name][..., c], g1[name]), name


def test_rotation():
    T, H, D = (1 << 18) + 5, 64, 128
    q, k, dq = big(1, T, H, D), big(1, T, 1, D), big(1, T, H, D)
    freq = 10000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float32) / 32)
    q2, _ = gdn.rope_fwd(q, k, freq)
    g = gdn.rope_bwd(q, k, freq, dq, k)
    a = T - 100
    pos = torch.arange(a, T, device=DEV, dtype=torch.int32)[None]
    part = [t[:, a:].contiguous() for t in (q, k, dq)]
    assert torch.equal(q2[:, a:], gdn.rope_fwd(part[0], part[1], freq, positions=pos)[0])
    assert torch.equal(g["dq"][:, a:], gdn.rope_bwd(part[0], part[1], freq, part[2], part[1], positions=pos)["dq"])


def test_window():
    T, H, D, W = (1 << 18) + 70, 64, 128, 100
    q, k, v, do = big(1, T, H, D), big(1, T, 1, D), big(1, T, 1, D), big(1, T, H, D)
    o, lse = gdn.swa_fwd(q, k, v, W, scale=0.1, return_lse=True)
    g = gdn.swa_bwd(q, k, v, o, lse, do, W, scale=0.1)
    a = T - 300
    want, err = ref.swa(*(t[:, a:] for t in (q, k, v)), W, 0, 0.1, None, do[:, a:])
    far = slice(W, None)  # those before see keys that lie before the piece
    for name, got in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.check(name, got[:, a:][:, far], want[name][:, far], err[name][:, far])


def test_cache_of_many_sequences():
    B, W, S, Hk, D = 33, 65530, 6, 16, 64
    kc, vc = (torch.empty(B, S + W, Hk, D, device=DEV, dtype=BF) for _ in range(2))
    gen = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF)  # noqa: E731
    lens = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    lens[-1] = 900
    k0, v0, q, k, v = r(1, 900, Hk, D), r(1, 900, Hk, D), r(B, 1, Hk, D), r(B, 1, Hk, D), r(B, 1, Hk, D)
    cu = [0] * B + [900]
    gdn.swa_fill(k0, v0, kc, vc, sinks=S, cu_seqlens=cu)
    assert torch.equal(kc[-1, :900], k0[0]) and torch.equal(vc[-1, :900], v0[0])
    o = gdn.swa_step(q, k, v, kc, vc, lens, sinks=S, scale=0.125)
    want, err, _, _ = ref.swa_step(q[-1:], k[-1:], v[-1:], kc[-1:, :S + 1000], vc[-1:, :S + 1000], lens[-1:], S, 0.125)
    ref.check("o", o[-1:], want, err)
    assert float(o[:-1].abs().max()) == 0.0 and torch.equal(kc[-1, 900], k[-1, 0])


def test_cache_of_one_long_sequence():
    """Two million slots whose keys are zero but for the last: their scores are 0, and their values
    zero, so they add their number to the sum."""
    W, Hk, D = (1 << 21) + 64, 16, 64
    kc, vc = (torch.zeros(1, W, Hk, D, device=DEV, dtype=BF) for _ in range(2))
    gen = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF)  # noqa: E731
    q, k, v = r(1, 1, Hk, D), r(1, 1, Hk, D), r(1, 1, Hk, D)
    kc[0, -40:], vc[0, -40:] = q[0] * 2, r(40, Hk, D)
    lens = torch.tensor([W - 1], dtype=torch.int32, device=DEV)
    o = gdn.swa_step(q, k, v, kc, vc, lens, scale=0.125)
    assert torch.equal(kc[0, -1], k[0, 0]) and torch.equal(vc[0, -1], v[0, 0])
    ks, vs = kc[0, -40:].double(), vc[0, -40:].double()
    p = ((ks * q[0].double()).sum(-1) * 0.125).exp()
    want = (p[..., None] * vs).sum(0) / (p.sum(0) + (W - 40))[:, None]
    # probabilities rounded to bf16 as operands (2^-8 of sum |p v|), the sum of 2^21 ones over lanes and
    # runs (some 2000 roundings each way, 2^-24), and the result's rounding
    bound = (2 ** -8 + 4000 * 2.0 ** -24) * (p[..., None] * vs.abs()).sum(0) / (p.sum(0) + (W - 40))[:, None]
    ref.check("o", o[0, 0], want.cpu(), bound.cpu())
