"""The float64 definitions of the layer operators (tests/_layer_oracle.py), pinned on
the CPU: gradients against central differences, packed rows against the sequences
alone, and limiting cases."""
import math

import torch

import _layer_oracle as ref

F64 = torch.float64


def _rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def _differences(f, x, dirs=6, eps=1e-6):
    """(derivative along random directions by central differences, the directions)"""
    out = []
    for k in range(dirs):
        d = _rand(*x.shape, seed=900 + k)
        out.append(((f(x + eps * d) - f(x - eps * d)) / (2 * eps), d))
    return out


def test_conv_gradients_are_those_of_differences():
    x, w, b, s0 = _rand(1, 9, 8, seed=1), _rand(8, 4, seed=2), _rand(8, seed=3), _rand(3, 3, 8, seed=4)
    cu, dy, dl = [0, 2, 2, 9], _rand(1, 9, 8, seed=5), _rand(3, 3, 8, seed=6)
    g = ref.conv_grads(x, w, b, s0, cu, True, dy, dl)

    def loss(**kw):
        a = dict(x=x, w=w, b=b, s0=s0) | kw
        y, last = ref.conv(a["x"], a["w"], a["b"], a["s0"], cu, True)
        return float((y * dy).sum() + (last * dl).sum())

    for key, name, t in (("x", "dx", x), ("w", "dweight", w), ("b", "dbias", b), ("s0", "dstate0", s0)):
        for slope, d in _differences(lambda v, key=key: loss(**{key: v}), t):
            assert abs(slope - float((g[name] * d).sum())) < 1e-7 * (1 + abs(slope)), name


def test_conv_worked_values():
    # one channel, width 3: p_t = 1 x_{t-2} + 10 x_{t-1} + 100 x_t + 0.5, state (7, 8)
    x = torch.tensor([1.0, 2.0, 3.0], dtype=F64).reshape(1, 3, 1)
    y, last = ref.conv(x, torch.tensor([[1.0, 10.0, 100.0]], dtype=F64), torch.tensor([0.5], dtype=F64),
                       torch.tensor([[[7.0], [8.0]]], dtype=F64), None, False)
    assert y.flatten().tolist() == [187.5, 218.5, 321.5]
    assert last.flatten().tolist() == [2.0, 3.0]


def _scan_inputs(cu=None, T=7, D=16, N=8, G=2):
    n = 1 if cu is None else len(cu) - 1
    return dict(u=_rand(1, T, D, seed=1), dt=_rand(1, T, D, seed=2), A=-_rand(D, N, seed=3).abs(),
                Bm=_rand(1, T, G, N, seed=4), Cm=_rand(1, T, G, N, seed=5), D=_rand(D, seed=6), z=_rand(1, T, D, seed=7),
                bias=_rand(D, seed=8), h0=_rand(n, D, N, seed=9))


def test_scan_gradients_are_those_of_differences():
    cu = [0, 3, 3, 7]
    a = _scan_inputs(cu)
    dy, dl = _rand(1, 7, 16, seed=10), _rand(3, 16, 8, seed=11)
    g = ref.scan(**a, cu=cu, softplus=True, dy=dy, dlast=dl)

    def loss(**kw):
        r = ref.scan(**(a | kw), cu=cu, softplus=True)
        return float((r["y"] * dy).sum() + (r["state"] * dl).sum())

    names = dict(u="du", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", bias="ddt_bias", h0="dh0")
    for key, name in names.items():
        for slope, d in _differences(lambda v, key=key: loss(**{key: v}), a[key]):
            assert abs(slope - float((g[name] * d).sum())) < 2e-7 * (1 + abs(slope)), name


def test_scan_packed_is_each_sequence_alone():
    cu = [0, 4, 4, 7]
    a = _scan_inputs(cu)
    whole = ref.scan(**a, cu=cu, softplus=True)
    for n in range(3):
        part = {k: (v[:, cu[n]:cu[n + 1]] if k in ("u", "dt", "Bm", "Cm", "z") else v) for k, v in a.items()}
        part["h0"] = a["h0"][n:n + 1]
        one = ref.scan(**part, cu=None, softplus=True)
        torch.testing.assert_close(whole["y"][:, cu[n]:cu[n + 1]], one["y"])
        torch.testing.assert_close(whole["state"][n:n + 1], one["state"])


def test_scan_limits():
    a = _scan_inputs(T=5)
    # no steps: the state stays and only the skip is left of C h
    still = ref.scan(**(a | dict(dt=torch.zeros_like(a["dt"]), bias=None, z=None)), cu=None, softplus=False)
    torch.testing.assert_close(still["state"], a["h0"])
    # A = 0 with steps of one: a running sum of u B
    flat = ref.scan(**(a | dict(A=torch.zeros_like(a["A"]), dt=torch.ones_like(a["dt"]), bias=None, z=None)), cu=None, softplus=False)
    want = a["h0"][0] + sum(a["u"][0, t].unsqueeze(-1) * a["Bm"][0, t].repeat_interleave(8, 0) for t in range(5))
    torch.testing.assert_close(flat["state"][0], want)
    # one state, one channel pair: exp(-softplus(0)) = 1/2 per token
    half = ref.scan(**(a | dict(A=torch.full_like(a["A"], -1.0), dt=torch.zeros_like(a["dt"]), bias=None, u=torch.zeros_like(a["u"]))),
                    cu=None, softplus=True)
    torch.testing.assert_close(half["state"], a["h0"] * 0.5 ** 5)
    assert math.isclose(0.5, math.exp(-math.log1p(1.0)))


def test_sizes_bound_the_values():
    cu = [0, 3, 3, 7]
    a = _scan_inputs(cu)
    dy, dl = _rand(1, 7, 16, seed=10), _rand(3, 16, 8, seed=11)
    r = ref.scan(**a, cu=cu, softplus=True, dy=dy, dlast=dl)
    s = ref.scan(**a, cu=cu, softplus=True, dy=dy, dlast=dl, size=True)
    for k in r:
        assert bool((r[k].abs() <= s[k] * (1 + 1e-12)).all()), k


def test_delta_step_against_the_recurrence_oracle():
    import numpy as np

    import oracle

    B, H, Dk, Dv = 2, 3, 12, 10
    q, k, v = _rand(B, 1, H, Dk, seed=1), _rand(B, 1, H, Dk, seed=2), _rand(B, 1, H, Dv, seed=3)
    g, beta, S = -_rand(B, 1, H, seed=4).abs(), torch.sigmoid(_rand(B, 1, H, seed=5)), _rand(B, H, Dk, Dv, seed=6)
    o, S1 = ref.delta_step(q, k, v, g, beta, S, 0.5)
    o_ref, S_ref = oracle.fwd(*(t.numpy() for t in (q, k, v, g, beta)), S0=S.numpy(), scale=0.5)
    np.testing.assert_allclose(o.numpy(), o_ref.reshape(o.shape), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(S1.numpy(), S_ref, rtol=1e-12, atol=1e-14)
    gc = -_rand(B, 1, H, Dk, seed=7).abs()
    o, S1 = ref.delta_step(q, k, v, gc, beta, S, 0.5)
    o_ref, S_ref = oracle.kda_fwd(*(t.numpy() for t in (q, k, v, gc, beta)), S0=S.numpy(), scale=0.5)
    np.testing.assert_allclose(o.numpy(), o_ref.reshape(o.shape), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(S1.numpy(), S_ref, rtol=1e-12, atol=1e-14)
