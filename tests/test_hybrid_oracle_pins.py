"""The float64 definitions of the hybrid operators against differences, closed forms and
planted mistakes (CPU)."""
import torch

import _hybrid_oracle as ref


def _glr_args(B=2, T=9, C=3, seed=0, z=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return [r(B, T, C), r(B, T, C), r(B, T, C), r(C) - 2, r(B, T, C) if z else None], r, B


def test_glr_gradients_against_differences():
    for z, cu in ((True, None), (False, None), (True, [0, 4, 4, 9])):
        args, r, B = _glr_args(B=1 if cu else 2, z=z)
        n = len(cu) - 1 if cu else B
        h0, dy, dl = r(n, 3), r(*args[0].shape), r(n, 3)
        out, _ = ref.glr(*args, h0, cu, dy=dy, dlast=dl)

        def loss(*leaves):
            o, _ = ref.glr(*leaves[:4], leaves[4] if z else None, leaves[-1], cu)
            return (o["y"] * dy).sum() + (o["state"] * dl).sum()

        leaves = [t for t in args if t is not None] + [h0]
        names = ["dx", "dr", "di", "dlam"] + (["dz"] if z else []) + ["dh0"]
        for k, name in enumerate(names):
            flat = leaves[k].reshape(-1)
            for j in range(0, flat.numel(), max(1, flat.numel() // 12)):
                keep, step = float(flat[j]), 1e-6
                flat[j] = keep + step
                up = loss(*leaves)
                flat[j] = keep - step
                down = loss(*leaves)
                flat[j] = keep
                assert abs(float(up - down) / (2 * step) - float(out[name].reshape(-1)[j])) <= 1e-7 * (1 + abs(float(up))), name


def test_glr_closed_forms():
    args, r, B = _glr_args(z=False)
    h0 = r(B, 3)
    shut = [args[0], torch.full_like(args[1], -60.0), *args[2:]]  # a gate that is shut keeps the state
    out, _ = ref.glr(*shut, h0, None)
    assert float((out["y"] - h0.unsqueeze(1)).abs().max()) <= 1e-11
    # one token of an open gate: a = exp(-c softplus(lam))
    out, _ = ref.glr(args[0][:, :1], torch.full((B, 1, 3), 60.0, dtype=torch.float64), torch.full((B, 1, 3), 60.0, dtype=torch.float64), args[3],
                     None, h0, None, c=2.0)
    a = (1 + torch.exp(args[3])) ** -2
    assert float((out["y"][:, 0] - (a * h0 + torch.sqrt(1 - a * a) * args[0][:, 0])).abs().max()) <= 1e-14
    # packed = each alone
    x, rr, i, lam, _ = args
    whole, _ = ref.glr(x[:1], rr[:1], i[:1], lam, None, h0, [0, 4, 9])
    for n, s in enumerate((slice(0, 4), slice(4, 9))):
        part, _ = ref.glr(x[:1, s], rr[:1, s], i[:1, s], lam, None, h0[n:n + 1], None)
        assert torch.equal(part["y"], whole["y"][:, s]) and torch.equal(part["state"][0], whole["state"][n])


def test_glr_bounds_notice_a_planted_mistake():
    """A state taken one token late, or sqrt(1 - a) for sqrt(1 - a^2), is far outside the bounds."""
    args, r, B = _glr_args(T=20)
    out, err = ref.glr(*args, r(B, 3), None, dy=r(*args[0].shape))
    for name in out:
        assert float((err[name] / out[name].abs().mean()).max()) <= 1e-3, name
        ref.check(name, out[name].float(), out[name], err[name] + 2 * ref.U * out[name].abs())
    bad = torch.cat([out["y"][:, 1:], out["y"][:, :1]], 1)
    try:
        ref.check("late", bad.float(), out["y"], err["y"])
    except AssertionError:
        return
    raise AssertionError("a planted mistake passed")


def test_rope_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    freq, pos = r(4).abs(), torch.tensor([[3, -7]], dtype=torch.int32)
    for norm in ("rms", "l2", None):
        for inter in (False, True):
            x, w, d = r(1, 2, 3, 12), r(12), r(1, 2, 3, 12)
            w = w if norm == "rms" else None
            out, _ = ref.rope(x, w, freq, pos, norm, 1e-3, inter, d)
            for leaf, name in ((x, "dx"), (w, "dw")):
                if leaf is None:
                    continue
                flat = leaf.reshape(-1)
                for j in range(0, flat.numel(), 5):
                    keep, vals = float(flat[j]), []
                    for sign in (1, -1):
                        flat[j] = keep + sign * 1e-6
                        vals.append(float((ref.rope(x, w, freq, pos, norm, 1e-3, inter)[0]["out"] * d).sum()))
                    flat[j] = keep
                    assert abs((vals[0] - vals[1]) / 2e-6 - float(out[name].reshape(-1)[j])) <= 1e-7, (norm, inter, name)


def test_rope_is_a_rotation():
    """Pairs as complex numbers; scores depend on the distance of the positions alone."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(1, 2, 1, 8, generator=g, dtype=torch.float64)
    freq = torch.tensor([1.0, 0.25, 0.01], dtype=torch.float64)
    pos = torch.tensor([[5, 11]])
    y, _ = ref.rope(x, None, freq, pos, None, 0.0, True)
    z = torch.view_as_complex(x[..., :6].reshape(1, 2, 1, 3, 2)) * torch.polar(torch.ones(1, 2, 1, 3, dtype=torch.float64),
                                                                                  pos[..., None, None] * freq)
    assert float((y["out"][..., :6] - torch.view_as_real(z).flatten(-2)).abs().max()) <= 1e-15
    assert torch.equal(y["out"][..., 6:], x[..., 6:])
    for inter in (False, True):
        near = ref.rope(x, None, freq, pos, None, 0.0, inter)[0]["out"]
        far = ref.rope(x, None, freq, pos + 1000, None, 0.0, inter)[0]["out"]
        assert abs(float((near[0, 0] * near[0, 1]).sum() - (far[0, 0] * far[0, 1]).sum())) <= 1e-12


def test_swa_gradients_against_differences():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for W, S, cu in ((3, 0, None), (2, 2, None), (4, 1, [0, 0, 3, 10]), (50, 5, None)):
        q, k, v, do = r(1, 10, 4, 5), r(1, 10, 2, 5), r(1, 10, 2, 5), r(1, 10, 4, 5)
        out, _ = ref.swa(q, k, v, W, S, 0.7, cu, do)
        for leaf, name in ((q, "dq"), (k, "dk"), (v, "dv")):
            flat = leaf.reshape(-1)
            for j in range(0, flat.numel(), 7):
                keep, vals = float(flat[j]), []
                for sign in (1, -1):
                    flat[j] = keep + sign * 1e-6
                    vals.append(float((ref.swa(q, k, v, W, S, 0.7, cu)[0]["o"] * do).sum()))
                flat[j] = keep
                assert abs((vals[0] - vals[1]) / 2e-6 - float(out[name].reshape(-1)[j])) <= 1e-7, (W, S, name)


def test_swa_masks():
    assert ref.seen(5, 2, 1).int().tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert torch.equal(ref.seen(6, 6, 0), torch.ones(6, 6).tril().bool())
    assert torch.equal(ref.seen(6, 1, 0), torch.eye(6).bool())


def test_swa_step_continues_the_sequence():
    """Token by token through the cache = the rows of the whole sequence."""
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for W, S in ((1, 0), (3, 0), (3, 2), (20, 4)):
        q, k, v = r(2, 11, 2, 4), r(2, 11, 1, 4), r(2, 11, 1, 4)
        want, _ = ref.swa(q, k, v, W, S, 0.5, None)
        kc, vc = r(2, S + W, 1, 4), r(2, S + W, 1, 4)
        for t in range(11):
            o, _, kc, vc = ref.swa_step(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], kc, vc, torch.tensor([t, t]), S, 0.5)
            assert float((o - want["o"][:, t:t + 1]).abs().max()) <= 1e-14, (W, S, t)
