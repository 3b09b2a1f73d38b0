"""float64 definitions of the operators of hybrid models (CPU), their gradients, and
bounds on the error of an fp32 evaluation.

The bounds are running error analyses: next to each value stands the sum of the absolute
values of its terms and what the roundings on the way of each term can add up to, in
units of 2^-24, with the true values of decays and gates.  ``check`` adds the final
rounding to the output's type, half a step of it.
"""
import torch

U = 2.0 ** -24


def spans(B, T, cu):
    """(first row, last row + 1) of every sequence of the flattened (B T) rows."""
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def f64(*ts):
    return [None if t is None else t.detach().double().cpu() for t in ts]


def check(name, got, want, bound):
    """|got - want| <= bound + half a step of got's type."""
    assert tuple(got.shape) == tuple(want.shape), (name, got.shape, want.shape)
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    off = (got.detach().double().cpu() - want).abs()
    # the rounded value may be of a size that the bound has moved
    room = bound + half * (want.abs() + bound) + torch.finfo(torch.float32).tiny
    bad = ~(off <= room)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / room).nan_to_num(9e9).max()):.3g} of the bound"


# --------------------------------------------------------------------------- gated linear recurrence

def glr(x, r, i, lam, z, h0, cu, c=8.0, dy=None, dlast=None):
    """(values, bounds): dicts y, state and, with dy, the gradients of <y, dy> + <state,
    dlast>, by the written-out formulas, token by token.

    Roundings: a sigmoid of v (|v| + 4: the exponent's, of the exponential's argument, and
    the quotient's), la that of r's sigmoid and 8 more (softplus, factors), kl in all; a
    kl |la| + 3; m half of kl and 14 for the difference (1 - a^2 >= 0.39 where it is taken,
    and the exponential's derivative is at most 1 over the rest), at most 12 + kl / 2; a state one for the
    multiply-add, and 100 for the joins of runs, waves and segments."""
    x, r, i, lam, z, h0, dy, dlast = f64(x, r, i, lam, z, h0, dy, dlast)
    B, T, C = x.shape
    shape = x.shape
    x, r, i, z, dy = [None if t is None else t.reshape(B * T, C) for t in (x, r, i, z, dy)]
    soft = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    la = -c * soft * sr
    kl = r.abs() + 12
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    ka, km = kl * la.abs() + 3, 12 + kl / 2
    ki = i.abs() + 4
    b = m * si * x
    kb = km + ki + 3
    seqs = spans(B, T, cu)
    n = len(seqs)
    h, hp = torch.zeros_like(x), torch.zeros_like(x)
    hs, hps, eh, ehp = (torch.zeros_like(x) for _ in range(4))  # sums of absolute terms, errors
    last, elast = x.new_zeros(n, C), x.new_zeros(n, C)
    for q, (t0, t1) in enumerate(seqs):
        v = h0[q] if h0 is not None else x.new_zeros(C)
        s, e = v.abs(), torch.zeros_like(v)
        for t in range(t0, t1):
            hp[t], hps[t], ehp[t] = v, s, e + 100 * U * s
            v = a[t] * v + b[t]
            e = a[t] * e + (ka[t] + 1) * U * a[t] * s + (kb[t] + 1) * U * b[t].abs()
            s = a[t] * s + b[t].abs()
            h[t], hs[t], eh[t] = v, s, e + 100 * U * s
        last[q], elast[q] = v, e + 100 * U * s
    if z is not None:
        sz = torch.sigmoid(z)
        gate, kz = z * sz, z.abs() + 7
        y, ey = h * gate, (eh + kz * U * hs) * gate.abs()
    else:
        y, ey = h, eh
    out, err = {"y": y.reshape(shape), "state": last}, {"y": ey.reshape(shape), "state": elast}
    if dy is None:
        return out, err
    ds = dy * gate if z is not None else dy
    kd = kz if z is not None else torch.zeros_like(x)
    G, Gs, eG = (torch.zeros_like(x) for _ in range(3))
    dh0, edh0 = x.new_zeros(n, C), x.new_zeros(n, C)
    for q, (t0, t1) in enumerate(seqs):
        v = dlast[q] if dlast is not None else x.new_zeros(C)
        s, e = v.abs(), torch.zeros_like(v)
        for t in range(t1 - 1, t0 - 1, -1):
            v, e = ds[t] + v, e + (kd[t] + 1) * U * ds[t].abs() + U * s
            s = ds[t].abs() + s
            G[t], Gs[t], eG[t] = v, s, e + 100 * U * s
            v, e, s = a[t] * v, a[t] * e + (ka[t] + 1) * U * a[t] * s, a[t] * s
        dh0[q], edh0[q] = v, e + 100 * U * s
    xs = x.abs()
    dx, edx = G * m * si, (eG + (km + ki + 3) * U * Gs) * m * si
    di = G * m * x * si * (1 - si)
    edi = (eG * (1 - si) + Gs * ((km + ki + 5) * (1 - si) + 4) * U) * m * xs * si  # 1 - s: off by roundings of 1
    lm = torch.where(m > 0, la / m, 0)
    one, two = a * la * hp, a * a * lm * si * x
    E = G * (one - two)
    both = (a * la.abs() * hps + a * a * lm.abs() * si * xs)
    eE = eG * both + Gs * (a * la.abs() * (ehp + (ka + kl + 6) * U * hps) + (2 * ka + kl + km + ki + 8) * U * a * a * lm.abs() * si * xs)
    Es = Gs * both
    dr, edr = E * (1 - sr), eE * (1 - sr) + 6 * U * Es
    ratio = torch.sigmoid(lam) / soft
    dlam, edlam = E.sum(0) * ratio, (eE.sum(0) + (min(B * T, 4096) + 40) * U * Es.sum(0)) * ratio
    out.update(dx=dx.reshape(shape), dr=dr.reshape(shape), di=di.reshape(shape), dlam=dlam, dh0=dh0)
    err.update(dx=edx.reshape(shape), dr=edr.reshape(shape), di=edi.reshape(shape), dlam=edlam, dh0=edh0)
    if z is not None:
        slope, wide = sz * (1 + z * (1 - sz)), sz * (1 + z.abs() * (1 - sz) + z.abs())
        out["dz"] = (dy * h * slope).reshape(shape)
        err["dz"] = (dy.abs() * (eh * slope.abs() + hs * (z.abs() + 16) * U * wide)).reshape(shape)
    return out, err


# --------------------------------------------------------------------------- norm and rotation

def turned(x, angle, inter, back=False):
    """The first pairs of x (..., H, D) turned by angle (..., R / 2), or back; with |sin| and
    |cos| as given where angle is a pair of tensors."""
    cos, sin = (torch.cos(angle), torch.sin(angle)) if isinstance(angle, torch.Tensor) else angle
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    if back:
        sin = -sin
    n = cos.shape[-1]
    out = x.clone()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _mixed(x, pairs, inter):
    """|x_j| + |x_j'| of every turned channel, |x| of the others."""
    one = torch.ones(*x.shape[:-2], pairs, dtype=x.dtype)
    return turned(x.abs(), (one, -one), inter).abs().maximum(turned(x.abs(), (one, one), inter).abs())


def rope(x, w, freq, pos, norm, eps, inter, d=None):
    """(values, bounds) of one of q, k: dicts out and, with d, dx, dw.

    Roundings: a row's sum of squares 20 (16 values a lane at most, six joins), inv 14 (half
    of that, a root, a quotient), n 17; a cosine or sine 6 of one and 2^-50 of the angle; the
    turned value two more.  Weights' gradients: an eighth of the rows one after another (16
    rows of a workgroup share them, or 8 of 256 values) and 150 for the joins."""
    x, w, freq, d = f64(x, w, freq, d)
    pos = pos.detach().double().cpu()
    angle = pos.unsqueeze(-1) * freq
    D, pairs = x.shape[-1], freq.numel()
    lost = 30 * U + angle.abs().amax() * 2.0 ** -50 if pairs else 30 * U
    ss = (x * x).sum(-1, keepdim=True)
    if norm == "rms":
        inv, share = 1 / torch.sqrt(ss / D + eps), 1 / D
    elif norm == "l2":
        inv, share = 1 / torch.sqrt(ss).clamp(min=1e-30), (ss.sqrt() > 1e-30).double()
    else:
        inv, share = torch.ones_like(ss), 0.0
    ww = w if w is not None else torch.ones(D, dtype=torch.float64)
    n = x * inv * ww
    out, err = {"out": turned(n, angle, inter)}, {"out": lost * _mixed(n, pairs, inter)}
    if d is None:
        return out, err
    g, gs = turned(d, angle, inter, back=True), _mixed(d, pairs, inter)
    u, us = g * ww, gs * ww.abs()
    dot, dots = (u * x).sum(-1, keepdim=True), (us * x.abs()).sum(-1, keepdim=True)
    out["dx"] = inv * (u - x * inv * inv * share * dot)
    err["dx"] = inv * ((lost + 20 * U) * us + (lost + 80 * U) * x.abs() * inv * inv * share * dots)
    rows = x.numel() // D
    out["dw"] = (g * x * inv).reshape(rows, D).sum(0)
    err["dw"] = ((lost + (rows / 8 + 150) * U) * gs * x.abs() * inv).reshape(rows, D).sum(0)
    return out, err


# --------------------------------------------------------------------------- window attention

def seen(Tq, W, S):
    i = torch.arange(Tq)
    return (i <= i[:, None]) & ((i > i[:, None] - W) | (i < S))


def _attend(q, k, v, mask, scale, half):
    """(o, lse, p, bound of o, relative bounds of p) of one head: q (n, D), k, v (m, D).

    Roundings: a score's D products summed (D + 3 of the absolute terms), the exponent's (its
    size, the maximum's and the sum's, twice, and 8); a probability that of its own score and
    the mean over its row's; `half` for its rounding as an operand; a sum over n keys n + 16."""
    n = mask.sum(-1, keepdim=True).double()
    s = (q @ k.T) * scale
    e = (q.shape[-1] + 3) * U * (q.abs() @ k.abs().T) * abs(scale)
    s = s.masked_fill(~mask, -torch.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    e = torch.where(mask, e + 2 * U * (s.abs().nan_to_num(posinf=0) + lse.abs() + 8), 0)
    mean = (p * e).sum(-1, keepdim=True)
    eta = torch.where(mask, e + mean + (n + 8) * U, 0)
    bound = (p * (eta + half + (n + 16) * U)) @ v.abs()
    return p @ v, lse, p, bound, eta


def swa(q, k, v, W, S, scale, cu, do=None):
    """(values, bounds): dicts o, lse and, with do, dq, dk, dv; every sequence and head alone."""
    io = q.dtype
    half = 0.0 if io == torch.float32 else torch.finfo(io).eps / 2
    q, k, v, do = f64(q, k, v, do)
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    group = Hq // Hk
    rows = lambda t: None if t is None else t.reshape(B * T, t.shape[2], D)  # noqa: E731
    q, k, v, do = rows(q), rows(k), rows(v), rows(do)
    out = {"o": torch.zeros_like(q), "lse": torch.zeros(B * T, Hq, dtype=torch.float64)}
    if do is not None:
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    err = {name: torch.zeros_like(t) for name, t in out.items()}
    for t0, t1 in spans(B, T, cu):
        if t1 == t0:
            continue
        mask = seen(t1 - t0, W, S)
        n, m = mask.sum(-1, keepdim=True).double(), mask.sum(0).double().unsqueeze(-1) * group
        for h in range(Hq):
            qs, ks, vs = q[t0:t1, h], k[t0:t1, h // group], v[t0:t1, h // group]
            o, lse, p, bo, eta = _attend(qs, ks, vs, mask, scale, half)
            out["o"][t0:t1, h], err["o"][t0:t1, h] = o, bo
            out["lse"][t0:t1, h] = lse[:, 0]
            err["lse"][t0:t1, h] = ((p * eta).sum(-1) + 8 * U * (lse[:, 0].abs() + 1))
            if do is None:
                continue
            d = do[t0:t1, h]
            dp, dps = d @ vs.T, d.abs() @ vs.abs().T
            delta = (d * o).sum(-1, keepdim=True)
            deltas = (d.abs() * o.abs()).sum(-1, keepdim=True)
            # from the stored o: its own bound, its rounding, the sum
            edelta = (d.abs() * (bo + half * (o.abs() + bo))).sum(-1, keepdim=True) + (D + 8) * U * deltas
            ds = p * (dp - delta) * scale
            eds = p * abs(scale) * (eta * (dp - delta).abs() + (D + 11) * U * dps + edelta + 8 * U * deltas) + half * ds.abs()
            eds = torch.where(mask, eds * (1 + half), 0)
            out["dq"][t0:t1, h] = ds @ ks
            err["dq"][t0:t1, h] = (eds + (n + 16) * U * ds.abs()) @ ks.abs()
            out["dk"][t0:t1, h // group] += ds.T @ qs
            err["dk"][t0:t1, h // group] += (eds.T + (m + 64) * U * ds.abs().T) @ qs.abs()
            out["dv"][t0:t1, h // group] += p.T @ d
            err["dv"][t0:t1, h // group] += (p * (eta + half)).T @ d.abs() + ((m + 64) * U * p.T) @ d.abs()
    shape = lambda t, H: t.reshape(B, T, H, *t.shape[2:])  # noqa: E731
    heads = {"o": Hq, "lse": Hq, "dq": Hq, "dk": Hk, "dv": Hk}
    return {x: shape(t, heads[x]) for x, t in out.items()}, {x: shape(t, heads[x]) for x, t in err.items()}


def slot_of(token, W, S):
    return token if token < S else S + (token - S) % W


def swa_step(q, k, v, kc, vc, lens, S, scale):
    """(o, its bound, keys' cache, values' cache) after one token of every sequence."""
    io = q.dtype
    half = 0.0 if io == torch.float32 else torch.finfo(io).eps / 2
    q, k, v, kc, vc = (t.clone() for t in f64(q, k, v, kc, vc))
    B, _, Hq, _ = q.shape
    W, group = kc.shape[1] - S, Hq // k.shape[2]
    o, err = torch.zeros_like(q), torch.zeros_like(q)
    for n, before in enumerate(lens.tolist()):
        if before < 0:
            continue
        slot = slot_of(before, W, S)
        kc[n, slot], vc[n, slot] = k[n, 0], v[n, 0]
        tokens = sorted(set(range(min(S, before + 1))) | set(range(max(0, before + 1 - W), before + 1)))
        slots = [slot_of(t, W, S) for t in tokens]
        assert len(set(slots)) == len(slots)
        for h in range(Hq):
            got, _, _, bound, _ = _attend(q[n, :, h], kc[n, slots, h // group], vc[n, slots, h // group],
                                          torch.ones(1, len(slots), dtype=torch.bool), scale, half)
            o[n, :, h], err[n, :, h] = got, bound
    return o, err, kc, vc
