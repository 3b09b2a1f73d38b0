"""float64 definitions of the layer operators (CPU, token by token), their gradients,
and the magnitudes that the tests' tolerances are counted in.

Every quantity the operators compute is a sum of products.  With ``size=True`` the
functions below replace each factor by its absolute value (the decays, which are
positive, stay), so that they return the sum of the absolute values of the terms:
an fp32 evaluation with K rounded operations on the way of a term is off by at most
K 2^-24 of that sum, however the terms cancel.
"""
import torch


def spans(B, T, cu):
    if cu is None:
        return [(i, 0, T) for i in range(B)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def _f64(*ts):
    return [None if t is None else t.detach().double().cpu() for t in ts]


def _abs(*ts):
    return [None if t is None else t.abs() for t in ts]


# --------------------------------------------------------------------------- convolution

def conv(x, w, b, s0, cu, silu):
    """(y, final state), differentiable."""
    B, T, C = x.shape
    W = w.shape[1]
    last = []
    parts = {i: [] for i in range(B)}
    for n, (i, t0, t1) in enumerate(spans(B, T, cu)):
        head = s0[n] if s0 is not None else x.new_zeros(W - 1, C)
        line = torch.cat([head, x[i, t0:t1]])
        p = sum(line[j:j + t1 - t0] * w[:, j] for j in range(W))
        if b is not None:
            p = p + b
        parts[i].append(p * torch.sigmoid(p) if silu else p)
        last.append(line[t1 - t0:])
    ys = torch.stack([torch.cat(parts[i]) if parts[i] else x.new_zeros(0, C) for i in range(B)]) if B else x
    return ys, torch.stack(last) if last else x.new_zeros(0, W - 1, C)


def conv_grads(x, w, b, s0, cu, silu, dy, dlast):
    """dx, dweight, dbias, dstate0 of <y, dy> + <final state, dlast>, by reverse mode."""
    x, w, b, s0, dy, dlast = _f64(x, w, b, s0, dy, dlast)
    leaves = [t.requires_grad_() for t in (x, w, b, s0) if t is not None]
    y, last = conv(x, w, b, s0, cu, silu)
    loss = (y * dy).sum()
    if dlast is not None:
        loss = loss + (last * dlast).sum()
    g = list(torch.autograd.grad(loss, leaves, allow_unused=True))
    g = [torch.zeros_like(t) if v is None else v for t, v in zip(leaves, g)]
    out = {"dx": g[0], "dweight": g[1]}
    out["dbias"] = g[2] if b is not None else None
    out["dstate0"] = g[-1] if s0 is not None else None
    return out


def conv_sizes(x, w, b, s0, cu, dy=None, dlast=None):
    """Sums of absolute terms: pre-activation, final state, gradients (|silu'| <= 1.1)."""
    x, w, b, s0, dy, dlast = _abs(*_f64(x, w, b, s0, dy, dlast))
    p, last = conv(x, w, b, s0, cu, False)
    out = {"y": p, "state": last}
    if dy is not None:
        out.update(conv_grads(x, w, b, s0, cu, False, 1.1 * dy, dlast))
    return out


# --------------------------------------------------------------------------- scan

def scan(u, dt, A, Bm, Cm, D, z, bias, h0, cu, softplus, dy=None, dlast=None, size=False):
    """dict y, state and, with dy, the gradients, by the written-out formulas."""
    u, dt, A, Bm, Cm, D, z, bias, h0, dy, dlast = _f64(u, dt, A, Bm, Cm, D, z, bias, h0, dy, dlast)
    nb, T, Dn = u.shape
    G, N = Bm.shape[2:]
    pre = dt if bias is None else dt + bias
    delta = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-pre.abs())) if softplus else pre
    slope = torch.sigmoid(pre) if softplus else torch.ones_like(pre)
    a = torch.exp(delta.unsqueeze(-1) * A)  # true decays, whatever `size`
    sg = torch.sigmoid(z) if z is not None else None
    gate = z * sg if z is not None else torch.ones_like(u)
    dgate = sg * (1 + z * (1 - sg)) if z is not None else None
    if size:
        u, A, Bm, Cm, D, h0, dy, dlast, gate, delta = _abs(u, A, Bm, Cm, D, h0, dy, dlast, gate, delta)
        if z is not None:  # the gate's derivative has two terms, of opposite signs for z < 0
            dgate = sg + z.abs() * sg * (1 - sg)
    if D is None:
        D = u.new_zeros(Dn)
    wide = lambda t: t.repeat_interleave(Dn // G, -2)  # noqa: E731
    seqs = spans(nb, T, cu)
    y, s_all = torch.zeros_like(u), torch.zeros_like(u)
    state = u.new_zeros(len(seqs), Dn, N)
    out = {"y": y, "state": state}
    if dy is not None:
        for key, like in (("du", u), ("ddt", u), ("dB", Bm), ("dC", Cm), ("dA", A), ("dD", D), ("dz", u), ("ddt_bias", D),
                          ("dh0", state)):
            out[key] = torch.zeros_like(like)
    for n, (i, t0, t1) in enumerate(seqs):
        h = h0[n] if h0 is not None else u.new_zeros(Dn, N)
        before = []
        for t in range(t0, t1):
            before.append(h)
            h = a[i, t] * h + (delta[i, t] * u[i, t]).unsqueeze(-1) * wide(Bm[i, t])
            s_all[i, t] = (wide(Cm[i, t]) * h).sum(-1) + D * u[i, t]
            y[i, t] = s_all[i, t] * gate[i, t]
        state[n] = h
        if dy is None:
            continue
        g = dlast[n] if dlast is not None else u.new_zeros(Dn, N)
        after = h
        for t in range(t1 - 1, t0 - 1, -1):
            ds = dy[i, t] * gate[i, t]
            g = g + wide(Cm[i, t]) * ds.unsqueeze(-1)
            out["dC"][i, t] = (after * ds.unsqueeze(-1)).reshape(G, Dn // G, N).sum(1)
            out["dB"][i, t] = (g * (delta[i, t] * u[i, t]).unsqueeze(-1)).reshape(G, Dn // G, N).sum(1)
            gB = (g * wide(Bm[i, t])).sum(-1)
            after = before[t - t0]
            g = g * a[i, t]
            q = g * after
            out["du"][i, t] = D * ds + delta[i, t] * gB
            out["ddt"][i, t] = (u[i, t] * gB + (A * q).sum(-1)) * slope[i, t]
            out["dA"] += delta[i, t].unsqueeze(-1) * q
            out["dD"] += ds * u[i, t]
            out["ddt_bias"] += out["ddt"][i, t]
            if z is not None:
                out["dz"][i, t] = dy[i, t] * s_all[i, t] * dgate[i, t]
        out["dh0"][n] = g
    return out


# --------------------------------------------------------------------------- delta rule step

def delta_step(q, k, v, g, beta, S, scale, size=False):
    """(o, S) after one token; q, k (B, 1, H, Dk), g (B, 1, H) or (B, 1, H, Dk)."""
    q, k, v, g, beta, S = _f64(q, k, v, g, beta, S)
    if size:
        q, k, v, S = _abs(q, k, v, S)
    q, k, v, g, beta = (t[:, 0] for t in (q, k, v, g, beta))
    a = torch.exp(g)
    S = S * (a.unsqueeze(-1) if g.dim() == 3 else a[..., None, None])
    held = (S * k.unsqueeze(-1)).sum(-2)
    e = beta.unsqueeze(-1) * (v + held if size else v - held)
    S = S + k.unsqueeze(-1) * e.unsqueeze(-2)
    return (scale * (S * q.unsqueeze(-1)).sum(-2)).unsqueeze(1), S


# --------------------------------------------------------------------------- comparison

def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def check(name, got, ref, size, roundings, stored=True):
    """|got - ref| <= roundings 2^-24 size, and one rounding of the result where it is
    stored in fewer bits."""
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    x, r = got.detach().double().cpu(), ref.double()
    allowed = roundings * 2.0 ** -24 * size + 1e-37
    if stored and got.dtype != torch.float32:
        allowed = allowed + half_step(got.dtype) * (r.abs() + allowed)
    off = (x - r).abs()
    bad = ~(off <= allowed)
    if bool(bad.any()):
        at = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values too far off; first at {at}: "
                             f"{x.flatten()[at]:.9g} for {r.flatten()[at]:.9g}, allowed {allowed.flatten()[at]:.3g}")
