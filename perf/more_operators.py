"""Workloads of the operators that hybrid models put next to the delta rule: the gated
linear recurrence, the norm and rotation of queries and keys, and causal attention over
a sliding window whose first tokens stay visible.

Each case is one pass through one operator.  With ``own`` false, ``run`` evaluates the
operator's plain form in fp32 torch arithmetic (angles in fp64); with ``own`` true it
makes the library's calls.  ``exact`` evaluates the definitions in fp64.
"""
import math
import random

import torch

own = False

_IO = {"bf16": torch.bfloat16, "fp32": torch.float32}
_DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one very long sequence (the repository's 65536 tokens) of 8 heads' width: few channels, many steps
        dict(name="recurrence prompt long", op="glr", io="bf16", B=1, T=65536, seqs=0, C=1024, z=True, state=False),
        # training step at the repository's training shape (4 x 4096 tokens, 2 x 8 heads of 128)
        dict(name="recurrence train", op="glr_train", io="bf16", B=4, T=4096, seqs=0, C=2048, z=True, state=False),
        # fp32 training over short odd sequences packed in a row, states in and out
        dict(name="recurrence train ragged fp32", op="glr_train", io="fp32", B=1, T=1501, seqs=5, C=328, z=False, state=True),
        # decoding: one token of each of 256 sequences
        dict(name="recurrence step", op="glr_step", io="bf16", B=256, C=4096, z=True),
        # prompts packed (the repository's 10240 rows), 16 query heads on 4 key heads, unit rows for the delta rule,
        # half of each head rotated
        dict(name="rotation prompts packed", op="rope", io="bf16", B=1, T=10240, Hq=16, Hk=4, D=128, R=64, norm="l2", inter=False, far=10240),
        # training step, normalised heads, whole heads rotated
        dict(name="rotation train", op="rope_train", io="bf16", B=4, T=4096, Hq=16, Hk=8, D=128, R=128, norm="rms", inter=False, far=4096),
        # decoding: one token of each of 64 sequences, some at far positions
        dict(name="rotation step", op="rope", io="bf16", B=64, T=1, Hq=16, Hk=4, D=128, R=128, norm="rms", inter=True, far=1 << 20),
        # prompts of a batch into a cache for decoding
        dict(name="window prompt", op="swa", io="bf16", B=2, T=4096, seqs=0, Hq=16, Hk=4, D=128, W=1024, S=4),
        # training step at the repository's training tokens
        dict(name="window train", op="swa_train", io="bf16", B=4, T=4096, seqs=0, Hq=16, Hk=8, D=128, W=512, S=4),
        # fp32 training over odd packed sequences, narrow heads, an odd window
        dict(name="window train ragged fp32", op="swa_train", io="fp32", B=1, T=1501, seqs=5, Hq=6, Hk=2, D=64, W=100, S=3),
        # decoding for a batch: sequences of all ages, most with a full window
        dict(name="window step batch", op="swa_step", io="bf16", B=64, Hq=16, Hk=4, D=128, W=4096, S=4, far=1 << 15),
        # decoding for one user: latency, one cache to spread over the chip
        dict(name="window step one", op="swa_step", io="bf16", B=1, Hq=16, Hk=4, D=128, W=2048, S=4, far=1 << 14),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr", "glr", "glr_train", "glr_train", "glr_step", "rope", "rope_train", "swa", "swa", "swa_train", "swa_train", "swa_step", "swa_step"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "glr_step":
        return dict(op=op, io=io, B=_log(rng, 1, 512), C=8 * _log(rng, 8, 512), z=flag())
    group = rng.choice([1, 2, 4, 8])
    Hk = _log(rng, 1, 16 // group)
    heads = dict(Hq=Hk * group, Hk=Hk)
    if op in ("rope", "rope_train"):
        D = rng.choice([64, 128, 128, 256])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, (1 << 25) // (B * D * (heads["Hq"] + Hk))))
        return dict(op=op, io=io, B=B, T=min(T, 8192), **heads, D=D, R=16 * rng.randint(1, D // 16), norm=rng.choice(["rms", "l2", None]),
                    inter=flag(), far=_log(rng, 1, 1 << 20))
    if op == "swa_step":
        D, W = rng.choice([64, 128]), _log(rng, 1, 4096)
        return dict(op=op, io=io, B=_log(rng, 1, 64), **heads, D=D, W=W, S=rng.randint(0, 16), far=_log(rng, 1, 1 << 17))
    packed = rng.random() < 0.4
    seqs = rng.randint(2, 9) if packed else 0
    B = 1 if packed else _log(rng, 1, 4)
    if op in ("glr", "glr_train"):
        C = 8 * _log(rng, 8, 256)
        T = _log(rng, 16 if packed else 1, min(65536, (1 << 25) // (B * C)))
        return dict(op=op, io=io, B=B, T=T, seqs=seqs, C=C, z=flag(), state=flag())
    # training over two tokens and more: the gradients of a softmax over one score are zero but for roundings
    train = op == "swa_train"
    T = _log(rng, 16 if packed or train else 1, 4096 if io == "bf16" else 2048)
    return dict(op=op, io=io, B=B, T=T, seqs=seqs, **heads, D=rng.choice([64, 128]), W=_log(rng, 2, 512) if train else _log(rng, 1, 1024),
                S=rng.randint(0, 16))


def _offsets(case):
    """Offsets of the sequences of a case: ragged where they are packed, with an empty one among four or more."""
    T, n = case.get("T", 1), case.get("seqs", 0)
    if not n:
        return [i * T for i in range(case["B"] + 1)]
    r = random.Random(1000 * T + n)
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    if n >= 4:
        cuts[1] = cuts[0]
    return [0] + cuts + [T]


# ----------------------------------------------------------------------------- inputs

def _inputs(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    io = _IO[case["io"]]
    B, T, op = case["B"], case.get("T", 1), case["op"]

    def normal(*shape, std=1.0, dtype=io):
        return (torch.randn(*shape, generator=g, device=_DEV) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=_DEV) * (hi - lo) + lo

    offsets = _offsets(case)
    s = dict(case=case, packed=bool(case.get("seqs")), offsets=offsets, cu=torch.tensor(offsets, dtype=torch.int64, device=_DEV))
    n = len(offsets) - 1
    if op.startswith("glr"):
        C = case["C"]
        s["x"], s["r"], s["i"] = normal(B, T, C), normal(B, T, C), normal(B, T, C)
        # decays of 0.9 .. 0.999 a token where the recurrence gate is open, at the usual factor of 8
        rate = -torch.log(uniform(0.9, 0.999, C)) / 8
        s["lam"] = torch.log(torch.expm1(rate))
        s["z"] = normal(B, T, C) if case["z"] else None
        s["state"] = normal(n, C, dtype=torch.float32) if case.get("state", True) else None
        if op == "glr_train":
            s["dy"] = normal(B, T, C)
            s["dstate"] = normal(n, C, dtype=torch.float32) if case["state"] else None
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if op.startswith("rope"):
        # queries, keys and values of one projection side by side: q and k are views of its rows
        rows = normal(B, T, (Hq + 2 * Hk) * D)
        s["q"], s["k"] = rows[..., :Hq * D].unflatten(-1, (Hq, D)), rows[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["freq"] = 10000.0 ** (-torch.arange(case["R"] // 2, device=_DEV, dtype=torch.float32) * 2 / case["R"])
        first = torch.randint(0, case["far"], (B, 1), generator=g, device=_DEV)
        s["pos"] = (first + torch.arange(T, device=_DEV)).to(torch.int32)
        rms = case["norm"] == "rms"
        s["wq"], s["wk"] = (uniform(0.5, 1.5, D), uniform(0.5, 1.5, D)) if rms else (None, None)
        s["eps"] = 1e-6
        if op == "rope_train":
            s["dq"], s["dk"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
        return s
    s["scale"] = D ** -0.5
    # queries and keys behind their norm and rotation: rows of unit variance
    s["q"], s["k"], s["v"] = normal(B, T, Hq, D), normal(B, T, Hk, D), normal(B, T, Hk, D)
    if op == "swa_train":
        s["do"] = normal(B, T, Hq, D)
    elif op == "swa":
        s["kc"], s["vc"] = (torch.zeros(n, case["S"] + case["W"], Hk, D, dtype=io, device=_DEV) for _ in range(2))
    else:
        s["kc"], s["vc"] = normal(B, case["S"] + case["W"], Hk, D), normal(B, case["S"] + case["W"], Hk, D)
        lens = (case["far"] * torch.rand(B, generator=g, device=_DEV)).to(torch.int32)
        lens[0] = 0 if B > 1 else case["far"]
        s["lens"] = lens
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import gated_deltanet_chunked_gdn_amd as gdn

        s["gdn"] = gdn
        # the packed offsets as a serving loop holds them: built once for a batch
        s["seqs"] = gdn.SeqLens(s["offsets"], _DEV) if s["packed"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    gdn, case, seqs = s["gdn"], s["case"], s["seqs"]
    op = case["op"]
    if op == "glr":
        y, h = gdn.glr_fwd(s["x"], s["r"], s["i"], s["lam"], z=s["z"], h0=s["state"], cu_seqlens=seqs)
        return {"y": y, "state": h}
    if op == "glr_train":
        y, h, saved = gdn.glr_fwd_save(s["x"], s["r"], s["i"], s["lam"], z=s["z"], h0=s["state"], cu_seqlens=seqs)
        return {"y": y, "state": h, **gdn.glr_bwd_saved(s["x"], s["r"], s["i"], s["lam"], s["dy"], saved, z=s["z"], dh_final=s["dstate"],
                                                        cu_seqlens=seqs, want_dh0=s["state"] is not None)}
    if op == "glr_step":
        return {"y": gdn.glr_step(s["x"], s["r"], s["i"], s["lam"], s["state"], z=s["z"]), "state": s["state"]}
    if op.startswith("rope"):
        how = dict(norm=case["norm"], eps=s["eps"], wq=s["wq"], wk=s["wk"], interleaved=case["inter"])
        q, k = gdn.rope_fwd(s["q"], s["k"], s["freq"], s["pos"], **how)
        if op == "rope":
            return {"q": q, "k": k}
        return {"q": q, "k": k, **gdn.rope_bwd(s["q"], s["k"], s["freq"], s["dq"], s["dk"], s["pos"], **how)}
    how = dict(sinks=case["S"], scale=s["scale"])
    if op == "swa":
        o = gdn.swa_fwd(s["q"], s["k"], s["v"], case["W"], cu_seqlens=seqs, **how)
        gdn.swa_fill(s["k"], s["v"], s["kc"], s["vc"], sinks=case["S"], cu_seqlens=seqs)
        return {"o": o, "kc": s["kc"], "vc": s["vc"]}
    if op == "swa_train":
        o, lse = gdn.swa_fwd(s["q"], s["k"], s["v"], case["W"], cu_seqlens=seqs, return_lse=True, **how)
        return {"o": o, **gdn.swa_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], case["W"], cu_seqlens=seqs, **how)}
    o = gdn.swa_step(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["lens"], **how)
    return {"o": o, "kc": s["kc"], "vc": s["vc"]}


# ----------------------------------------------------------------------------- plain forms, fp32

def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("glr"):
        return _plain_glr(s)
    if op.startswith("rope"):
        return _plain_rope(s)
    return _plain_step(s) if op == "swa_step" else _plain_swa(s)


def _sequence_of_rows(cu, rows):
    return torch.searchsorted(cu, torch.arange(rows, device=_DEV), right=True) - 1


def _running(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0, by doubling."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_glr(s):
    case, shape, io = s["case"], s["x"].shape, s["x"].dtype
    rows, C = shape[0] * shape[1], shape[2]
    x, r, i = (s[k].reshape(rows, C).float() for k in ("x", "r", "i"))
    soft = torch.clamp(s["lam"], min=0) + torch.log1p(torch.exp(-s["lam"].abs()))
    gate_r, gate_i = torch.sigmoid(r), torch.sigmoid(i)
    la = -8.0 * soft * gate_r
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    b = m * gate_i * x
    h0 = s["state"] if s["state"] is not None else torch.zeros(s["cu"].numel() - 1, C, device=_DEV)
    if case["op"] == "glr_step":
        h = a * h0 + b
        s["state"].copy_(h)
        y = h if s["z"] is None else h * (s["z"].reshape(rows, C).float() * torch.sigmoid(s["z"].reshape(rows, C).float()))
        return {"y": y.to(io).reshape(shape), "state": s["state"]}
    first, some = s["cu"][:-1], s["cu"][1:] > s["cu"][:-1]
    starts, ends = first[some], s["cu"][1:][some] - 1
    cut = a.clone()
    cut[starts] = 0
    h = b.clone()
    h[starts] += a[starts] * h0[some]
    h = _running(cut, h)
    z = sig = None
    y = h
    if s["z"] is not None:
        z = s["z"].reshape(rows, C).float()
        sig = torch.sigmoid(z)
        y = h * z * sig
    last = h0.clone()
    last[some] = h[ends]
    out = {"y": y.to(io).reshape(shape), "state": last}
    if case["op"] == "glr":
        return out
    dy = s["dy"].reshape(rows, C).float()
    dlast = s["dstate"] if s["dstate"] is not None else torch.zeros_like(h0)
    d = dy.clone() if z is None else dy * z * sig
    d[ends] += dlast[some]
    after = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    grad = _running(after.flip(0), d.flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[starts] = h0[some]
    # with la times its own gradient every quotient stays bounded: m ~ sqrt(-2 la) where la is small
    e = grad * (a * la * before - a * a * torch.where(m > 0, la / m, 0) * gate_i * x)
    dh0 = dlast.clone()
    dh0[some] = a[starts] * grad[starts]
    rest = {"dx": grad * m * gate_i, "dr": e * (1 - gate_r), "di": grad * m * x * gate_i * (1 - gate_i)}
    if z is not None:
        rest["dz"] = dy * h * sig * (1 + z * (1 - sig))
    out.update({k: v.to(io).reshape(shape) for k, v in rest.items()})
    out.update(dlam=e.sum(0) * torch.sigmoid(s["lam"]) / soft, dh0=dh0 if s["state"] is not None else None)
    return out


def _turn(x, cos, sin, inter):
    """The first pairs of the last dimension turned by their angles, what lies behind them as it is."""
    n = cos.shape[-1]
    if inter:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([u * cos - v * sin, v * cos + u * sin], dim=-1).flatten(-2)
    else:
        u, v = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([u * cos - v * sin, v * cos + u * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * n:]], dim=-1)


def _plain_rope(s):
    case, io = s["case"], s["q"].dtype
    angle = s["pos"].double().unsqueeze(-1) * s["freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(-2), torch.sin(angle).float().unsqueeze(-2)

    def norm(x, w):
        if case["norm"] is None:
            return torch.ones_like(x[..., :1]), x, x
        square = (x * x).sum(-1, keepdim=True)
        inv = 1 / torch.sqrt(square / x.shape[-1] + s["eps"]) if case["norm"] == "rms" else 1 / torch.clamp(torch.sqrt(square), min=1e-30)
        return inv, x * inv, x * inv * w if w is not None else x * inv

    iq, uq, nq = norm(s["q"].float(), s["wq"])
    ik, uk, nk = norm(s["k"].float(), s["wk"])
    out = {"q": _turn(nq, cos, sin, case["inter"]).to(io), "k": _turn(nk, cos, sin, case["inter"]).to(io)}
    if case["op"] == "rope":
        return out

    def back(d, inv, unit, w):
        d = _turn(d.float(), cos, -sin, case["inter"])
        dw = (d * unit).sum((0, 1, 2)) if w is not None else None
        if w is not None:
            d = d * w
        if case["norm"] is None:
            return d.to(io), dw
        along = (d * unit).sum(-1, keepdim=True)
        return (inv * (d - unit * (along / d.shape[-1] if case["norm"] == "rms" else along))).to(io), dw

    (out["dq"], out["dwq"]), (out["dk"], out["dwk"]) = back(s["dq"], iq, uq, s["wq"]), back(s["dk"], ik, uk, s["wk"])
    return out


def _plain_swa(s):
    """Blocks of at least a window's queries, each against its own and the previous block's keys and its sequence's first tokens."""
    case, io, scale = s["case"], s["q"].dtype, s["scale"]
    B, T, Hq, D = s["q"].shape
    Hk, W, S = case["Hk"], case["W"], case["S"]
    rows, group = B * T, Hq // Hk
    size = min(max(W, 64), rows)
    count = -(-rows // size)
    pad = count * size - rows
    seq, cu = _sequence_of_rows(s["cu"], rows), s["cu"]

    def queries(x):  # (count, Hk, group * size, D)
        x = torch.nn.functional.pad(x.reshape(rows, Hk, group, D).float(), (0, 0, 0, 0, 0, 0, 0, pad))
        return x.reshape(count, size, Hk, group, D).permute(0, 2, 3, 1, 4).reshape(count, Hk, group * size, D)

    index = torch.arange(count, device=_DEV).unsqueeze(-1) * size
    near = index - size + torch.arange(2 * size, device=_DEV)  # rows of a block's keys
    inside = (near >= 0) & (near < rows)
    near = near.clamp(0, rows - 1)
    mine = (index + torch.arange(size, device=_DEV)).clamp(max=rows - 1)  # rows of a block's queries
    q, k, v = queries(s["q"]), s["k"].reshape(rows, Hk, D).float(), s["v"].reshape(rows, Hk, D).float()
    kn, vn = (x[near].permute(0, 2, 1, 3).contiguous() for x in (k, v))
    ok = inside.unsqueeze(1) & (seq[near].unsqueeze(1) == seq[mine].unsqueeze(2)) & (near.unsqueeze(1) <= mine.unsqueeze(2)) & (
        near.unsqueeze(1) > mine.unsqueeze(2) - W)
    # first tokens that the window has left behind, gathered for every query
    first = cu[seq][mine].unsqueeze(-1) + torch.arange(S, device=_DEV)
    ok_first = first <= mine.unsqueeze(-1) - W
    first = first.clamp(max=rows - 1)
    spread = lambda t: t.unsqueeze(1).unsqueeze(1).expand(count, Hk, group, size, t.shape[-1]).reshape(count, Hk, group * size, t.shape[-1])  # noqa: E731
    kf, vf = (x[first].permute(0, 3, 1, 2, 4) for x in (k, v))  # (count, Hk, size, S, D)
    q5 = q.reshape(count, Hk, group, size, 1, D)
    scores = torch.cat([torch.matmul(q, kn.transpose(-1, -2)), (q5 * kf.unsqueeze(2)).sum(-1).reshape(count, Hk, group * size, S)], dim=-1) * scale
    scores = torch.where(torch.cat([spread(ok), spread(ok_first)], dim=-1), scores, -math.inf)
    top = scores.max(-1, keepdim=True).values
    p = torch.exp(scores - top)
    p = p / p.sum(-1, keepdim=True)
    pn, pf = p[..., :2 * size], p[..., 2 * size:]
    weigh = lambda pf, x: (pf.reshape(count, Hk, group, size, S, 1) * x.unsqueeze(2)).sum(-2).reshape(count, Hk, group * size, D)  # noqa: E731
    back = lambda x: x.reshape(count, Hk, group, size, D).permute(0, 3, 1, 2, 4).reshape(count * size, Hq, D)[:rows].reshape(B, T, Hq, D)  # noqa: E731
    o = torch.matmul(pn, vn) + weigh(pf, vf)
    out = {"o": back(o).to(io)}
    if case["op"] == "swa":
        # slots of the first tokens, then a ring of the last W behind them
        slot = torch.arange(S + W, device=_DEV)
        length = (cu[1:] - cu[:-1]).unsqueeze(-1)
        turn = length - 1 - S - (length - 1 - S - (slot - S)) % W  # the last token behind the first S that falls on the slot
        token = torch.where(slot < S, slot, turn + S)
        live = torch.where(slot < S, slot < length, turn >= 0).unsqueeze(-1).unsqueeze(-1)
        row = (cu[:-1].unsqueeze(-1) + token).clamp(0, rows - 1)
        for cache, x in ((s["kc"], s["k"]), (s["vc"], s["v"])):
            cache.copy_(torch.where(live, x.reshape(rows, Hk, D)[row], cache))
        return {**out, "kc": s["kc"], "vc": s["vc"]}
    do = queries(s["do"])
    dp = torch.cat([torch.matmul(do, vn.transpose(-1, -2)), (do.reshape(q5.shape) * vf.unsqueeze(2)).sum(-1).reshape(count, Hk, group * size, S)], dim=-1)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    dsn, dsf = ds[..., :2 * size], ds[..., 2 * size:]
    out["dq"] = back(torch.matmul(dsn, kn) + weigh(dsf, kf)).to(io)

    def keys(pn, pf, x):
        """The sum over queries of p x, at each key's row."""
        wide = torch.matmul(pn.transpose(-1, -2), x).permute(0, 2, 1, 3).reshape(-1, Hk, D)
        total = torch.zeros(rows, Hk, D, device=_DEV).index_add_(0, near.reshape(-1), wide * inside.reshape(-1, 1, 1))
        few = (pf.reshape(count, Hk, group, size, S, 1) * x.reshape(q5.shape)).sum(2).permute(0, 2, 3, 1, 4)
        return total.index_add_(0, first.reshape(-1), few.reshape(-1, Hk, D)).to(io).reshape(B, T, Hk, D)

    out["dk"], out["dv"] = keys(dsn, dsf, q), keys(pn, pf, do)
    return out


def _plain_step(s):
    case, io = s["case"], s["q"].dtype
    B, _, Hq, D = s["q"].shape
    Hk, W, S = case["Hk"], case["W"], case["S"]
    lens = s["lens"].long()
    slot = torch.where(lens < S, lens, S + (lens - S) % W)
    each = torch.arange(B, device=_DEV)
    s["kc"][each, slot] = s["k"].squeeze(1)
    s["vc"][each, slot] = s["v"].squeeze(1)
    at = torch.arange(S + W, device=_DEV)
    n = lens.unsqueeze(-1) + 1
    live = at < n  # the slots fill up in order
    q = s["q"].reshape(B, Hk, Hq // Hk, D).float()
    k, v = (s[c].float().permute(0, 2, 1, 3).contiguous() for c in ("kc", "vc"))
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    scores = torch.where(live.unsqueeze(1).unsqueeze(1), scores, -math.inf)
    p = torch.exp(scores - scores.max(-1, keepdim=True).values)
    o = torch.matmul(p / p.sum(-1, keepdim=True), v)
    return {"o": o.reshape(B, 1, Hq, D).to(io), "kc": s["kc"], "vc": s["vc"]}


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, io = case["op"], 2 if case["io"] == "bf16" else 4
    B, T = case["B"], case.get("T", 1)
    offsets = _offsets(case)
    n, rows = len(offsets) - 1, B * T
    if op.startswith("glr"):
        C, z = case["C"], int(case["z"])
        state = n * C * 4
        some = state if case.get("state", True) else 0
        wide = 4 + z  # x, r, i, z in, y out
        if op == "glr_train":  # those, dy in, dx, dr, di and dz out
            return {"bytes": (wide + 4 + z) * rows * C * io + 3 * some + state + 2 * C * 4, "flops": rows * C * (55 + 12 * z)}
        return {"bytes": wide * rows * C * io + some + state + C * 4, "flops": rows * C * (20 + 4 * z)}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if op.startswith("rope"):
        values = rows * (Hq + Hk) * D
        small = rows * 4 + case["R"] * 2 + (2 * D * 4 if case["norm"] == "rms" else 0)
        if op == "rope_train":  # q, k and their outputs' gradients in; outputs and gradients out
            return {"bytes": 5 * values * io + small, "flops": values * 18}
        return {"bytes": 2 * values * io + small, "flops": values * 7}
    W, S = case["W"], case["S"]
    if op == "swa_step":
        # ages are spread evenly up to `far`: slots in use on average, each read once, and the new row written
        full, far = S + W, case["far"]
        seen = B * (full - full * full / (2 * far) if full < far else far / 2 + 1) if B > 1 else min(full, far + 1)
        return {"bytes": (2 * seen * Hk + 4 * B * Hk + 2 * B * Hq) * D * io, "flops": 4 * seen * Hq * D}
    pairs = 0
    for a, b in zip(offsets, offsets[1:]):
        L = b - a
        inner = min(L, W)
        pairs += inner * (inner + 1) // 2 + max(0, L - W) * W
        if L > W:  # first tokens behind the window
            left = L - W
            pairs += min(left, S) * (min(left, S) + 1) // 2 + max(0, left - S) * S
    if op == "swa_train":
        return {"bytes": (4 * Hq + 4 * Hk) * rows * D * io, "flops": 14 * pairs * Hq * D}
    kept = sum(min(b - a, S + W) for a, b in zip(offsets, offsets[1:]))
    return {"bytes": ((2 * Hq + 2 * Hk) * rows + 2 * kept * Hk) * D * io, "flops": 4 * pairs * Hq * D}


# ----------------------------------------------------------------------------- definitions, fp64

def exact(case, seed):
    s = _inputs(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op.startswith("glr"):
        return _exact_glr(case, s)
    if op.startswith("rope"):
        return _exact_rope(case, s)
    return _exact_step(case, s) if op == "swa_step" else _exact_swa(case, s)


def _exact_glr(case, s):
    """Token by token."""
    x = s["x"]
    B, T, C = x.shape
    soft = torch.logaddexp(s["lam"], torch.zeros_like(s["lam"]))
    gr, gi = 1 / (1 + torch.exp(-s["r"])), 1 / (1 + torch.exp(-s["i"]))
    la = -8 * gr * soft
    a = torch.exp(la)
    m = (-torch.special.expm1(la + la)).sqrt()
    b = gi * x * m
    spans = list(zip(s["offsets"], s["offsets"][1:]))
    af, bf = a.view(-1, C), b.view(-1, C)
    h, before = torch.empty_like(bf), torch.empty_like(bf)
    last = torch.zeros(len(spans), C, dtype=torch.float64, device=_DEV)
    for n, (t0, t1) in enumerate(spans):
        state = s["state"][n] if s["state"] is not None else last[n].clone()
        for t in range(t0, t1):
            before[t] = state
            state = torch.addcmul(bf[t], af[t], state, out=h[t])
        last[n] = state
    h, before = h.view_as(x), before.view_as(x)
    y = h if s["z"] is None else h * s["z"] / (1 + torch.exp(-s["z"]))
    if case["op"] != "glr_train":
        return {"y": y, "state": last}
    gz = None if s["z"] is None else 1 / (1 + torch.exp(-s["z"]))
    into = (s["dy"] if gz is None else s["dy"] * s["z"] * gz).reshape(-1, C)
    total = torch.empty_like(into)
    dh0 = torch.zeros_like(last)
    for n, (t0, t1) in enumerate(spans):
        back = s["dstate"][n] if s["dstate"] is not None else dh0[n].clone()
        for t in range(t1 - 1, t0 - 1, -1):
            torch.add(into[t], back, out=total[t])
            back = total[t] * af[t]
        dh0[n] = back
    total = total.view_as(x)
    dla = total * (a * before - gi * x * a * a / m)
    out = {"y": y, "state": last, "dx": total * gi * m, "dr": dla * -8 * soft * gr * (1 - gr), "di": total * m * x * gi * (1 - gi),
           "dlam": (dla * -8 * gr).sum((0, 1)) / (1 + torch.exp(-s["lam"])), "dh0": dh0 if s["state"] is not None else None}
    if gz is not None:
        out["dz"] = s["dy"] * h * (gz + s["z"] * gz * (1 - gz))
    return out


def _exact_rope(case, s):
    """Pairs as complex numbers, the gradient through the explicit Jacobian of the norm."""
    R, D = case["R"], case["D"]
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV), s["pos"].double()[..., None] * s["freq"])[:, :, None]

    def spin(x, by):
        head = x[..., :R].reshape(*x.shape[:-1], R // 2, 2) if case["inter"] else torch.stack(x[..., :R].chunk(2, -1), -1)
        head = torch.view_as_real(torch.view_as_complex(head.contiguous()) * by)
        head = head.flatten(-2) if case["inter"] else torch.cat([head[..., 0], head[..., 1]], -1)
        return torch.cat([head, x[..., R:]], -1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name], s["w" + name]
        if case["norm"] == "rms":
            length = (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt()
        elif case["norm"] == "l2":
            length = x.norm(dim=-1, keepdim=True).clamp(min=1e-30)
        else:
            length = torch.ones_like(x[..., :1])
        scaled = x / length * (w if w is not None else 1)
        out[name] = spin(scaled, phase)
        if case["op"] == "rope_train":
            d = spin(s["d" + name], phase.conj())
            dw = (d * x / length).sum((0, 1, 2)) if w is not None else None
            d = d * w if w is not None else d
            # length's own derivative: x / length, over D of them for the mean
            share = {"rms": 1 / D, "l2": 1.0, None: 0.0}[case["norm"]]
            out["d" + name] = d / length - share * x * (d * x).sum(-1, keepdim=True) / length ** 3
            out["dw" + name] = dw
    return out


def _seen(i, j, W, S):
    return (j <= i) & ((j > i - W) | (j < S))


def _exact_swa(case, s):
    """Every sequence and query head alone, over whole rows of scores."""
    q, k, v = (s[x].reshape(-1, s[x].shape[2], case["D"]) for x in "qkv")
    train = case["op"] == "swa_train"
    W, S, group = case["W"], case["S"], case["Hq"] // case["Hk"]
    o = torch.empty_like(q)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t0, t1 in zip(s["offsets"], s["offsets"][1:]):
        at = torch.arange(t1 - t0, device=_DEV)
        mask = ~_seen(at[:, None], at, W, S)
        for h in range(case["Hq"] if t1 > t0 else 0):
            qs, ks, vs = q[t0:t1, h], k[t0:t1, h // group], v[t0:t1, h // group]
            p = torch.softmax((qs @ ks.T * s["scale"]).masked_fill(mask, -math.inf), -1)
            o[t0:t1, h] = p @ vs
            if train:
                do = s["do"].reshape(q.shape)[t0:t1, h]
                dv[t0:t1, h // group] += p.T @ do
                dp = do @ vs.T
                ds = p * (dp - (do * o[t0:t1, h]).sum(-1, keepdim=True)) * s["scale"]
                dq[t0:t1, h] = ds @ ks
                dk[t0:t1, h // group] += ds.T @ qs
    if train:
        return {"o": o.view_as(s["q"]), "dq": dq.view_as(s["q"]), "dk": dk.view_as(s["k"]), "dv": dv.view_as(s["v"])}
    for n, (t0, t1) in enumerate(zip(s["offsets"], s["offsets"][1:])):
        for cache, rows in ((s["kc"], k), (s["vc"], v)):
            head = min(S, t1 - t0)
            cache[n, :head] = rows[t0:t0 + head]
            late = torch.arange(max(S, t1 - t0 - W), max(S, t1 - t0), device=_DEV)
            cache[n, S + (late - S) % W] = rows[t0 + late]
    return {"o": o.view_as(s["q"]), "kc": s["kc"], "vc": s["vc"]}


def _exact_step(case, s):
    W, S, group = case["W"], case["S"], case["Hq"] // case["Hk"]
    o = torch.empty_like(s["q"])
    for n, length in enumerate(s["lens"].tolist()):
        slot = length if length < S else S + (length - S) % W
        s["kc"][n, slot], s["vc"][n, slot] = s["k"][n, 0], s["v"][n, 0]
        # every token the new one sees, by its slot
        late = torch.arange(max(S, length + 1 - W), max(S, length + 1), device=_DEV)
        slots = torch.cat([torch.arange(min(S, length + 1), device=_DEV), S + (late - S) % W])
        k, v = (s[c][n, slots].repeat_interleave(group, 1) for c in ("kc", "vc"))
        p = torch.softmax(torch.einsum("hd,khd->hk", s["q"][n, 0], k) * s["scale"], -1)
        o[n, 0] = torch.einsum("hk,khd->hd", p, v)
    return {"o": o, "kc": s["kc"], "vc": s["vc"]}
