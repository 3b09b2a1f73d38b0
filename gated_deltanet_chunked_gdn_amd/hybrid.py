"""Python entry points of the operators that hybrid models put next to the delta rule,
over libgdn's C ABI (include/gdn.h): the gated linear recurrence, the norm and rotation of
queries and keys, and attention over a sliding window.  As in ``layer``, PyTorch supplies
device memory and the current stream, and every step of the computation runs in libgdn's
HIP kernels.

    y, h     = glr_fwd(x, r, i, lam, z=None, h0=None)
    y, h, saved = glr_fwd_save(...)
    grads    = glr_bwd_saved(x, r, i, lam, dy, saved, ...)
    y        = glr_step(x, r, i, lam, state, z=None)  # one token, state updated in place

    q, k     = rope_fwd(q, k, inv_freq, positions=None, norm="rms", wq=None, wk=None)
    grads    = rope_bwd(q, k, inv_freq, dq_out, dk_out, positions=None, ...)

    o        = swa_fwd(q, k, v, window, sinks=0)      # with return_lse: (o, lse)
    grads    = swa_bwd(q, k, v, o, lse, do, window, sinks=0)
    swa_fill(k, v, kcache, vcache, sinks=0)           # a prompt's keys and values
    o        = swa_step(q, k, v, kcache, vcache, lens, sinks=0)  # one token, cache updated in place

Tensors are contiguous; q, k and v of the last two operators may also be columns of
contiguous rows, as a projection leaves them side by side, with up to 2^21 values from
token to token (for single tokens: from sequence to sequence; a slice of one token out of
longer sequences lies further apart and has to be made contiguous).  Activations are bf16
or fp32 (one dtype a call), parameters and recurrent states fp32.
Packed sequences: B == 1 and ``cu_seqlens`` the N + 1 offsets, best built once as a
``SeqLens``.  Outputs and gradients that were not asked for are None.  A ``workspace``
holds nothing between calls, but calls that may overlap (on two streams, in graphs
replayed at once) need one each; without one a call takes a fresh buffer.

As in ``layer``, no call records anything for autograd: outputs carry no history, a tensor
that is updated in place keeps its version, and gradients come from the ``_bwd`` calls.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as nat
from .layer import _F32, _buffer, _call, _first, _may, _packed, _result, _want
from .ops import _IO


def _problem(kind, sizes, *rest):
    """A problem whose sizes 32 bits hold (ctypes would cut them off)."""
    if max(sizes) >= 1 << 31:
        raise ValueError(f"a size of {max(sizes)} is more than the library's 32 bits hold")
    return kind(*sizes, *rest)


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# a problem of dense tensors: the same sizes give the same (never written) structure
_dense = functools.lru_cache(maxsize=256)(_problem)


def _size(name, prob, *args):
    n = ctypes.c_size_t(0)
    nat.check(getattr(nat.load(), name)(prob, *args, n), name)
    return n.value


# --------------------------------------------------------------------------- gated linear recurrence

def _glr_problem(x, c, cu_seqlens):
    """(device index, offsets, problem)"""
    dev = _first(x, "x", 3, "x must be (B, T, C)")
    B, T, C = x.shape
    io, c = _IO[x.dtype], float(c)
    if cu_seqlens is None:
        return dev, None, _dense(nat.GlrProblem, (B, T, C, B), None, None, io, c)
    s = _packed(cu_seqlens, dev)
    return dev, s, _problem(nat.GlrProblem, (B, T, C, s.num_seqs), s.host.ctypes.data, s.dev.data_ptr(), io, c)


def _glr_inputs(x, r, i, lam, z, dev):
    xs, io = x.shape, x.dtype
    return (_want(x, xs, io, dev, "x"), _want(r, xs, io, dev, "r"), _want(i, xs, io, dev, "i"),
            _want(lam, (xs[2],), _F32, dev, "lam"), _may(z, xs, io, dev, "z"))


def _glr_size(prob, pass_):
    if not prob.cu_seqlens_host:
        return _dense_glr_size(prob.B, prob.T, prob.C, prob.io_dtype, prob.c, pass_)
    return _size("gdn_glr_workspace_size", prob, pass_)


@functools.lru_cache(maxsize=1024)
def _dense_glr_size(B, T, C, io, c, pass_):
    return _size("gdn_glr_workspace_size", nat.GlrProblem(B, T, C, B, None, None, io, c), pass_)


def glr_buffers(x, cu_seqlens=None):
    """Sizes in bytes of the buffers the recurrence takes: dict forward (workspace of
    glr_fwd and glr_fwd_save), saved, backward (workspace of glr_bwd_saved)."""
    _, seqs, prob = _glr_problem(x, 8.0, cu_seqlens)  # seqs: keeps the offsets alive
    return {"forward": _glr_size(prob, nat.GDN_GLR_FWD), "saved": _glr_size(prob, nat.GDN_GLR_SAVED),
            "backward": _glr_size(prob, nat.GDN_GLR_BWD)}


def _glr_fwd(save, x, r, i, lam, z, h0, c, cu_seqlens, output_final_state, out, final_state_out, saved, workspace):
    dev, seqs, prob = _glr_problem(x, c, cu_seqlens)  # seqs: keeps the offsets alive
    ins = _glr_inputs(x, r, i, lam, z, dev)
    shape = (prob.num_seqs, prob.C)
    h0p = _may(h0, shape, _F32, dev, "h0")
    y, yptr = _result(out, x, dev)
    h = final_state_out
    if h is None and output_final_state:
        h = lam.new_empty(shape)
    outs = (yptr, _may(h, shape, _F32, dev, "final_state_out"))
    buf, ws, nws = _buffer(workspace, _glr_size(prob, nat.GDN_GLR_FWD), dev, "workspace")
    if not save:
        _call(dev, "gdn_glr_fwd", prob, *ins, h0p, *outs, ws, nws)
        return y, h
    saved, sv, nsv = _buffer(saved, _glr_size(prob, nat.GDN_GLR_SAVED), dev, "saved")
    _call(dev, "gdn_glr_fwd_save", prob, *ins, h0p, *outs, sv, nsv, ws, nws)
    return y, h, saved


def glr_fwd(x, r, i, lam, z=None, h0=None, c: float = 8.0, cu_seqlens=None, output_final_state: bool = True, out=None,
            final_state_out=None, workspace=None):
    """Gated linear recurrence (gdn_glr_fwd): x, r, i, z (B, T, C) of the io dtype, the
    gates before their sigmoid; lam (C,) fp32; ``h0`` (sequences, C) fp32 or None (zero).
    Returns (y, h_final or None)."""
    return _glr_fwd(False, x, r, i, lam, z, h0, c, cu_seqlens, output_final_state, out, final_state_out, None, workspace)


def glr_fwd_save(x, r, i, lam, z=None, h0=None, c: float = 8.0, cu_seqlens=None, saved=None, workspace=None):
    """glr_fwd that also keeps what the backward needs (gdn_glr_fwd_save).  Returns
    (y, h_final, saved); pass ``saved`` to glr_bwd_saved with the same inputs."""
    return _glr_fwd(True, x, r, i, lam, z, h0, c, cu_seqlens, True, None, None, saved, workspace)


def glr_bwd_saved(x, r, i, lam, dy, saved, z=None, dh_final=None, c: float = 8.0, cu_seqlens=None, want_dh0: bool = True,
                  workspace=None):
    """Backward of glr_fwd_save (gdn_glr_bwd_saved) with the same inputs and cu_seqlens.
    Returns dict dx, dr, di, dlam, dz (None without z), dh0."""
    dev, seqs, prob = _glr_problem(x, c, cu_seqlens)  # seqs: keeps the offsets alive
    ins = _glr_inputs(x, r, i, lam, z, dev)
    shape = (prob.num_seqs, prob.C)
    dyp, dhp = _want(dy, x.shape, x.dtype, dev, "dy"), _may(dh_final, shape, _F32, dev, "dh_final")
    if saved is None and _glr_size(prob, nat.GDN_GLR_SAVED):
        raise ValueError("saved must be the buffer glr_fwd_save filled")
    _, sv, nsv = _buffer(saved, 0, dev, "saved")
    buf, ws, nws = _buffer(workspace, _glr_size(prob, nat.GDN_GLR_BWD), dev, "workspace")
    out = {"dx": torch.empty_like(x), "dr": torch.empty_like(x), "di": torch.empty_like(x), "dlam": torch.empty_like(lam),
           "dz": torch.empty_like(x) if z is not None else None, "dh0": lam.new_empty(shape) if want_dh0 else None}
    _call(dev, "gdn_glr_bwd_saved", prob, *ins, dyp, dhp, sv, nsv, *(t.data_ptr() if t is not None else None for t in out.values()),
          ws, nws)
    return out


def glr_step(x, r, i, lam, state, z=None, c: float = 8.0, out=None):
    """One token of glr_fwd for every sequence (gdn_glr_step): x, r, i, z (B, 1, C);
    ``state`` (B, C) fp32 is updated in place.  Returns y."""
    dev, _, prob = _glr_problem(x, c, None)
    if prob.T != 1:
        raise ValueError("x must be (B, 1, C)")
    ins = _glr_inputs(x, r, i, lam, z, dev)
    s = _want(state, (prob.B, prob.C), _F32, dev, "state")
    y, yptr = _result(out, x, dev)
    _call(dev, "gdn_glr_step", prob, *ins, s, yptr)
    return y


# --------------------------------------------------------------------------- norm and rotation

_NORM = {None: nat.GDN_ROPE_NONE, "none": nat.GDN_ROPE_NONE, "rms": nat.GDN_ROPE_RMS, "l2": nat.GDN_ROPE_L2}
_I32 = torch.int32


def _rows(t, shape, dtype, dev, name):
    """(address, values from token to token) of a (B, T, H, D) tensor whose tokens' heads and
    values are contiguous and whose tokens lie evenly apart: a contiguous one, or a view of
    the columns of a contiguous (B, T, more) one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.is_contiguous():
        return t.data_ptr(), shape[2] * shape[3]
    B, T, H, D = shape
    sb, st, sh, sd = t.stride()
    if T == 1:  # a token's own stride says nothing: the rows of the batch count
        st = sb if B > 1 else H * D
    if (sd != 1 and D > 1) or (sh != D and H > 1) or st < H * D or (B > 1 and sb != T * st):
        raise ValueError(f"{name} must be contiguous, or a view of the columns of contiguous rows (strides {t.stride()})")
    return t.data_ptr(), st


def _rope_problem(q, k, inv_freq, norm, eps, interleaved):
    """(device index, problem, addresses of q and k)"""
    what = "q must be (B, T, Hq, D) and k (B, T, Hk, D)"
    dev = _first(q, "q", 4, what)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError(what)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be an (R / 2,) tensor")
    if norm not in _NORM:
        raise ValueError(f"norm must be one of {sorted(map(str, _NORM))}")
    B, T, Hq, D = q.shape
    Hk, io = k.shape[2], q.dtype
    qp, qs = _rows(q, q.shape, io, dev, "q")
    kp, ks = _rows(k, (B, T, Hk, D), io, dev, "k")
    prob = _dense(nat.RopeProblem, (B, T, Hq, Hk, D, 2 * inv_freq.shape[0]), _NORM[norm], int(bool(interleaved)), _IO[io],
                  float(eps), qs, ks)
    return dev, prob, qp, kp


def _rope_inputs(p, inv_freq, positions, wq, wk, dev):
    return (_want(inv_freq, (p.R // 2,), _F32, dev, "inv_freq") or None, _may(positions, (p.B, p.T), _I32, dev, "positions"),
            _may(wq, (p.D,), _F32, dev, "wq"), _may(wk, (p.D,), _F32, dev, "wk"))


def rope_fwd(q, k, inv_freq, positions=None, norm="rms", eps: float = 1e-6, wq=None, wk=None, interleaved: bool = False,
             q_out=None, k_out=None):
    """Norm of queries and keys per head and rotation by position (gdn_rope_fwd): q
    (B, T, Hq, D), k (B, T, Hk, D) of the io dtype, contiguous or columns of contiguous
    rows; inv_freq (R / 2,) fp32; ``positions`` (B, T) int32 or None (0 .. T - 1); ``norm``
    "rms" (with weights wq, wk (D,) fp32 or None), "l2" or None.  Returns (q, k)."""
    dev, prob, qp, kp = _rope_problem(q, k, inv_freq, norm, eps, interleaved)
    ins = _rope_inputs(prob, inv_freq, positions, wq, wk, dev)
    outs = []
    for out, like, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        out = _like(like) if out is None else out
        outs.append((out, _want(out, like.shape, like.dtype, dev, name)))
    _call(dev, "gdn_rope_fwd", prob, qp, kp, *ins, outs[0][1], outs[1][1])
    return outs[0][0], outs[1][0]


def rope_bwd(q, k, inv_freq, dq_out, dk_out, positions=None, norm="rms", eps: float = 1e-6, wq=None, wk=None,
             interleaved: bool = False, workspace=None):
    """Backward of rope_fwd (gdn_rope_bwd).  Returns dict dq, dk, dwq, dwk (None without
    their weights)."""
    dev, prob, qp, kp = _rope_problem(q, k, inv_freq, norm, eps, interleaved)
    ins = _rope_inputs(prob, inv_freq, positions, wq, wk, dev)
    grads = (_want(dq_out, q.shape, q.dtype, dev, "dq_out"), _want(dk_out, k.shape, q.dtype, dev, "dk_out"))
    need = _size("gdn_rope_workspace_size", prob) if wq is not None or wk is not None else 0
    buf, ws, nws = _buffer(workspace, need, dev, "workspace")
    out = {name: _like(t) if t is not None else None for name, t in (("dq", q), ("dk", k), ("dwq", wq), ("dwk", wk))}
    _call(dev, "gdn_rope_bwd", prob, qp, kp, *ins, *grads, *(t.data_ptr() if t is not None else None for t in out.values()),
          ws, nws)
    return out


# --------------------------------------------------------------------------- window attention

def _swa_problem(q, k, v, window, sinks, scale, cu_seqlens):
    """(device index, offsets, problem, addresses of q, k, v)"""
    what = "q must be (B, T, Hq, D) and k, v (B, T, Hk, D)"
    dev = _first(q, "q", 4, what)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError(what)
    B, T, Hq, D = q.shape
    Hk, io = k.shape[2], q.dtype
    (qp, qs), (kp, ks), (vp, vs) = (_rows(q, q.shape, io, dev, "q"), _rows(k, (B, T, Hk, D), io, dev, "k"),
                                    _rows(v, (B, T, Hk, D), io, dev, "v"))
    sizes, rest = (B, T, Hq, Hk, D, int(window), int(sinks)), (_IO[io], float(scale), qs, ks, vs)
    if cu_seqlens is None:
        return dev, None, _dense(nat.SwaProblem, sizes + (B,), None, None, *rest), (qp, kp, vp)
    s = _packed(cu_seqlens, dev)
    return dev, s, _problem(nat.SwaProblem, sizes + (s.num_seqs,), s.host.ctypes.data, s.dev.data_ptr(), *rest), (qp, kp, vp)


def swa_fwd(q, k, v, window: int, sinks: int = 0, scale: float = 1.0, cu_seqlens=None, out=None, return_lse: bool = False):
    """Causal attention over a sliding window whose first tokens stay visible
    (gdn_swa_fwd): q (B, T, Hq, D), k, v (B, T, Hk, D) of the io dtype, Hq a multiple of Hk,
    D 64 or 128.  A query sees the last ``window`` tokens, itself among them, and the first
    ``sinks`` of its sequence.  Returns o, or (o, lse) with lse (B, T, Hq) fp32."""
    dev, seqs, prob, ptrs = _swa_problem(q, k, v, window, sinks, scale, cu_seqlens)  # seqs: keeps the offsets alive
    o = _like(q) if out is None else out
    optr = _want(o, q.shape, q.dtype, dev, "out")
    lse = torch.empty(q.shape[:3], dtype=_F32, device=dev) if return_lse else None
    _call(dev, "gdn_swa_fwd", prob, *ptrs, optr, lse.data_ptr() if return_lse else None)
    return (o, lse) if return_lse else o


def swa_bwd(q, k, v, o, lse, do, window: int, sinks: int = 0, scale: float = 1.0, cu_seqlens=None, workspace=None):
    """Backward of swa_fwd (gdn_swa_bwd) from its o and lse.  Returns dict dq, dk, dv."""
    dev, seqs, prob, ptrs = _swa_problem(q, k, v, window, sinks, scale, cu_seqlens)  # seqs: keeps the offsets alive
    ins = (_want(o, q.shape, q.dtype, dev, "o"), _want(lse, q.shape[:3], _F32, dev, "lse"), _want(do, q.shape, q.dtype, dev, "do"))
    buf, ws, nws = _buffer(workspace, _size("gdn_swa_workspace_size", prob, nat.GDN_SWA_BWD), dev, "workspace")
    out = {name: _like(t) for name, t in (("dq", q), ("dk", k), ("dv", v))}
    _call(dev, "gdn_swa_bwd", prob, *ptrs, *ins, *(t.data_ptr() for t in out.values()), ws, nws)
    return out


def _cache_slots(kcache, sinks):
    if not isinstance(kcache, torch.Tensor) or kcache.dim() != 4 or kcache.shape[1] <= sinks:
        raise ValueError("kcache must be (sequences, sinks + window, Hk, D)")
    return kcache.shape[1]


def swa_fill(k, v, kcache, vcache, sinks: int = 0, cu_seqlens=None):
    """Writes the keys and values of prompts into the caches that swa_step continues
    (gdn_swa_fill): kcache, vcache (sequences, sinks + window, Hk, D) of the io dtype, whose
    size says the window.  Slots that the prompts do not reach are left as they were."""
    slots = _cache_slots(kcache, sinks)
    dev, seqs, prob, ptrs = _swa_problem(k, k, v, slots - sinks, sinks, 1.0, cu_seqlens)  # seqs: keeps the offsets alive
    shape = (prob.num_seqs, slots, prob.Hk, prob.D)
    _call(dev, "gdn_swa_fill", prob, *ptrs[1:], _want(kcache, shape, k.dtype, dev, "kcache"), _want(vcache, shape, k.dtype, dev, "vcache"))


def swa_step(q, k, v, kcache, vcache, lens, sinks: int = 0, scale: float = 1.0, out=None, workspace=None):
    """One token of swa_fwd for every sequence (gdn_swa_step): q (B, 1, Hq, D), k, v
    (B, 1, Hk, D); kcache, vcache (B, sinks + window, Hk, D), updated in place; ``lens``
    (B,) int32: the tokens that each sequence had before, negative where its place is idle
    (o is zero there).  The caller adds one to lens behind its last layer.  Returns o."""
    slots = _cache_slots(kcache, sinks)
    dev, _, prob, ptrs = _swa_problem(q, k, v, slots - sinks, sinks, scale, None)
    if prob.T != 1:
        raise ValueError("q must be (B, 1, Hq, D)")
    shape = (prob.B, slots, prob.Hk, prob.D)
    caches = (_want(kcache, shape, q.dtype, dev, "kcache"), _want(vcache, shape, q.dtype, dev, "vcache"))
    lp = _want(lens, (prob.B,), _I32, dev, "lens")
    o = _like(q) if out is None else out
    optr = _want(o, q.shape, q.dtype, dev, "out")
    need = _step_size(prob.B, prob.Hq, prob.Hk, prob.D, prob.window, prob.sinks, prob.io_dtype)
    buf, ws, nws = _buffer(workspace, need, dev, "workspace")
    _call(dev, "gdn_swa_step", prob, *ptrs, *caches, lp, optr, ws, nws)
    return o


@functools.lru_cache(maxsize=1024)
def _step_size(B, Hq, Hk, D, window, sinks, io):
    return _size("gdn_swa_workspace_size", nat.SwaProblem(B, 1, Hq, Hk, D, window, sinks, B, None, None, io, 1.0, 0, 0, 0), nat.GDN_SWA_STEP)
