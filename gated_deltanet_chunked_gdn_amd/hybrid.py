"""Python entry points of the operators that hybrid models put next to the delta rule,
over libgdn's C ABI (include/gdn.h): the gated linear recurrence.  As in ``layer``,
PyTorch supplies device memory and the current stream, and every step of the computation
runs in libgdn's HIP kernels.

    y, h     = glr_fwd(x, r, i, lam, z=None, h0=None)
    y, h, saved = glr_fwd_save(...)
    grads    = glr_bwd_saved(x, r, i, lam, dy, saved, ...)
    y        = glr_step(x, r, i, lam, state, z=None)  # one token, state updated in place

Activations are bf16 or fp32 (one dtype a call), parameters and recurrent states fp32.
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
    if saved is None:
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
