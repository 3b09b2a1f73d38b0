"""Python entry points of the layer operators over libgdn's C ABI (include/gdn.h):
the single-token step of the delta rule, the short causal convolution and the
selective state space scan.  As in ``ops``, PyTorch supplies device memory and the
current stream, and every step of the computation runs in libgdn's HIP kernels.

    o = step(q, k, v, g, beta, state)             # one token, state updated in place
    o = kda_step(q, k, v, g, beta, state)         # g (B, 1, H, Dk)
    y, state = conv_fwd(x, weight, bias, state0)
    grads    = conv_bwd(x, weight, dy, ...)
    y        = conv_step(x, weight, state, bias)  # one token, state updated in place
    y, h     = scan_fwd(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None)
    y, h, saved = scan_fwd_save(...)
    grads    = scan_bwd_saved(u, dt, A, Bm, Cm, dy, saved, ...)
    y        = scan_step(u, dt, A, Bm, Cm, state, ...)

Tensors are contiguous; activations are bf16 or fp32 (one dtype a call), parameters
and recurrent states fp32, the convolution's state the io dtype (it keeps input
rows).  Packed sequences: B == 1 and ``cu_seqlens`` the N + 1 offsets, best built
once as a ``SeqLens``.  Outputs and gradients that were not asked for are None.  A
``workspace`` holds nothing between calls, but calls that may overlap (on two streams,
in graphs replayed at once) need one each; without one a call takes a fresh buffer.

As in ``ops``, no call records anything for autograd: outputs carry no history, whatever
requires gradients, a tensor that is updated in place keeps its version, and gradients come
from the ``_bwd`` calls.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _native as nat
from .ops import _IO, _seqlens

# A single-token call is a few microseconds, so the checks are kept to what costs little:
# the device as its index, the raw current stream, problems by their sizes.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)

_ACT = {None: nat.GDN_ACT_NONE, "none": nat.GDN_ACT_NONE, "silu": nat.GDN_ACT_SILU}
_F32 = torch.float32


def _first(t, name, dims, what):
    """Index of the device of the tensor that the others have to share it with."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (got {t.device})")
    if t.dtype not in _IO:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if t.dim() != dims:
        raise ValueError(what)
    return t.get_device()


def _want(t, shape, dtype, dev, name):
    """The address of a contiguous tensor of this shape, dtype and device (index).  A host
    pointer that reached a kernel would be a GPU memory fault, which the C ABI cannot
    detect."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    raise ValueError(f"{name} must be contiguous with shape {tuple(shape)} (got {tuple(t.shape)})")


def _may(t, shape, dtype, dev, name):
    """_want, or None for an absent tensor."""
    return None if t is None else _want(t, shape, dtype, dev, name)


def _call(dev, name, *args):
    """The library call on the device's current stream, with that device current."""
    fn = getattr(nat.load(), name)
    if dev == _current_device():
        st = fn(*args, _current_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _current_stream(dev))
    if st:
        nat.check(st, name)


def _problem(kind, *fields):
    """A problem, its first five fields sizes that 32 bits hold (ctypes would cut them off)."""
    if max(fields[:5]) >= 1 << 31:
        raise ValueError(f"a size of {max(fields[:5])} is more than the library's 32 bits hold")
    return kind(*fields)


# a problem of dense tensors: the same sizes give the same (never written) structure
_dense = functools.lru_cache(maxsize=256)(_problem)


def _packed(cu_seqlens, dev):
    seqs = _seqlens(cu_seqlens, torch.device("cuda", dev))
    if seqs.dev.get_device() != dev:
        raise ValueError(f"cu_seqlens must be on cuda:{dev} (got {seqs.dev.device})")
    return seqs


def _buffer(buf, nbytes, dev, name):
    """(buffer, address, bytes) of a caller's uint8 buffer, or of a fresh one of the size
    the library asks for."""
    if buf is None:
        if not nbytes:
            return None, None, 0
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return buf, buf.data_ptr(), nbytes
    if not isinstance(buf, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if buf.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {buf.device})")
    if not buf.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return buf, buf.data_ptr(), buf.numel() * buf.element_size()


def _result(out, like, dev):
    """(tensor, address) of the caller's output or a fresh one like `like`."""
    if out is None:
        out = torch.empty_like(like)
        return out, out.data_ptr()
    return out, _want(out, like.shape, like.dtype, dev, "out")


# --------------------------------------------------------------------------- delta rule, one token

def _step(name, q, k, v, g, beta, state, scale, out, channel):
    what = "q and k must be (B, 1, H, Dk) and v (B, 1, H, Dv)"
    dev = _first(q, "q", 4, what)
    qs, io = q.shape, q.dtype
    B, one, H, Dk = qs
    if one != 1 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError(what)
    Dv = v.shape[3]
    gs = (B, 1, H)
    ptrs = (_want(q, qs, io, dev, "q"), _want(k, qs, io, dev, "k"), _want(v, (B, 1, H, Dv), io, dev, "v"),
            _want(g, qs if channel else gs, _F32, dev, "g"), _want(beta, gs, _F32, dev, "beta"),
            _want(state, (B, H, Dk, Dv), _F32, dev, "state"))
    o, optr = _result(out, v, dev)
    prob = _dense(nat.Problem, B, 1, H, Dk, Dv, B, None, None, _IO[io], float(scale), 64, 1, nat.GDN_PRECISION_IO)
    _call(dev, name, prob, *ptrs, optr)
    return o


def step(q, k, v, g, beta, state, scale: float = 1.0, out=None):
    """One token of the gated delta rule (gdn_step): q, k (B, 1, H, Dk), v (B, 1, H, Dv)
    of the io dtype, g, beta (B, 1, H) fp32; ``state`` (B, H, Dk, Dv) fp32 is updated in
    place.  Returns o, shaped like v."""
    return _step("gdn_step", q, k, v, g, beta, state, scale, out, False)


def kda_step(q, k, v, g, beta, state, scale: float = 1.0, out=None):
    """step with one log-decay per key channel (gdn_kda_step): g (B, 1, H, Dk) fp32."""
    return _step("gdn_kda_step", q, k, v, g, beta, state, scale, out, True)


# --------------------------------------------------------------------------- short causal convolution

def _conv_problem(x, weight, cu_seqlens, activation):
    """(device index, offsets, problem)"""
    dev = _first(x, "x", 3, "x must be (B, T, C)")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a (C, W) tensor")
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(map(str, _ACT))}")
    B, T, C = x.shape
    W, io, act = weight.shape[1], _IO[x.dtype], _ACT[activation]
    if cu_seqlens is None:
        return dev, None, _dense(nat.ConvProblem, B, T, C, W, B, None, None, io, act)
    s = _packed(cu_seqlens, dev)
    return dev, s, _problem(nat.ConvProblem, B, T, C, W, s.num_seqs, s.host.ctypes.data, s.dev.data_ptr(), io, act)


def _conv_inputs(x, weight, bias, dev):
    xs = x.shape
    C = xs[2]
    return (_want(x, xs, x.dtype, dev, "x"), _want(weight, (C, weight.shape[1]), _F32, dev, "weight"),
            _may(bias, (C,), _F32, dev, "bias"))


def conv_fwd(x, weight, bias=None, state0=None, cu_seqlens=None, activation: Optional[str] = "silu",
             output_final_state: bool = True, out=None, final_state_out=None):
    """Short causal depthwise convolution (gdn_conv_fwd): x (B, T, C) of the io dtype,
    weight (C, W) and bias (C,) fp32, W in 2..4; ``activation`` "silu" or None.
    ``state0`` (N, W - 1, C) of the io dtype holds the rows before every sequence
    (oldest first; None: zeros).  Returns (y, state_final or None)."""
    dev, seqs, prob = _conv_problem(x, weight, cu_seqlens, activation)  # seqs: keeps the offsets alive
    shape = (prob.num_seqs, prob.W - 1, prob.C)
    ins = _conv_inputs(x, weight, bias, dev)
    s0 = _may(state0, shape, x.dtype, dev, "state0")
    y, yptr = _result(out, x, dev)
    last = final_state_out
    if last is None and output_final_state:
        last = x.new_empty(shape)
    _call(dev, "gdn_conv_fwd", prob, *ins, s0, yptr, _may(last, shape, x.dtype, dev, "final_state_out"))
    return y, last


def conv_bwd(x, weight, dy, bias=None, state0=None, dstate_final=None, cu_seqlens=None,
             activation: Optional[str] = "silu", workspace=None):
    """Backward of conv_fwd (gdn_conv_bwd).  Returns dict dx, dweight, dbias (None
    without bias), dstate0 (None without state0)."""
    dev, seqs, prob = _conv_problem(x, weight, cu_seqlens, activation)  # seqs: keeps the offsets alive
    shape = (prob.num_seqs, prob.W - 1, prob.C)
    ins = _conv_inputs(x, weight, bias, dev)
    s0 = _may(state0, shape, x.dtype, dev, "state0")
    grads = (_want(dy, x.shape, x.dtype, dev, "dy"), _may(dstate_final, shape, x.dtype, dev, "dstate_final"))
    n = ctypes.c_size_t(0)
    nat.check(nat.load().gdn_conv_workspace_size(prob, n), "gdn_conv_workspace_size")
    buf, ws, nws = _buffer(workspace, n.value, dev, "workspace")
    out = {"dx": torch.empty_like(x), "dweight": torch.empty_like(weight),
           "dbias": torch.empty_like(bias) if bias is not None else None,
           "dstate0": torch.empty_like(state0) if state0 is not None else None}
    _call(dev, "gdn_conv_bwd", prob, *ins, s0, *grads, *(t.data_ptr() if t is not None else None for t in out.values()),
          ws, nws)
    return out


def conv_step(x, weight, state, bias=None, activation: Optional[str] = "silu", out=None):
    """One token of conv_fwd for every sequence (gdn_conv_step): x (B, 1, C); ``state``
    (B, W - 1, C) is shifted by one row in place.  Returns y."""
    dev, _, prob = _conv_problem(x, weight, None, activation)
    if prob.T != 1:
        raise ValueError("x must be (B, 1, C)")
    ins = _conv_inputs(x, weight, bias, dev)
    s = _want(state, (prob.B, prob.W - 1, prob.C), x.dtype, dev, "state")
    y, yptr = _result(out, x, dev)
    _call(dev, "gdn_conv_step", prob, *ins, s, yptr)
    return y


# --------------------------------------------------------------------------- selective scan

def _scan_problem(u, Bm, cu_seqlens, dt_softplus):
    """(device index, offsets, problem)"""
    what = "u must be (B, T, D) and Bm, Cm (B, T, G, N)"
    dev = _first(u, "u", 3, what)
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise ValueError(what)
    B, T, D = u.shape
    _, _, G, N = Bm.shape
    io, softplus = _IO[u.dtype], int(bool(dt_softplus))
    if cu_seqlens is None:
        return dev, None, _dense(nat.ScanProblem, B, T, D, N, G, B, None, None, io, softplus)
    s = _packed(cu_seqlens, dev)
    return dev, s, _problem(nat.ScanProblem, B, T, D, N, G, s.num_seqs, s.host.ctypes.data, s.dev.data_ptr(), io, softplus)


def _scan_inputs(p, u, dt, A, Bm, Cm, D, z, dt_bias, dev):
    us, io, bc, chan = u.shape, u.dtype, (p.B, p.T, p.G, p.N), (p.D,)
    return (_want(u, us, io, dev, "u"), _want(dt, us, io, dev, "dt"), _want(A, (p.D, p.N), _F32, dev, "A"),
            _want(Bm, bc, io, dev, "Bm"), _want(Cm, bc, io, dev, "Cm"), _may(D, chan, _F32, dev, "D"),
            _may(z, us, io, dev, "z"), _may(dt_bias, chan, _F32, dev, "dt_bias"))


def _scan_size(prob, pass_):
    if not prob.cu_seqlens_host:
        return _dense_scan_size(prob.B, prob.T, prob.D, prob.N, prob.G, prob.io_dtype, pass_)
    n = ctypes.c_size_t(0)
    nat.check(nat.load().gdn_scan_workspace_size(prob, pass_, n), "gdn_scan_workspace_size")
    return n.value


@functools.lru_cache(maxsize=1024)
def _dense_scan_size(B, T, D, N, G, io, pass_):
    n = ctypes.c_size_t(0)
    prob = nat.ScanProblem(B, T, D, N, G, B, None, None, io, 1)
    nat.check(nat.load().gdn_scan_workspace_size(prob, pass_, n), "gdn_scan_workspace_size")
    return n.value


def scan_buffers(u, Bm, cu_seqlens=None):
    """Sizes in bytes of the buffers the scan takes: dict forward (workspace of
    scan_fwd and scan_fwd_save), saved, backward (workspace of scan_bwd_saved)."""
    _, seqs, prob = _scan_problem(u, Bm, cu_seqlens, True)  # seqs: keeps the offsets alive
    return {"forward": _scan_size(prob, nat.GDN_SCAN_FWD), "saved": _scan_size(prob, nat.GDN_SCAN_SAVED),
            "backward": _scan_size(prob, nat.GDN_SCAN_BWD)}


def _scan_fwd(save, u, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus, h0, cu_seqlens, output_final_state, out,
              final_state_out, saved, workspace):
    dev, seqs, prob = _scan_problem(u, Bm, cu_seqlens, dt_softplus)  # seqs: keeps the offsets alive
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    shape = (prob.num_seqs, prob.D, prob.N)
    h0p = _may(h0, shape, _F32, dev, "h0")
    y, yptr = _result(out, u, dev)
    h = final_state_out
    if h is None and output_final_state:
        h = A.new_empty(shape)
    outs = (yptr, _may(h, shape, _F32, dev, "final_state_out"))
    buf, ws, nws = _buffer(workspace, _scan_size(prob, nat.GDN_SCAN_FWD), dev, "workspace")
    if not save:
        _call(dev, "gdn_scan_fwd", prob, *ins, h0p, *outs, ws, nws)
        return y, h
    saved, sv, nsv = _buffer(saved, _scan_size(prob, nat.GDN_SCAN_SAVED), dev, "saved")
    _call(dev, "gdn_scan_fwd_save", prob, *ins, h0p, *outs, sv, nsv, ws, nws)
    return y, h, saved


def scan_fwd(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus: bool = True, h0=None, cu_seqlens=None,
             output_final_state: bool = True, out=None, final_state_out=None, workspace=None):
    """Selective state space scan (gdn_scan_fwd): u, dt, z (B, T, D) and Bm, Cm
    (B, T, G, N) of the io dtype; A (D, N), D and dt_bias (D,) fp32; ``h0`` (sequences,
    D, N) fp32 or None (zero).  N in {8, 16, 32, 64}.  Returns (y, h_final or None)."""
    return _scan_fwd(False, u, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus, h0, cu_seqlens, output_final_state, out,
                     final_state_out, None, workspace)


def scan_fwd_save(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus: bool = True, h0=None,
                  cu_seqlens=None, saved=None, workspace=None):
    """scan_fwd that also keeps what the backward needs (gdn_scan_fwd_save).  Returns
    (y, h_final, saved); pass ``saved`` to scan_bwd_saved with the same inputs."""
    return _scan_fwd(True, u, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus, h0, cu_seqlens, True, None, None, saved,
                     workspace)


def scan_bwd_saved(u, dt, A, Bm, Cm, dy, saved, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                   dh_final=None, cu_seqlens=None, want_dh0: bool = True, workspace=None):
    """Backward of scan_fwd_save (gdn_scan_bwd_saved) with the same inputs and
    cu_seqlens.  Returns dict du, ddt, dA, dB, dC, dD (None without D), dz (None
    without z), ddt_bias (None without dt_bias), dh0."""
    dev, seqs, prob = _scan_problem(u, Bm, cu_seqlens, dt_softplus)  # seqs: keeps the offsets alive
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    shape = (prob.num_seqs, prob.D, prob.N)
    dyp = _want(dy, u.shape, u.dtype, dev, "dy")
    dhp = _may(dh_final, shape, _F32, dev, "dh_final")
    need = _scan_size(prob, nat.GDN_SCAN_SAVED)
    if saved is None and need:
        raise ValueError("saved must be the buffer scan_fwd_save filled")
    _, sv, nsv = _buffer(saved, 0, dev, "saved")
    buf, ws, nws = _buffer(workspace, _scan_size(prob, nat.GDN_SCAN_BWD), dev, "workspace")
    empty = lambda t: torch.empty_like(t) if t is not None else None  # noqa: E731
    out = {"du": empty(u), "ddt": empty(dt), "dA": empty(A), "dB": empty(Bm), "dC": empty(Cm), "dD": empty(D),
           "dz": empty(z), "ddt_bias": empty(dt_bias),
           "dh0": A.new_empty(shape) if want_dh0 else None}
    _call(dev, "gdn_scan_bwd_saved", prob, *ins, dyp, dhp, sv, nsv,
          *(t.data_ptr() if t is not None else None for t in out.values()), ws, nws)
    return out


def scan_step(u, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus: bool = True, out=None):
    """One token of scan_fwd for every sequence (gdn_scan_step): u, dt, z (B, 1, D),
    Bm, Cm (B, 1, G, N); ``state`` (B, D, N) fp32 is updated in place.  Returns y."""
    dev, _, prob = _scan_problem(u, Bm, None, dt_softplus)
    if prob.T != 1:
        raise ValueError("u must be (B, 1, D)")
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    s = _want(state, (prob.B, prob.D, prob.N), _F32, dev, "state")
    y, yptr = _result(out, u, dev)
    _call(dev, "gdn_scan_step", prob, *ins, s, yptr)
    return y
