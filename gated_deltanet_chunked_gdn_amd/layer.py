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
once as a ``SeqLens``.  Outputs and gradients that were not asked for are None.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native as nat
from .ops import _IO, SeqLens, _seqlens

# the current device and the raw current stream, without building Python objects: a
# single-token call is a few microseconds
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)

_ACT = {None: nat.GDN_ACT_NONE, "none": nat.GDN_ACT_NONE, "silu": nat.GDN_ACT_SILU}


def _first(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (got {t.device})")
    if t.dtype not in _IO:
        raise TypeError(f"{name} must be bfloat16 or float32")
    return t.device


def _want(t, shape, dtype, device, name, optional=False):
    """A contiguous tensor of this shape, dtype and device, as an address (None for an
    absent optional one).  A host pointer that reached a kernel would be a GPU memory
    fault, which the C ABI cannot detect."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    raise ValueError(f"{name} must be contiguous with shape {tuple(shape)} (got {tuple(t.shape)})")


def _out(out, like, device, name):
    if out is None:
        return torch.empty_like(like)
    _want(out, like.shape, like.dtype, device, name)
    return out


def _call(device, name, *args):
    """The library call on the device's current stream, with that device current."""
    fn = getattr(nat.load(), name)
    index = device.index
    if index == _current_device():
        st = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _current_stream(index))
    if st:
        nat.check(st, name)


def _offsets(seqs: Optional[SeqLens], device, batch):
    """(sequences, host offsets, device offsets)"""
    if seqs is None:
        return batch, None, None
    if seqs.dev.device != device:
        raise ValueError(f"cu_seqlens must be on {device} (got {seqs.dev.device})")
    return seqs.num_seqs, seqs.host.ctypes.data, seqs.dev.data_ptr()


def _buffer(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _buffer_arg(buf, nbytes, device, name):
    """A caller's uint8 buffer, or a fresh one of the size the library asks for."""
    if buf is None:
        buf = _buffer(nbytes, device)
        return buf, (buf.data_ptr() if buf is not None else None), nbytes
    if not isinstance(buf, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if buf.device != device:
        raise ValueError(f"{name} must be on {device} (got {buf.device})")
    if not buf.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return buf, buf.data_ptr(), buf.numel() * buf.element_size()


# --------------------------------------------------------------------------- delta rule, one token

def _step(name, q, k, v, g, beta, state, scale, out, channel):
    dev = _first(q, "q")
    if q.dim() != 4 or q.shape[1] != 1 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q and k must be (B, 1, H, Dk) and v (B, 1, H, Dv)")
    B, _, H, Dk = q.shape
    Dv = v.shape[3]
    io, f32 = q.dtype, torch.float32
    args = (_want(q, q.shape, io, dev, "q"), _want(k, q.shape, io, dev, "k"), _want(v, (B, 1, H, Dv), io, dev, "v"),
            _want(g, q.shape if channel else (B, 1, H), f32, dev, "g"), _want(beta, (B, 1, H), f32, dev, "beta"),
            _want(state, (B, H, Dk, Dv), f32, dev, "state"))
    o = _out(out, v, dev, "out")
    prob = nat.Problem(B, 1, H, Dk, Dv, B, None, None, _IO[io], scale, 64, 1, nat.GDN_PRECISION_IO)
    _call(dev, name, prob, *args, o.data_ptr())
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

def _conv_problem(x, weight, seqs, activation, dev):
    if x.dim() != 3:
        raise ValueError("x must be (B, T, C)")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a (C, W) tensor")
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(map(str, _ACT))}")
    B, T, C = x.shape
    n, host, ptr = _offsets(seqs, dev, B)
    return nat.ConvProblem(B, T, C, weight.shape[1], n, host, ptr, _IO[x.dtype], _ACT[activation])


def _conv_inputs(x, weight, bias, dev):
    C, f32 = x.shape[2], torch.float32
    return (_want(x, x.shape, x.dtype, dev, "x"), _want(weight, (C, weight.shape[1]), f32, dev, "weight"),
            _want(bias, (C,), f32, dev, "bias", optional=True))


def conv_fwd(x, weight, bias=None, state0=None, cu_seqlens=None, activation: Optional[str] = "silu",
             output_final_state: bool = True, out=None, final_state_out=None):
    """Short causal depthwise convolution (gdn_conv_fwd): x (B, T, C) of the io dtype,
    weight (C, W) and bias (C,) fp32, W in 2..4; ``activation`` "silu" or None.
    ``state0`` (N, W - 1, C) of the io dtype holds the rows before every sequence
    (oldest first; None: zeros).  Returns (y, state_final or None)."""
    dev = _first(x, "x")
    seqs = _seqlens(cu_seqlens, dev)
    prob = _conv_problem(x, weight, seqs, activation, dev)
    shape = (prob.num_seqs, prob.W - 1, prob.C)
    ins = _conv_inputs(x, weight, bias, dev)
    s0 = _want(state0, shape, x.dtype, dev, "state0", optional=True)
    y = _out(out, x, dev, "out")
    last = final_state_out
    if last is None and output_final_state:
        last = torch.empty(shape, dtype=x.dtype, device=dev)
    _call(dev, "gdn_conv_fwd", prob, *ins, s0, y.data_ptr(),
          _want(last, shape, x.dtype, dev, "final_state_out", optional=True))
    return y, last


def conv_bwd(x, weight, dy, bias=None, state0=None, dstate_final=None, cu_seqlens=None,
             activation: Optional[str] = "silu", workspace=None):
    """Backward of conv_fwd (gdn_conv_bwd).  Returns dict dx, dweight, dbias (None
    without bias), dstate0 (None without state0)."""
    dev = _first(x, "x")
    seqs = _seqlens(cu_seqlens, dev)
    prob = _conv_problem(x, weight, seqs, activation, dev)
    shape = (prob.num_seqs, prob.W - 1, prob.C)
    ins = _conv_inputs(x, weight, bias, dev)
    s0 = _want(state0, shape, x.dtype, dev, "state0", optional=True)
    grads = (_want(dy, x.shape, x.dtype, dev, "dy"),
             _want(dstate_final, shape, x.dtype, dev, "dstate_final", optional=True))
    n = ctypes.c_size_t(0)
    nat.check(nat.load().gdn_conv_workspace_size(prob, n), "gdn_conv_workspace_size")
    _, ws, nws = _buffer_arg(workspace, n.value, dev, "workspace")
    out = {"dx": torch.empty_like(x), "dweight": torch.empty_like(weight),
           "dbias": torch.empty_like(bias) if bias is not None else None,
           "dstate0": torch.empty_like(state0) if state0 is not None else None}
    _call(dev, "gdn_conv_bwd", prob, *ins, s0, *grads, *(t.data_ptr() if t is not None else None for t in out.values()),
          ws, nws)
    return out


def conv_step(x, weight, state, bias=None, activation: Optional[str] = "silu", out=None):
    """One token of conv_fwd for every sequence (gdn_conv_step): x (B, 1, C); ``state``
    (B, W - 1, C) is shifted by one row in place.  Returns y."""
    dev = _first(x, "x")
    prob = _conv_problem(x, weight, None, activation, dev)
    if x.shape[1] != 1:
        raise ValueError("x must be (B, 1, C)")
    ins = _conv_inputs(x, weight, bias, dev)
    s = _want(state, (prob.B, prob.W - 1, prob.C), x.dtype, dev, "state")
    y = _out(out, x, dev, "out")
    _call(dev, "gdn_conv_step", prob, *ins, s, y.data_ptr())
    return y


# --------------------------------------------------------------------------- selective scan

def _scan_problem(u, A, Bm, seqs, dt_softplus, dev):
    if u.dim() != 3 or not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise ValueError("u must be (B, T, D) and Bm, Cm (B, T, G, N)")
    B, T, D = u.shape
    n, host, ptr = _offsets(seqs, dev, B)
    return nat.ScanProblem(B, T, D, Bm.shape[3], Bm.shape[2], n, host, ptr, _IO[u.dtype], bool(dt_softplus))


def _scan_inputs(p, u, dt, A, Bm, Cm, D, z, dt_bias, dev):
    io, f32, bc = u.dtype, torch.float32, (p.B, p.T, p.G, p.N)
    return (_want(u, u.shape, io, dev, "u"), _want(dt, u.shape, io, dev, "dt"), _want(A, (p.D, p.N), f32, dev, "A"),
            _want(Bm, bc, io, dev, "Bm"), _want(Cm, bc, io, dev, "Cm"), _want(D, (p.D,), f32, dev, "D", optional=True),
            _want(z, u.shape, io, dev, "z", optional=True), _want(dt_bias, (p.D,), f32, dev, "dt_bias", optional=True))


def _scan_size(prob, pass_):
    n = ctypes.c_size_t(0)
    nat.check(nat.load().gdn_scan_workspace_size(prob, pass_, n), "gdn_scan_workspace_size")
    return n.value


def scan_buffers(u, A, Bm, cu_seqlens=None):
    """Sizes in bytes of the buffers the scan takes: dict forward (workspace of
    scan_fwd and scan_fwd_save), saved, backward (workspace of scan_bwd_saved)."""
    dev = _first(u, "u")
    prob = _scan_problem(u, A, Bm, _seqlens(cu_seqlens, dev), True, dev)
    return {"forward": _scan_size(prob, nat.GDN_SCAN_FWD), "saved": _scan_size(prob, nat.GDN_SCAN_SAVED),
            "backward": _scan_size(prob, nat.GDN_SCAN_BWD)}


def _scan_fwd(save, u, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus, h0, cu_seqlens, output_final_state, out,
              final_state_out, saved, workspace):
    dev = _first(u, "u")
    seqs = _seqlens(cu_seqlens, dev)
    prob = _scan_problem(u, A, Bm, seqs, dt_softplus, dev)
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    shape = (prob.num_seqs, prob.D, prob.N)
    h0p = _want(h0, shape, torch.float32, dev, "h0", optional=True)
    y = _out(out, u, dev, "out")
    h = final_state_out
    if h is None and output_final_state:
        h = torch.empty(shape, dtype=torch.float32, device=dev)
    outs = (y.data_ptr(), _want(h, shape, torch.float32, dev, "final_state_out", optional=True))
    _, ws, nws = _buffer_arg(workspace, _scan_size(prob, nat.GDN_SCAN_FWD), dev, "workspace")
    if not save:
        _call(dev, "gdn_scan_fwd", prob, *ins, h0p, *outs, ws, nws)
        return y, h
    saved, sv, nsv = _buffer_arg(saved, _scan_size(prob, nat.GDN_SCAN_SAVED), dev, "saved")
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
    dev = _first(u, "u")
    seqs = _seqlens(cu_seqlens, dev)
    prob = _scan_problem(u, A, Bm, seqs, dt_softplus, dev)
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    shape = (prob.num_seqs, prob.D, prob.N)
    dyp = _want(dy, u.shape, u.dtype, dev, "dy")
    dhp = _want(dh_final, shape, torch.float32, dev, "dh_final", optional=True)
    need = _scan_size(prob, nat.GDN_SCAN_SAVED)
    if saved is None and need:
        raise ValueError("saved must be the buffer scan_fwd_save filled")
    _, sv, nsv = _buffer_arg(saved, 0, dev, "saved")
    _, ws, nws = _buffer_arg(workspace, _scan_size(prob, nat.GDN_SCAN_BWD), dev, "workspace")
    empty = lambda t: torch.empty_like(t) if t is not None else None  # noqa: E731
    out = {"du": empty(u), "ddt": empty(dt), "dA": empty(A), "dB": empty(Bm), "dC": empty(Cm), "dD": empty(D),
           "dz": empty(z), "ddt_bias": empty(dt_bias),
           "dh0": torch.empty(shape, dtype=torch.float32, device=dev) if want_dh0 else None}
    _call(dev, "gdn_scan_bwd_saved", prob, *ins, dyp, dhp, sv, nsv,
          *(t.data_ptr() if t is not None else None for t in out.values()), ws, nws)
    return out


def scan_step(u, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus: bool = True, out=None):
    """One token of scan_fwd for every sequence (gdn_scan_step): u, dt, z (B, 1, D),
    Bm, Cm (B, 1, G, N); ``state`` (B, D, N) fp32 is updated in place.  Returns y."""
    dev = _first(u, "u")
    prob = _scan_problem(u, A, Bm, None, dt_softplus, dev)
    if u.shape[1] != 1:
        raise ValueError("u must be (B, 1, D)")
    ins = _scan_inputs(prob, u, dt, A, Bm, Cm, D, z, dt_bias, dev)
    s = _want(state, (prob.B, prob.D, prob.N), torch.float32, dev, "state")
    y = _out(out, u, dev, "out")
    _call(dev, "gdn_scan_step", prob, *ins, s, y.data_ptr())
    return y
