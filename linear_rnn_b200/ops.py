"""Python entry points with the names of the C ABI (include/gla.h): gla_fwd, gla_bwd,
gla_workspace_bytes, gla_check_device_status.

They marshal torch tensors into the C calls: shape/dtype checks, the gate mode read
from g's rank, a workspace allocated with torch (the library itself allocates nothing),
and the current torch CUDA stream. Tensors on the host are copied to the current CUDA
device and results copied back (the end-to-end call of a host-side user); tensors
already on the device are used in place.
"""
from __future__ import annotations

import ctypes
import math
from typing import Dict, Optional, Tuple

import torch

from . import _lib
from ._lib import GlaError, GlaNormProblem, GlaProblem

_PLANS = {"auto": _lib.GLA_PLAN_AUTO, "simt": _lib.GLA_PLAN_SIMT, "tc": _lib.GLA_PLAN_TC}
_SCAN_INPUTS = {"plain": _lib.GLA_SCAN_PLAIN, "complement": _lib.GLA_SCAN_COMPLEMENT, "norm": _lib.GLA_SCAN_NORM}
_NORM_KINDS = {"rms": _lib.GLA_NORM_RMS, "layer": _lib.GLA_NORM_LAYER}
_ACTS = {"silu": _lib.GLA_ACT_SILU, "sigmoid": _lib.GLA_ACT_SIGMOID}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _io_dtype(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return _lib.GLA_F32
    if dt == torch.bfloat16:
        return _lib.GLA_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {dt}")


def make_problem(q: torch.Tensor, v: torch.Tensor, g: Optional[torch.Tensor], *, scale: Optional[float],
                 chunk: int, plan: str) -> GlaProblem:
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, L, D]")
    B, H, L, Dk = q.shape
    Dv = v.shape[-1]
    if g is None:
        gate = _lib.GLA_GATE_NONE
    elif g.dim() == 4:
        gate = _lib.GLA_GATE_PER_KEY
    elif g.dim() == 3:
        gate = _lib.GLA_GATE_PER_HEAD
    else:
        raise ValueError("g must be [B,H,L,Dk] (per key dim) or [B,H,L] (per head)")
    if plan not in _PLANS:
        raise ValueError(f"plan must be one of {sorted(_PLANS)}")
    return GlaProblem(B, H, L, Dk, Dv, int(chunk), float(1.0 / math.sqrt(Dk) if scale is None else scale),
                      _io_dtype(q.dtype), gate, _PLANS[plan])


def gla_workspace_bytes(problem: GlaProblem, for_backward: bool) -> int:
    return int(_lib.lib.gla_workspace_bytes(ctypes.byref(problem), int(for_backward)))


def _stream_handle(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _to_dev(t: Optional[torch.Tensor], device: torch.device) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("inputs must be contiguous (BHLD)")
    if t.device.type == "cuda":
        return t
    return t.to(device, non_blocking=True)


def _to_host(tensors):
    """Copy device results into pinned host tensors (asynchronously on the current
    stream), then wait for the stream once."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        h = torch.empty(t.shape, dtype=t.dtype, pin_memory=True)
        h.copy_(t, non_blocking=True)
        out.append(h)
    torch.cuda.current_stream().synchronize()
    return out


def _check(status: int, where: str):
    if status != _lib.GLA_OK:
        raise GlaError(status, where)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise GlaError(_lib.GLA_ERR_WORKSPACE, "workspace")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def gla_saved_states_bytes(problem: GlaProblem) -> int:
    return int(_lib.lib.gla_saved_states_bytes(ctypes.byref(problem)))


def gla_fwd(q, k, v, g=None, igate=None, h0=None, *, scale: Optional[float] = None, chunk: int = 64,
            plan: str = "auto", output_final_state: bool = True,
            workspace: Optional[torch.Tensor] = None,
            saved_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Forward pass. Returns (o, hT); hT is None when output_final_state is False.
    saved_states: optional device buffer (at least gla_saved_states_bytes) that receives the
    states gla_bwd(..., saved_states=) then uses instead of recomputing them."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, g, igate, h0 = (_to_dev(t, device) for t in (q, k, v, g, igate, h0))
    prob = make_problem(q, v, g, scale=scale, chunk=chunk, plan=plan)
    o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=device)
    hT = torch.empty(q.shape[0], q.shape[1], q.shape[-1], v.shape[-1], dtype=torch.float32,
                     device=device) if output_final_state else None
    nbytes = gla_workspace_bytes(prob, False)
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_workspace_bytes")
    ws = _workspace(nbytes, device, workspace)
    _check_saved(saved_states, prob)
    st = _lib.lib.gla_fwd_save(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(igate), _ptr(h0),
                               _ptr(o), _ptr(hT), _ptr(saved_states), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream_handle(device))
    _check(st, "gla_fwd")
    if host:
        o, hT = _to_host([o, hT])
    return o, hT


def _mlstm_problem(q, v, g, itil, scale, chunk, plan):
    if g is None or g.dim() != 3 or g.dtype != torch.float32:
        raise ValueError("g (log forget gate) must be float32 [B, H, L]")
    if itil is None or itil.dtype != torch.float32 or tuple(itil.shape) != tuple(g.shape):
        raise ValueError("itil (log input gate) must be float32 [B, H, L] like g")
    return make_problem(q, v, g, scale=scale, chunk=chunk, plan=plan)


def gla_mlstm_saved_bytes(problem: GlaProblem) -> int:
    return int(_lib.lib.gla_mlstm_saved_bytes(ctypes.byref(problem)))


def _check_ml_saved(saved, prob):
    if saved is None:
        return
    if saved.device.type != "cuda" or not saved.is_contiguous():
        raise ValueError("saved_states must be a contiguous CUDA tensor")
    if saved.numel() * saved.element_size() < gla_mlstm_saved_bytes(prob):
        raise GlaError(_lib.GLA_ERR_WORKSPACE, "saved_states")


def gla_mlstm_fwd(q, k, v, g, itil, *, scale: Optional[float] = None, chunk: int = 64, plan: str = "auto",
                  workspace: Optional[torch.Tensor] = None,
                  saved_states: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mLSTM cell (exponential input gate, normaliser, stabiliser): q, k [B,H,L,Dk], v [B,H,L,Dv],
    g = log forget gate and itil = log input gate, both fp32 [B,H,L]. Returns h [B,H,L,Dv].
    saved_states: optional device buffer (at least gla_mlstm_saved_bytes) that keeps the forward's
    results for gla_mlstm_bwd(..., saved_states=), which then does not run the forward again."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, g, itil = (_to_dev(t, device) for t in (q, k, v, g, itil))
    prob = _mlstm_problem(q, v, g, itil, scale, chunk, plan)
    nbytes = int(_lib.lib.gla_mlstm_workspace_bytes(ctypes.byref(prob), 0))
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_mlstm_workspace_bytes")
    ws = _workspace(nbytes, device, workspace)
    _check_ml_saved(saved_states, prob)
    h = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=device)
    st = _lib.lib.gla_mlstm_fwd_save(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(itil), _ptr(h),
                                     _ptr(saved_states), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream_handle(device))
    _check(st, "gla_mlstm_fwd")
    if host:
        (h,) = _to_host([h])
    return h


def gla_mlstm_bwd(q, k, v, g, itil, dh, *, scale: Optional[float] = None, chunk: int = 64, plan: str = "auto",
                  workspace: Optional[torch.Tensor] = None,
                  saved_states: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(dh * h) of gla_mlstm_fwd: dict dq, dk, dv (io dtype), dg, ditil (fp32).
    saved_states: the buffer a gla_mlstm_fwd with the same inputs and plan filled, or None to
    run the forward passes again."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, g, itil, dh = (_to_dev(t, device) for t in (q, k, v, g, itil, dh))
    prob = _mlstm_problem(q, v, g, itil, scale, chunk, plan)
    nbytes = int(_lib.lib.gla_mlstm_workspace_bytes(ctypes.byref(prob), 1))
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_mlstm_workspace_bytes")
    ws = _workspace(nbytes, device, workspace)
    _check_ml_saved(saved_states, prob)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, ditil = torch.empty_like(g), torch.empty_like(itil)
    st = _lib.lib.gla_mlstm_bwd_saved(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(itil), _ptr(dh),
                                      _ptr(saved_states), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ditil),
                                      _ptr(ws), ws.numel() * ws.element_size(), _stream_handle(device))
    _check(st, "gla_mlstm_bwd")
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "ditil": ditil}
    if host:
        out = dict(zip(out, _to_host(list(out.values()))))
    return out


def gla_decode(q, k, v, g, igate, state, *, scale: Optional[float] = None) -> torch.Tensor:
    """One recurrent step per (b, h) from `state` (fp32 [B,H,Dk,Dv] on the GPU, updated in
    place): q, k [B,H,1,Dk], v [B,H,1,Dv], g [B,H,1,Dk] / [B,H,1] / None, igate [B,H,1] / None.
    Returns o [B,H,1,Dv]."""
    if state.device.type != "cuda" or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor (it is updated in place)")
    device = state.device
    q, k, v, g, igate = (_to_dev(t, device) for t in (q, k, v, g, igate))
    if q.shape[2] != 1:
        raise ValueError("gla_decode takes one token per (b, h): q must be [B, H, 1, Dk]")
    prob = make_problem(q, v, g, scale=scale, chunk=64, plan="auto")
    o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=device)
    st = _lib.lib.gla_decode(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(igate), _ptr(state),
                             _ptr(o), _stream_handle(device))
    _check(st, "gla_decode")
    return o


def gla_deltanet_saved_bytes(problem: GlaProblem) -> int:
    return int(_lib.lib.gla_deltanet_saved_bytes(ctypes.byref(problem)))


def _check_dn_saved(saved, prob):
    if saved is None:
        return
    if saved.device.type != "cuda" or not saved.is_contiguous():
        raise ValueError("saved_states must be a contiguous CUDA tensor")
    if saved.numel() * saved.element_size() < gla_deltanet_saved_bytes(prob):
        raise GlaError(_lib.GLA_ERR_WORKSPACE, "saved_states")


def gla_deltanet_fwd(q, k, v, beta, h0=None, *, scale: Optional[float] = None,
                     output_final_state: bool = True,
                     saved_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunkwise DeltaNet forward: q, k [B,H,L,Dk], v [B,H,L,Dv] (bf16 or fp32), beta [B,H,L]
    fp32, h0 [B,H,Dk,Dv] fp32 or None. Returns o [B,H,L,Dv] and the final state (fp32, or None
    when output_final_state is False). saved_states: optional device buffer (at least
    gla_deltanet_saved_bytes) that receives the chunk start states, which
    gla_deltanet_bwd(..., saved_states=) then reads instead of walking the recurrence again.
    Host tensors are copied to the current device and the results back."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, beta, h0 = (_to_dev(t, device) for t in (q, k, v, beta, h0))
    if beta is None or beta.dtype != torch.float32 or tuple(beta.shape) != tuple(q.shape[:3]):
        raise ValueError("beta must be float32 [B, H, L]")
    prob = make_problem(q, v, None, scale=scale, chunk=64, plan="auto")
    _check_dn_saved(saved_states, prob)
    o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=device)
    hT = torch.empty(q.shape[0], q.shape[1], q.shape[-1], v.shape[-1], dtype=torch.float32,
                     device=device) if output_final_state else None
    st = _lib.lib.gla_deltanet_fwd_save(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(h0),
                                        _ptr(o), _ptr(hT), _ptr(saved_states), _stream_handle(device))
    _check(st, "gla_deltanet_fwd")
    if host:
        o, hT = _to_host([o, hT])
    return o, hT


def gla_deltanet_bwd(q, k, v, beta, h0, dO, dhT=None, *, scale: Optional[float] = None,
                     output_dh0: bool = True, workspace: Optional[torch.Tensor] = None,
                     saved_states: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """DeltaNet backward: dict dq, dk, dv (io dtype), dbeta (fp32 [B,H,L]) and dh0 (fp32, or
    None when output_dh0 is False). saved_states: the buffer a gla_deltanet_fwd on the same
    inputs filled, or None to recompute the chunk start states. Host tensors are copied to the
    current device and the results back."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, beta, h0, dO, dhT = (_to_dev(t, device) for t in (q, k, v, beta, h0, dO, dhT))
    if beta is None or beta.dtype != torch.float32 or tuple(beta.shape) != tuple(q.shape[:3]):
        raise ValueError("beta must be float32 [B, H, L]")
    prob = make_problem(q, v, None, scale=scale, chunk=64, plan="auto")
    nbytes = _lib.lib.gla_deltanet_bwd_workspace_bytes(ctypes.byref(prob))
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_deltanet_bwd_workspace_bytes")
    ws = _workspace(nbytes, device, workspace)
    _check_dn_saved(saved_states, prob)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta = torch.empty_like(beta)
    dh0 = torch.empty(q.shape[0], q.shape[1], q.shape[-1], v.shape[-1], dtype=torch.float32,
                      device=device) if output_dh0 else None
    st = _lib.lib.gla_deltanet_bwd_saved(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(h0),
                                         _ptr(dO), _ptr(dhT), _ptr(saved_states), _ptr(dq), _ptr(dk), _ptr(dv),
                                         _ptr(dbeta), _ptr(dh0), _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream_handle(device))
    _check(st, "gla_deltanet_bwd")
    out = {"dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dh0": dh0}
    if host:
        names = list(out)
        out = dict(zip(names, _to_host([out[n] for n in names])))
    return out


# The operators below are also called where a pass takes a few microseconds on the GPU, so their
# host work is kept short: descriptors are looked up by sizes and types, and every tensor is
# checked once.
# torch's own short cuts for the current device and stream, where it has them (a build without CUDA does not)
_getDevice = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_rawStream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_f32 = torch.float32


def _check_tensor(name, t, shape, dtype, dev):
    """Refuses a tensor that has not this shape and dtype, is not on CUDA device `dev` or not contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _ptr_of(name, t, shape, dtype, dev):
    """The address of a checked argument; None stays None."""
    if t is None:
        return None
    _check_tensor(name, t, shape, dtype, dev)
    return t.data_ptr()


def _need(name, t):
    if t is None:
        raise ValueError(f"{name} is needed")
    return t


def _choice(name, value, table):
    got = table.get(value)
    if got is None:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return got


def _launch(where, fn, dev, args):
    """Calls fn with the current stream of CUDA device `dev`, with that device current."""
    if dev == _getDevice():
        st = fn(*args, _rawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _rawStream(dev))
    if st:
        raise GlaError(st, where)


def _from_host(fn, tensors, kw):
    """A call on host tensors: copies to the current device, the call, copies back. The caller's buffers are not
    copied: they are written, and must be on the device."""
    device = torch.device("cuda", torch.cuda.current_device())
    moved = [t if t is None or t.is_cuda else t.contiguous().to(device, non_blocking=True) for t in tensors]
    kw = {k: v.to(device) if k == "rscale" and v is not None else v for k, v in kw.items()}
    out = fn(*moved, **kw)
    if isinstance(out, dict):
        return dict(zip(out, _to_host(list(out.values()))))
    if isinstance(out, tuple):
        return tuple(_to_host(list(out)))
    return _to_host([out])[0]


def _buffer(name, t, nbytes, dev):
    """The address of a workspace or saved-states buffer of the caller."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on cuda:{dev}")
    if t.numel() * t.element_size() < nbytes:
        raise GlaError(_lib.GLA_ERR_WORKSPACE, name)
    return t.data_ptr()


_descriptors = {}


def _descriptor(key, make):
    """The C descriptor of a problem, made once per sizes and types: (struct, reference to it). The key holds
    plain numbers only: a tensor in it would be found by its identity, whatever its value had become."""
    d = _descriptors.get(key)
    if d is None:
        if len(_descriptors) >= 1024:
            _descriptors.clear()
        prob = make()
        d = _descriptors[key] = (prob, ctypes.byref(prob))
    return d


def _sizes(where, *sizes):
    """The sizes of a descriptor, whose fields have 32 bits."""
    if max(sizes) > 2147483647:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, where)
    return sizes


def make_scan_problem(x: torch.Tensor) -> GlaProblem:
    """The gla_problem of the vector-state recurrence over x [B,H,L,D]."""
    if x.dim() != 4:
        raise ValueError("x must be [B, H, L, D]")
    B, H, L, D = _sizes("x's sizes", *x.shape)
    return GlaProblem(B, H, L, D, D, 64, 1.0, _io_dtype(x.dtype), _lib.GLA_GATE_PER_KEY, _lib.GLA_PLAN_AUTO)


def gla_scan_saved_bytes(problem: GlaProblem) -> int:
    return _lib.lib.gla_scan_saved_bytes(ctypes.byref(problem))


def gla_scan_bwd_workspace_bytes(problem: GlaProblem) -> int:
    return _lib.lib.gla_scan_bwd_workspace_bytes(ctypes.byref(problem))


def gla_scan_fwd(x, g, h0=None, *, input: str = "plain", output_final_state: bool = True,
                 saved_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence with a vector state, h_t = e^{g_t} h_{t-1} + m(g_t) x_t per channel:
    x [B,H,L,D] (bf16 or fp32), g [B,H,L,D] fp32 (log-decay; -inf starts anew), h0 [B,H,D] fp32 or
    None (zero). input picks m: "plain" 1, "complement" 1 - e^g, "norm" sqrt(1 - e^{2g}). Returns
    o [B,H,L,D] (every h_t) and hT [B,H,D] fp32 (or None when output_final_state is False).
    saved_states: optional device buffer (at least gla_scan_saved_bytes) that receives the states
    entering every 64 tokens, for gla_scan_bwd(..., saved_states=). Host tensors are copied to the
    current device and the results back."""
    if not x.is_cuda:
        return _from_host(gla_scan_fwd, (x, _need("g", g), h0),
                          dict(input=input, output_final_state=output_final_state, saved_states=saved_states))
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    prob, ref = _descriptor((shape, dtype), lambda: make_scan_problem(x))
    ends = (shape[0], shape[1], shape[3])
    mode = _choice("input", input, _SCAN_INPUTS)
    px = _ptr_of("x", x, shape, dtype, dev)
    pg = _ptr_of("g", _need("g", g), shape, _f32, dev)
    ph = _ptr_of("h0", h0, ends, _f32, dev)
    ps = None if saved_states is None else _buffer("saved_states", saved_states, gla_scan_saved_bytes(prob), dev)
    o = torch.empty_like(x)
    hT = g.new_empty(ends) if output_final_state else None
    _launch("gla_scan_fwd", _lib.lib.gla_scan_fwd_save, dev,
            (ref, mode, px, pg, ph, o.data_ptr(), None if hT is None else hT.data_ptr(), ps))
    return o, hT


def gla_scan_bwd(x, g, h0, dO, dhT=None, *, input: str = "plain", output_dh0: bool = True,
                 workspace: Optional[torch.Tensor] = None,
                 saved_states: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of sum(dO * o) + sum(dhT * hT) of gla_scan_fwd: dict dx (io dtype), dg (fp32) and
    dh0 (fp32, or None when output_dh0 is False). saved_states: the buffer a gla_scan_fwd on the
    same x, g, h0 and input filled, or None to run the recurrence again (which needs a workspace
    of gla_scan_bwd_workspace_bytes, allocated when None)."""
    if not x.is_cuda:
        return _from_host(gla_scan_bwd, (x, _need("g", g), h0, _need("dO", dO), dhT),
                          dict(input=input, output_dh0=output_dh0, workspace=workspace, saved_states=saved_states))
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    prob, ref = _descriptor((shape, dtype), lambda: make_scan_problem(x))
    ends = (shape[0], shape[1], shape[3])
    mode = _choice("input", input, _SCAN_INPUTS)
    px = _ptr_of("x", x, shape, dtype, dev)
    pg = _ptr_of("g", _need("g", g), shape, _f32, dev)
    pd = _ptr_of("dO", _need("dO", dO), shape, dtype, dev)
    ph = _ptr_of("h0", h0, ends, _f32, dev)
    pT = _ptr_of("dhT", dhT, ends, _f32, dev)
    ps = pw = None
    nbytes = 0
    if saved_states is not None:
        ps = _buffer("saved_states", saved_states, gla_scan_saved_bytes(prob), dev)
    else:
        nbytes = gla_scan_bwd_workspace_bytes(prob)
        if nbytes == 0:
            raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_scan_bwd_workspace_bytes")
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        pw = _buffer("workspace", workspace, nbytes, dev)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    dh0 = g.new_empty(ends) if output_dh0 else None
    _launch("gla_scan_bwd", _lib.lib.gla_scan_bwd_saved, dev,
            (ref, mode, px, pg, ph, pd, pT, ps, dx.data_ptr(), dg.data_ptr(), None if dh0 is None else dh0.data_ptr(),
             pw, nbytes))
    return {"dx": dx, "dg": dg, "dh0": dh0}


def gla_scan_decode(x, g, state, *, input: str = "plain") -> torch.Tensor:
    """One token of gla_scan_fwd per (b, h) from `state` (fp32 [B,H,D] on the GPU, updated in
    place): x, g [B,H,1,D]. Returns o [B,H,1,D], on the GPU. x and g may be on the host; then the call waits for
    their copies, so that their buffers may be written again when it returns."""
    if not state.is_cuda or state.dtype is not _f32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor (it is updated in place)")
    if not x.is_cuda or not _need("g", g).is_cuda:
        x, g = (t.contiguous().to(state.device) for t in (x, _need("g", g)))
    shape, dtype, dev = x.shape, x.dtype, state.get_device()
    _, ref = _descriptor((shape, dtype), lambda: make_scan_problem(x))
    if shape[2] != 1:
        raise ValueError("gla_scan_decode takes one token per (b, h): x must be [B, H, 1, D]")
    mode = _choice("input", input, _SCAN_INPUTS)
    px = _ptr_of("x", x, shape, dtype, dev)
    pg = _ptr_of("g", g, shape, _f32, dev)
    ps = _ptr_of("state", state, (shape[0], shape[1], shape[3]), _f32, dev)
    o = torch.empty_like(x)
    _launch("gla_scan_decode", _lib.lib.gla_scan_decode, dev, (ref, mode, px, pg, ps, o.data_ptr()))
    return o


def gla_scan_check_device_status(device=None) -> int:
    """Waits for the current stream of `device` (None: the current one) and returns the status of the gla_scan_* calls on
    it since the last check: GLA_OK, or GLA_ERR_TIMEOUT where a bounded wait on the GPU gave up."""
    with torch.cuda.device(device):
        return int(_lib.lib.gla_scan_check_device_status(_rawStream(_getDevice())))


def _addnorm_problem(x, res_dtype, kind, eps, alpha) -> GlaNormProblem:
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    if D < 1:
        raise ValueError("x must have channels")
    rows, D = _sizes("rows and channels", x.numel() // D, D)
    return GlaNormProblem(1, 1, rows, D, _io_dtype(x.dtype), _io_dtype(res_dtype), _choice("kind", kind, _NORM_KINDS),
                          _lib.GLA_ACT_SILU, 0, eps, alpha)


def gla_addnorm_fwd(x, res=None, w=None, *, rscale=None, alpha: float = 1.0, kind: str = "rms", eps: float = 1e-6,
                    res_dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Residual sum and norm before a block: r = res + alpha * rscale * x, y = norm(r) * w.
    x [..., D] (bf16 or fp32) is the last block's output; res [..., D] the residual stream, of
    x's dtype or fp32 (None: zero, with r in res_dtype, x's by default); w, rscale [D] fp32 or
    None (one); kind "rms" or "layer". Returns r (res's dtype) and y (x's dtype); y is the norm of
    the fp32 sum, before r is rounded. Host tensors are copied to the current device and the
    results back."""
    if not x.is_cuda:
        return _from_host(gla_addnorm_fwd, (x, res, w),
                          dict(rscale=rscale, alpha=alpha, kind=kind, eps=eps, res_dtype=res_dtype))
    shape, dtype, dev, alpha, eps = x.shape, x.dtype, x.get_device(), float(alpha), float(eps)
    if res is not None:
        if res_dtype not in (None, res.dtype):
            raise ValueError("res_dtype is res's dtype when res is given")
        res_dtype = res.dtype
    elif res_dtype is None:
        res_dtype = dtype
    _, ref = _descriptor((shape, dtype, res_dtype, kind, eps, alpha),
                         lambda: _addnorm_problem(x, res_dtype, kind, eps, alpha))
    cols = shape[-1:]
    px = _ptr_of("x", x, shape, dtype, dev)
    pr = _ptr_of("res", res, shape, res_dtype, dev)
    pw = _ptr_of("w", w, cols, _f32, dev)
    ps = _ptr_of("rscale", rscale, cols, _f32, dev)
    y = torch.empty_like(x)
    r = torch.empty_like(x) if res_dtype is dtype else torch.empty_like(x, dtype=res_dtype)
    _launch("gla_addnorm_fwd", _lib.lib.gla_addnorm_fwd, dev, (ref, px, pr, ps, pw, r.data_ptr(), y.data_ptr()))
    return r, y


def _partials(name, workspace, nbytes, dev, like):
    """(address, bytes) of the workspace for the partial rows of column sums; none is needed where a single
    block writes them (256 bytes or less)."""
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, name)
    if workspace is None:
        if nbytes <= 256:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return workspace, _buffer("workspace", workspace, nbytes, dev), nbytes


def gla_addnorm_bwd(x, r, w, dy, dr=None, *, rscale=None, alpha: float = 1.0, kind: str = "rms", eps: float = 1e-6,
                    output_dx: bool = True,
                    workspace: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of sum(dy * y) + sum(dr * r) of gla_addnorm_fwd at the r it returned: dict dres
    (r's dtype), dx (dy's dtype; None when output_dx is False: with alpha = 1, no rscale and one
    dtype it equals dres), dw (fp32 [D], None without w) and drscale (fp32 [D], None without
    rscale). x is only read for drscale and may be None without rscale; dr [..., D] is the
    gradient that reaches r from later blocks, or None."""
    if not dy.is_cuda:
        return _from_host(gla_addnorm_bwd, (x, _need("r", r), w, dy, dr),
                          dict(rscale=rscale, alpha=alpha, kind=kind, eps=eps, output_dx=output_dx,
                               workspace=workspace))
    shape, dtype, dev, res_dtype = dy.shape, dy.dtype, dy.get_device(), _need("r", r).dtype
    alpha, eps = float(alpha), float(eps)
    _, ref = _descriptor((shape, dtype, res_dtype, kind, eps, alpha),
                         lambda: _addnorm_problem(dy, res_dtype, kind, eps, alpha))
    cols = shape[-1:]
    pdy = _ptr_of("dy", dy, shape, dtype, dev)
    pr = _ptr_of("r", r, shape, res_dtype, dev)
    pdr = _ptr_of("dr", dr, shape, res_dtype, dev)
    pw = _ptr_of("w", w, cols, _f32, dev)
    px = ps = ds = None
    if rscale is not None:
        ps = _ptr_of("rscale", rscale, cols, _f32, dev)
        px = _ptr_of("x (for rscale's gradient)", _need("x (for rscale's gradient)", x), shape, dtype, dev)
        ds = torch.empty_like(rscale)
    ws, pws, nbytes = _partials("gla_addnorm_workspace_bytes", workspace, _lib.lib.gla_addnorm_workspace_bytes(ref),
                                dev, dy)
    dres = torch.empty_like(r)
    dx = torch.empty_like(dy) if output_dx else None
    dw = torch.empty_like(w) if w is not None else None
    _launch("gla_addnorm_bwd", _lib.lib.gla_addnorm_bwd, dev,
            (ref, px, pr, ps, pw, pdy, pdr, dres.data_ptr(), None if dx is None else dx.data_ptr(),
             None if dw is None else dw.data_ptr(), None if ds is None else ds.data_ptr(), pws, nbytes))
    return {"dres": dres, "dx": dx, "dw": dw, "drscale": ds}


def _headnorm_problem(o, w, act, kind, eps) -> GlaNormProblem:
    if o.dim() != 4:
        raise ValueError("o must be [B, H, L, D]")
    B, H, L, D = _sizes("o's sizes", *o.shape)
    io = _io_dtype(o.dtype)
    return GlaNormProblem(B, H, L, D, io, io, _choice("kind", kind, _NORM_KINDS), _choice("act", act, _ACTS),
                          1 if w is not None and w.dim() == 2 else 0, eps, 1.0)


def gla_headnorm_fwd(o, z=None, w=None, *, act: str = "silu", kind: str = "rms", eps: float = 1e-6) -> torch.Tensor:
    """Norm and gate after a cell: y = norm(o) * w * act(z), normalised over the D channels of each
    head and token. o [B,H,L,D] (bf16 or fp32) as the cells return it; z [B,L,H,D] the gate before
    act ("silu" or "sigmoid"), None: no gate; w fp32 [D] (shared by the heads) or [H,D], None: one;
    kind "rms" or "layer". Returns y [B,L,H,D]: y.view(B, L, H * D) is the out-projection's input.
    Host tensors are copied to the current device and the result back."""
    if not o.is_cuda:
        return _from_host(gla_headnorm_fwd, (o, z, w), dict(act=act, kind=kind, eps=eps))
    shape, dtype, dev, eps = o.shape, o.dtype, o.get_device(), float(eps)
    heads = w is not None and w.dim() == 2
    _, ref = _descriptor((shape, dtype, heads, act, kind, eps), lambda: _headnorm_problem(o, w, act, kind, eps))
    B, H, L, D = shape
    tokens = (B, L, H, D)
    po = _ptr_of("o", o, shape, dtype, dev)
    pz = _ptr_of("z", z, tokens, dtype, dev)
    pw = _ptr_of("w", w, (H, D) if heads else (D,), _f32, dev)
    y = o.new_empty(tokens)
    _launch("gla_headnorm_fwd", _lib.lib.gla_headnorm_fwd, dev, (ref, po, pz, pw, y.data_ptr()))
    return y


def gla_headnorm_bwd(o, z, w, dy, *, act: str = "silu", kind: str = "rms", eps: float = 1e-6,
                     workspace: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of sum(dy * y) of gla_headnorm_fwd: dict do [B,H,L,D], dz [B,L,H,D] (None without
    z), dw (fp32, shaped like w; None without w)."""
    if not o.is_cuda:
        return _from_host(gla_headnorm_bwd, (o, z, w, _need("dy", dy)),
                          dict(act=act, kind=kind, eps=eps, workspace=workspace))
    shape, dtype, dev, eps = o.shape, o.dtype, o.get_device(), float(eps)
    heads = w is not None and w.dim() == 2
    _, ref = _descriptor((shape, dtype, heads, act, kind, eps), lambda: _headnorm_problem(o, w, act, kind, eps))
    B, H, L, D = shape
    tokens = (B, L, H, D)
    po = _ptr_of("o", o, shape, dtype, dev)
    pz = _ptr_of("z", z, tokens, dtype, dev)
    pdy = _ptr_of("dy", _need("dy", dy), tokens, dtype, dev)
    pw = _ptr_of("w", w, (H, D) if heads else (D,), _f32, dev)
    ws, pws, nbytes = _partials("gla_headnorm_workspace_bytes", workspace, _lib.lib.gla_headnorm_workspace_bytes(ref),
                                dev, o)
    d_o = torch.empty_like(o)
    dz = torch.empty_like(z) if z is not None else None
    dw = torch.empty_like(w) if w is not None else None
    _launch("gla_headnorm_bwd", _lib.lib.gla_headnorm_bwd, dev,
            (ref, po, pz, pw, pdy, d_o.data_ptr(), None if dz is None else dz.data_ptr(),
             None if dw is None else dw.data_ptr(), pws, nbytes))
    return {"do": d_o, "dz": dz, "dw": dw}


def gla_shard_state(k, v, g=None, igate=None, *, chunk: int = 64) -> Tuple[torch.Tensor, torch.Tensor]:
    """(state, gamma) of one sequence shard: its end state from a zero initial state
    [B,H,Dk,Dv] and its total log-decay per key dim [B,H,Dk], both fp32 on the GPU."""
    device = k.device
    prob = make_problem(k, v, g, scale=1.0, chunk=chunk, plan="tc")
    B, H, _, Dk = k.shape
    state = torch.empty(B, H, Dk, v.shape[-1], dtype=torch.float32, device=device)
    gamma = torch.empty(B, H, Dk, dtype=torch.float32, device=device)
    nb = max(int(_lib.lib.gla_shard_workspace_bytes(ctypes.byref(prob))), 256)
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    st = _lib.lib.gla_shard_state(ctypes.byref(prob), _ptr(k), _ptr(v), _ptr(g), _ptr(igate), _ptr(state),
                                  _ptr(gamma), _ptr(ws), nb, _stream_handle(device))
    _check(st, "gla_shard_state")
    return state, gamma


def gla_shard_state_grad(q, dO, g=None, *, scale: Optional[float] = None,
                         chunk: int = 64) -> Tuple[torch.Tensor, torch.Tensor]:
    """(state_grad, gamma) of one sequence shard: the gradient w.r.t. the state before its
    first token from its own outputs alone [B,H,Dk,Dv], and its total log-decay per key dim
    [B,H,Dk], both fp32 on the GPU."""
    device = q.device
    prob = make_problem(q, dO, g, scale=scale, chunk=chunk, plan="tc")
    B, H, _, Dk = q.shape
    dS = torch.empty(B, H, Dk, dO.shape[-1], dtype=torch.float32, device=device)
    gamma = torch.empty(B, H, Dk, dtype=torch.float32, device=device)
    nb = max(int(_lib.lib.gla_shard_workspace_bytes(ctypes.byref(prob))), 256)
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    st = _lib.lib.gla_shard_state_grad(ctypes.byref(prob), _ptr(q), _ptr(dO), _ptr(g), _ptr(dS), _ptr(gamma),
                                       _ptr(ws), nb, _stream_handle(device))
    _check(st, "gla_shard_state_grad")
    return dS, gamma


def gla_state_fold(states: torch.Tensor, gammas: torch.Tensor, count: int,
                   h0: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The state after the first `count` shards, given all shards' (state, gamma) stacked along
    a leading shard axis ([n,B,H,Dk,Dv], [n,B,H,Dk]), starting from h0 (or 0)."""
    if states.dim() != 5 or gammas.dim() != 4 or not (0 <= count <= states.shape[0]):
        raise ValueError("states [n,B,H,Dk,Dv], gammas [n,B,H,Dk], 0 <= count <= n")
    _, B, H, Dk, Dv = states.shape
    prob = GlaProblem(B, H, 1, Dk, Dv, 64, 1.0, _lib.GLA_F32, _lib.GLA_GATE_PER_KEY, _PLANS["auto"])
    out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=states.device)
    st = _lib.lib.gla_state_fold(ctypes.byref(prob), int(count), _ptr(states.contiguous()), _ptr(gammas.contiguous()),
                                 _ptr(h0), _ptr(out), _stream_handle(states.device))
    _check(st, "gla_state_fold")
    return out


def gla_fwd_sequence_sharded(q, k, v, g=None, igate=None, h0=None, *, scale: Optional[float] = None,
                             chunk: int = 64, group=None, _shard_ops=None):
    """Forward over a sequence cut into contiguous shards, one per rank of `group` (rank order =
    sequence order): each rank passes its own shard of q, k, v, g, igate (and every rank the
    same h0), and gets its shard's o and end state (the last rank's is the sequence's hT).
    One all-gather of the shards' (end state from zero, total log-decay) is the only exchange.
    _shard_ops replaces the three per-rank steps (shard_state, fold, forward) for tests of the
    exchange on CPU ranks."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    rank = dist.get_rank(group)
    shard_state, fold, fwd = _shard_ops or (
        lambda: gla_shard_state(k, v, g, igate, chunk=chunk),
        lambda states, gammas: gla_state_fold(states, gammas, rank, h0),
        lambda s_in: gla_fwd(q, k, v, g, igate, s_in, scale=scale, chunk=chunk))
    state, gamma = shard_state()
    parts_s = [torch.empty_like(state) for _ in range(world)]
    parts_g = [torch.empty_like(gamma) for _ in range(world)]
    dist.all_gather(parts_s, state.contiguous(), group=group)
    dist.all_gather(parts_g, gamma.contiguous(), group=group)
    return fwd(fold(torch.stack(parts_s), torch.stack(parts_g)))


def gla_bwd_sequence_sharded(q, k, v, g, igate, h0, dO, dhT=None, *, scale: Optional[float] = None,
                             chunk: int = 64, group=None, _shard_ops=None) -> Dict[str, Optional[torch.Tensor]]:
    """Backward over a sequence cut into contiguous shards, one per rank of `group` (rank order =
    sequence order): each rank passes its own shard of q, k, v, g, igate, dO, and every rank the
    same h0 and dhT (the gradient at the sequence's end). Returns gla_bwd's dict for the rank's
    shard; rank 0's dh0 is the sequence's, the other ranks' dh0 is None. One all-gather of the
    shards' (end state from zero, start-state gradient from zero, total log-decay) is the only
    exchange: rank r's initial state folds shards 0..r-1 from h0, the gradient at its end folds
    shards P-1..r+1 in reverse order from dhT. _shard_ops replaces the per-rank steps
    (shard_state, shard_state_grad, fold, backward) for tests of the exchange on CPU ranks."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    rank = dist.get_rank(group)
    shard_state, shard_grad, fold, bwd = _shard_ops or (
        lambda: gla_shard_state(k, v, g, igate, chunk=chunk),
        lambda: gla_shard_state_grad(q, dO, g, scale=scale, chunk=chunk),
        gla_state_fold,
        lambda s_in, d_end: gla_bwd(q, k, v, g, igate, s_in, dO, d_end, scale=scale, chunk=chunk,
                                    output_dh0=rank == 0))
    S, gamma = shard_state()
    dS, _ = shard_grad()
    n_s, n_g = S.numel(), gamma.numel()
    pack = torch.cat([S.reshape(-1), dS.reshape(-1), gamma.reshape(-1)])
    parts = [torch.empty_like(pack) for _ in range(world)]
    dist.all_gather(parts, pack, group=group)
    allp = torch.stack(parts)
    states = allp[:, :n_s].reshape(world, *S.shape)
    grads = allp[:, n_s:2 * n_s].reshape(world, *S.shape)
    gammas = allp[:, 2 * n_s:2 * n_s + n_g].reshape(world, *gamma.shape)
    s_in = fold(states, gammas, rank, h0)
    d_end = fold(grads.flip(0).contiguous(), gammas.flip(0).contiguous(), world - 1 - rank, dhT)
    return bwd(s_in, d_end)


def _check_saved(saved, prob):
    if saved is None:
        return
    if saved.device.type != "cuda" or saved.dtype != torch.float32 or not saved.is_contiguous():
        raise ValueError("saved_states must be a contiguous float32 CUDA tensor")
    if saved.numel() * 4 < gla_saved_states_bytes(prob):
        raise GlaError(_lib.GLA_ERR_WORKSPACE, "saved_states")


def gla_bwd(q, k, v, g, igate, h0, dO, dhT=None, *, scale: Optional[float] = None, chunk: int = 64,
            plan: str = "auto", output_dh0: bool = True,
            workspace: Optional[torch.Tensor] = None,
            saved_states: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Backward pass. Returns dict dq, dk, dv, dg (None if ungated), di (None without an
    input gate), dh0 (None when output_dh0 is False). saved_states: the buffer a gla_fwd on
    the same inputs filled, or None to recompute."""
    host = q.device.type != "cuda"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    q, k, v, g, igate, h0, dO, dhT = (_to_dev(t, device) for t in (q, k, v, g, igate, h0, dO, dhT))
    prob = make_problem(q, v, g, scale=scale, chunk=chunk, plan=plan)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    dg = torch.empty_like(g) if g is not None else None
    di = torch.empty_like(igate) if igate is not None else None
    dh0 = torch.empty(q.shape[0], q.shape[1], q.shape[-1], v.shape[-1], dtype=torch.float32,
                      device=device) if output_dh0 else None
    nbytes = gla_workspace_bytes(prob, True)
    if nbytes == 0:
        raise GlaError(_lib.GLA_ERR_UNSUPPORTED, "gla_workspace_bytes")
    ws = _workspace(nbytes, device, workspace)
    _check_saved(saved_states, prob)
    st = _lib.lib.gla_bwd_saved(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(igate), _ptr(h0),
                                _ptr(dO), _ptr(dhT), _ptr(saved_states), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                                _ptr(di), _ptr(dh0), _ptr(ws), ws.numel() * ws.element_size(),
                                _stream_handle(device))
    _check(st, "gla_bwd")
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "di": di, "dh0": dh0}
    if host:
        names = list(out)
        out = dict(zip(names, _to_host([out[n] for n in names])))
    return out


def gla_check_device_status(workspace: torch.Tensor) -> int:
    device = workspace.device
    return int(_lib.lib.gla_check_device_status(_ptr(workspace), _stream_handle(device)))
