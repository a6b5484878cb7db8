"""Python binding of the gated delta rule (``include/ssd_delta.h``): argument marshalling only.

Tensors of a batched call are q, k [B,T,G,N], v [B,T,H,P], log_a, beta [B,T,H]; of a packed call (``cu_seqlens`` given)
q, k [T,G,N], v [T,H,P], log_a, beta [T,H].  States are [nseq,H,N,P] fp32.  One token's heads are dense; q, k and v may be
views of wider rows, such as a fused projection's output.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPE_CODE, _in_stream, _on_stream, load_library
from .attention import _addr, _call, _dense, _offsets, _stride, _workspace


class DeltaDims(ctypes.Structure):
    """Mirror of ``ssd_delta_dims``."""
    _fields_ = [("nseq", ctypes.c_int64), ("total", ctypes.c_int64), ("nheads", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("keydim", ctypes.c_int64), ("valuedim", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


def declare(lib):
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(DeltaDims)
    lib.ssd_delta_forward_workspace_bytes.argtypes = [dp]
    lib.ssd_delta_forward_workspace_bytes.restype = sz
    lib.ssd_delta_forward.argtypes = [dp] + [vp] * 10 + [sz, vp]
    lib.ssd_delta_forward.restype = i32
    lib.ssd_delta_backward_workspace_bytes.argtypes = [dp]
    lib.ssd_delta_backward_workspace_bytes.restype = sz
    lib.ssd_delta_backward.argtypes = [dp] + [vp] * 16 + [sz, vp]
    lib.ssd_delta_backward.restype = i32
    lib.ssd_delta_step.argtypes = [dp] + [vp] * 8
    lib.ssd_delta_step.restype = i32


def _dims(q, k, v, log_a, beta, cu_seqlens, scale, dim):
    """ssd_delta_dims of a call, its arguments checked; dim: of q, without cu_seqlens 4, or 3 for one token each."""
    dev = q.device
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("q must be float32 or bfloat16, got %s" % q.dtype)
    strides = _stride(q, "q", dim, q.dtype, dev), _stride(k, "k", dim, q.dtype, dev), _stride(v, "v", dim, q.dtype, dev)
    if k.shape != q.shape or v.shape[:-2] != q.shape[:-2]:
        raise ValueError("q, k and v must have the same tokens, and q and k be alike: q %s, k %s, v %s"
                         % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    G, N = q.shape[-2:]
    H, P = v.shape[-2:]
    if G < 1 or H % G != 0:
        raise ValueError("v's %d heads are not a multiple of k's %d" % (H, G))
    _dense(log_a, "log_a", v.shape[:-1], torch.float32, dev)
    _dense(beta, "beta", v.shape[:-1], torch.float32, dev)
    if cu_seqlens is not None:
        _offsets(cu_seqlens, "cu_seqlens", dev)
        nseq, total = cu_seqlens.numel() - 1, q.shape[0]
    elif dim == 4:
        nseq, total = q.shape[0], q.shape[0] * q.shape[1]
    else:
        nseq = total = q.shape[0]
    return DeltaDims(nseq, total, H, G, N, P, *strides, N ** -0.5 if scale is None else float(scale), _DTYPE_CODE[q.dtype])


def ssd_delta_forward_workspace_bytes(dims: DeltaDims) -> int:
    return int(load_library().ssd_delta_forward_workspace_bytes(ctypes.byref(dims)))


@_in_stream
def ssd_delta_forward(q, k, v, log_a, beta, cu_seqlens=None, scale=None, init_state=None, y=None, final_state=None,
                      workspace=None, stream=None):
    """Run ``ssd_delta_forward``: S = a (I - beta k k^T) S + beta k v^T and y = scale S^T q, token by token, a = exp(log_a).

    ``cu_seqlens``: int64 offsets [nseq + 1] on the GPU of a packed batch.  ``scale`` defaults to N ** -0.5.  ``y`` is
    allocated when not given; ``final_state`` may be a tensor to write (init_state itself among them), True to allocate one, or
    None/False to skip it.  Keys are expected to be of about unit length.  Tokens of no sequence are not written.
    Returns (y, final_state)."""
    dims = _dims(q, k, v, log_a, beta, cu_seqlens, scale, 4 if cu_seqlens is None else 3)
    dev, states = q.device, (dims.nseq, dims.nheads, dims.keydim, dims.valuedim)
    _dense(init_state, "init_state", states, torch.float32, dev)
    if y is None:
        y = torch.empty(v.shape, dtype=q.dtype, device=dev)
    _dense(y, "y", v.shape, q.dtype, dev)
    if final_state is True:
        final_state = torch.empty(states, dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    _dense(final_state, "final_state", states, torch.float32, dev)
    workspace, ws_bytes = _workspace(workspace, ssd_delta_forward_workspace_bytes(dims), dev)
    _on_stream(stream, q, k, v, log_a, beta, cu_seqlens, init_state, y, final_state, workspace)
    _call("ssd_delta_forward", dev, stream, ctypes.byref(dims), _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(log_a),
          _addr(beta), _addr(init_state), _addr(y), _addr(final_state), _addr(workspace), ws_bytes)
    return y, final_state


def ssd_delta_backward_workspace_bytes(dims: DeltaDims) -> int:
    return int(load_library().ssd_delta_backward_workspace_bytes(ctypes.byref(dims)))


@_in_stream
def ssd_delta_backward(q, k, v, log_a, beta, dy, cu_seqlens=None, scale=None, init_state=None, dfinal=None, want_dinit=None,
                       workspace=None, stream=None):
    """Run ``ssd_delta_backward``: the gradients of <dy, y> + <dfinal, final_state> for ssd_delta_forward, whose arguments
    these are.  Returns a dict: dq, dk, dv (dtype of q, dense), dlog_a, dbeta (fp32), and dinit where an init_state is
    given (want_dinit=False skips it, True returns it without one).  Tokens of no sequence are not written."""
    dims = _dims(q, k, v, log_a, beta, cu_seqlens, scale, 4 if cu_seqlens is None else 3)
    dev, states = q.device, (dims.nseq, dims.nheads, dims.keydim, dims.valuedim)
    _dense(dy, "dy", v.shape, q.dtype, dev)
    _dense(init_state, "init_state", states, torch.float32, dev)
    _dense(dfinal, "dfinal", states, torch.float32, dev)
    out = {"d" + n: torch.empty(t.shape, dtype=q.dtype, device=dev) for n, t in (("q", q), ("k", k), ("v", v))}
    out["dlog_a"] = torch.empty(log_a.shape, dtype=torch.float32, device=dev)
    out["dbeta"] = torch.empty(beta.shape, dtype=torch.float32, device=dev)
    if init_state is not None if want_dinit is None else want_dinit:
        out["dinit"] = torch.empty(states, dtype=torch.float32, device=dev)
    workspace, ws_bytes = _workspace(workspace, ssd_delta_backward_workspace_bytes(dims), dev)
    _on_stream(stream, q, k, v, log_a, beta, dy, cu_seqlens, init_state, dfinal, workspace, *out.values())
    _call("ssd_delta_backward", dev, stream, ctypes.byref(dims), _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(log_a),
          _addr(beta), _addr(init_state), _addr(dy), _addr(dfinal), _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]),
          _addr(out["dlog_a"]), _addr(out["dbeta"]), _addr(out.get("dinit")), _addr(workspace), ws_bytes)
    return out


@_in_stream
def ssd_delta_step(state, q_t, k_t, v_t, log_a_t, beta_t, scale=None, y_t=None, stream=None):
    """Run ``ssd_delta_step``: one token for each sequence, ``state`` [nseq,H,N,P] fp32 updated in place.  q_t, k_t
    [nseq,G,N], v_t [nseq,H,P], log_a_t, beta_t [nseq,H].  Returns y_t [nseq,H,P]."""
    dims = _dims(q_t, k_t, v_t, log_a_t, beta_t, None, scale, 3)
    dev = q_t.device
    _dense(state, "state", (dims.nseq, dims.nheads, dims.keydim, dims.valuedim), torch.float32, dev)
    if y_t is None:
        y_t = torch.empty(v_t.shape, dtype=q_t.dtype, device=dev)
    _dense(y_t, "y_t", v_t.shape, q_t.dtype, dev)
    _on_stream(stream, state, q_t, k_t, v_t, log_a_t, beta_t, y_t)
    _call("ssd_delta_step", dev, stream, ctypes.byref(dims), _addr(state), _addr(q_t), _addr(k_t), _addr(v_t), _addr(log_a_t),
          _addr(beta_t), _addr(y_t))
    return y_t
