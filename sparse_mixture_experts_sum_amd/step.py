"""The layer norms around the layer with their gradient, and the experts' update step.

Bindings of the entry points in the section "A training step's other ends" of
``include/moe.h``, in the manner of ``training.py``: tensor metadata is checked, outputs and
workspaces are allocated with torch, and pointers and the current HIP stream of the tensors'
device are passed on.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from .training import _F32, _call, _matrix, _pointers, _scratch, _type, _workspace_bytes

# the structs of include/moe.h, native alignment
_NORM_SHAPE = struct.Struct("@qqiff0q").pack
_ORTH_SHAPE = struct.Struct("@qqiiiffff0q").pack
_MUON_PARAMS = struct.Struct("@ffffi").pack

NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def declare(lib):
    """Argument types of the entry points (called once by load_library). The structs are passed
    as bytes."""
    P, SZ = ctypes.c_void_p, ctypes.c_size_t
    lib.moe_layer_norm.argtypes = [P] * 10
    lib.moe_layer_norm_backward_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
    lib.moe_layer_norm_backward.argtypes = [P] * 12 + [SZ, P]
    lib.moe_orthogonalize_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
    lib.moe_orthogonalize.argtypes = [P] * 4 + [SZ, P]
    lib.moe_muon_update.argtypes = [P] * 6 + [SZ, P]
    for name in ("moe_layer_norm", "moe_layer_norm_backward_workspace_size", "moe_layer_norm_backward",
                 "moe_orthogonalize_workspace_size", "moe_orthogonalize", "moe_muon_update"):
        getattr(lib, name).restype = ctypes.c_int32


def moe_layer_norm(x, gamma, beta=None, *, y=None, residual_scale=1.0, eps=1e-5, want_stats=True) -> dict:
    """Layer norm of the residual sum, in one pass:

    out = residual_scale * x + y   (x itself without y)
    u = (out - mean(out)) / sqrt(var(out) + eps) * gamma + beta

    x [T,d] bf16 or fp32; y [T,d] fp32, moe_forward's output; gamma, beta [d] fp32 (beta may be
    None). Returns out and u (x's type) and, for the gradient, mean and rstd = 1 / sqrt(var + eps),
    [T] fp32 (None without want_stats). residual_scale belongs to y: without it, it has to be 1."""
    T, d = rows = _matrix(x, "x", "d")
    if gamma is None:
        raise ValueError("moe_layer_norm needs gamma")
    if y is None and residual_scale != 1.0:
        raise ValueError("residual_scale belongs to the sum with y")
    dev = x.device
    s = _NORM_SHAPE(T, d, _type(x), eps, residual_scale)
    px, py, pg, pb = _pointers(((x, "x", rows, x.dtype), (y, "y", rows, _F32), (gamma, "gamma", (d,), _F32),
                                (beta, "beta", (d,), _F32)), dev)
    out = mean = rstd = pout = pm = pr = None
    if y is not None:
        out = torch.empty_like(x)
        pout = out.data_ptr()
    u = torch.empty_like(x)
    if want_stats:
        mean, rstd = torch.empty(T, dtype=_F32, device=dev), torch.empty(T, dtype=_F32, device=dev)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
    _call("moe_layer_norm", dev, s, px, py, pg, pb, pout, u.data_ptr(), pm, pr)
    return {"out": x if y is None else out, "u": u, "mean": mean, "rstd": rstd}


def moe_layer_norm_backward(out, d_u, mean, rstd, gamma, *, d_out=None, residual_scale=1.0, want_dy=False,
                            workspace=None) -> dict:
    """Gradient of moe_layer_norm. out is the forward's `out` (x where it had no y), d_u and d_out
    the gradients of u and out (d_out may be None). Returns dx and, with want_dy, dy (out's type;
    dx = residual_scale * dy) and dgamma and dbeta [d] (fp32)."""
    T, d = rows = _matrix(out, "out", "d")
    if d_u is None or mean is None or rstd is None or gamma is None:
        raise ValueError("moe_layer_norm_backward needs d_u, mean, rstd and gamma")
    dev, dtype = out.device, out.dtype
    s = _NORM_SHAPE(T, d, _type(out), 1.0, residual_scale)
    po, pdu, pdo, pm, pr, pg = _pointers(
        ((out, "out", rows, dtype), (d_u, "d_u", rows, dtype), (d_out, "d_out", rows, dtype),
         (mean, "mean", (T,), _F32), (rstd, "rstd", (T,), _F32), (gamma, "gamma", (d,), _F32)), dev)
    ws = pws = None
    ws_bytes = _workspace_bytes("moe_layer_norm_backward_workspace_size", s)
    if ws_bytes:
        ws, ws_bytes = _scratch("moe_layer_norm_backward_workspace_size", s, dev, workspace)
        pws = ws.data_ptr()
    dx = torch.empty_like(out)
    dy = torch.empty_like(out) if want_dy else None
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
    _call("moe_layer_norm_backward", dev, s, po, pdu, pdo, pm, pr, pg, dx.data_ptr(),
          None if dy is None else dy.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), pws, ws_bytes)
    return {"dx": dx, "dy": dy, "dgamma": dgamma, "dbeta": dbeta}


def _matrices(t, name):
    """(E, m, n) of a matrix or a stack of them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [m, n] or [E, m, n], got shape {tuple(t.shape)}")
    E = t.shape[0] if t.dim() == 3 else 1
    m, n = t.shape[-2:]
    if E < 1 or m < 1 or n < 1:
        raise ValueError(f"{name} has no elements: shape {tuple(t.shape)}")
    return E, m, n


def _overlap(a, b):
    """Whether two contiguous tensors share memory."""
    pa, pb = a.data_ptr(), b.data_ptr()
    return pa < pb + b.numel() * b.element_size() and pb < pa + a.numel() * a.element_size()


def _orth_shape(t, E, m, n, steps, coefficients, eps):
    if len(coefficients) != 3:
        raise ValueError("coefficients are three numbers: a, b, c")
    if not isinstance(steps, int) or steps < 1:
        raise ValueError(f"steps must be a whole number of 1 or more, got {steps!r}")
    a, b, c = (float(v) for v in coefficients)
    if not all(math.isfinite(v) for v in (a, b, c, eps)) or eps < 0:
        raise ValueError("coefficients and eps must be finite, eps not negative")
    return _ORTH_SHAPE(m, n, E, _type(t), steps, a, b, c, eps)


def moe_orthogonalize(g, *, steps=5, coefficients=NEWTON_SCHULZ, eps=1e-7, out=None, workspace=None) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of a matrix [m,n], or of each of a stack [E,m,n] of them (E
    up to 64), bf16 or fp32:

    X = g / (|g| + eps), then `steps` times  X = a X + (b A + c A^2) X with A = X X^T

    (of the transpose where m > n). `out` (g itself may be given) takes the result, of g's type.
    bf16 matrices whose sides are both over 128 may be computed in fp16 with fp32 sums: within
    2e-3 of the norm beside the result's own rounding, at a rank below the sides within 2e-2 (rows
    or columns far smaller than the others may be off by more of themselves). Others, and those of more steps than the bound allows (five of the default coefficients), are
    computed as in fp32."""
    E, m, n = _matrices(g, "g")
    dev = g.device
    s = _orth_shape(g, E, m, n, steps, coefficients, eps)
    pg, pout = _pointers(((g, "g", g.shape, g.dtype), (out, "out", g.shape, g.dtype)), dev)
    if out is not None and pout != pg and _overlap(g, out):
        raise ValueError("out must be g itself or apart from it")
    ws, ws_bytes = _scratch("moe_orthogonalize_workspace_size", s, dev, workspace)
    if out is None:
        out = torch.empty_like(g)
        pout = out.data_ptr()
    _call("moe_orthogonalize", dev, s, pg, pout, ws.data_ptr(), ws_bytes)
    return out


def _muon_args(w, g, m, lr, momentum, nesterov, weight_decay, scale, steps, coefficients, eps):
    """An update's tensors and numbers, checked: (shape, arguments of the call before its workspace)."""
    E, rows, cols = _matrices(w, "w")
    dev, dtype = w.device, w.dtype
    if not all(math.isfinite(v) for v in (lr, momentum, weight_decay, scale)):
        raise ValueError("lr, momentum, weight_decay and scale must be finite")
    if g is None or m is None:
        raise ValueError("moe_muon_update needs g and m")
    s = _orth_shape(w, E, rows, cols, steps, coefficients, eps)
    pw, pg, pm = _pointers(((w, "w", w.shape, dtype), (g, "g", w.shape, dtype), (m, "m", w.shape, _F32)), dev)
    if _overlap(w, g) or _overlap(w, m) or _overlap(g, m):
        raise ValueError("w, g and m must be three tensors that share no memory")
    return s, (dev, s, _MUON_PARAMS(lr, momentum, weight_decay, scale, 1 if nesterov else 0), pw, pg, pm)


def moe_muon_update(w, g, m, *, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, steps=5,
                    coefficients=NEWTON_SCHULZ, eps=1e-7, workspace=None) -> torch.Tensor:
    """One step of orthogonalised updates with momentum, in place, of a matrix or a stack of them:

    m = momentum * m + g;  u = g + momentum * m (nesterov) or m
    w = (1 - lr * weight_decay) * w - lr * scale * moe_orthogonalize(u)

    w, g [m,n] or [E,m,n] bf16 or fp32, m fp32 of their shape. The update is rounded with w alone.
    Returns the workspace, for the next call."""
    s, args = _muon_args(w, g, m, lr, momentum, nesterov, weight_decay, scale, steps, coefficients, eps)
    ws, ws_bytes = _scratch("moe_orthogonalize_workspace_size", s, w.device, workspace)
    _call("moe_muon_update", *args, ws.data_ptr(), ws_bytes)
    return ws


def _muon_updates(updates, *, lr, momentum=0.95, nesterov=True, weight_decay=0.0, steps=5, coefficients=NEWTON_SCHULZ,
                  eps=1e-7, workspace=None) -> torch.Tensor:
    """moe_muon_update of each (w, g, m, scale), on one workspace, which it returns: all are checked and the
    workspace is there before the first is launched, so that a refused call changes nothing."""
    calls = [_muon_args(w, g, m, lr, momentum, nesterov, weight_decay, scale, steps, coefficients, eps)
             for w, g, m, scale in updates]
    dev = calls[0][1][0]
    if any(args[0] != dev for _, args in calls):
        raise ValueError("the weights must be on one device")
    largest = max((s for s, _ in calls), key=lambda s: _workspace_bytes("moe_orthogonalize_workspace_size", s))
    ws, ws_bytes = _scratch("moe_orthogonalize_workspace_size", largest, dev, workspace)
    if ws.data_ptr() % 256:
        raise ValueError("workspace must be 256-byte aligned")
    for _, args in calls:
        _call("moe_muon_update", *args, ws.data_ptr(), ws_bytes)
    return ws
