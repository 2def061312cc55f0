"""The layer's training operators: products grouped by expert, the experts' and the router's
gradients, and the norms around the layer with their gradient.

Bindings of the entry points in the "Training" section of ``include/moe.h``; like the
forward's, they check tensor metadata, allocate outputs and workspaces with torch and pass
pointers and the current HIP stream of the tensors' device.

The smallest calls are bound by the host: a call checks each tensor once, in one expression,
and only a failed check goes through the binding's full checks for its error; shape structs
travel as packed bytes; the workspace size of a shape is asked for once.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import (MOE_BF16, MOE_FP32, MOE_TOKEN_CHOICE, _check, _dtype_name, _need, _shape_is,
               load_library)

MATMUL_FORMS = {"nn": 0, "nt": 1, "tn": 2}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_TYPES = {_BF16: MOE_BF16, _F32: MOE_FP32}

# the structs of include/moe.h, native alignment
_MATMUL_SHAPE = struct.Struct("@qqqqqiiiii0q").pack
_SWIGLU_SHAPE = struct.Struct("@qqqiii0q").pack
_ROUTE_UPSTREAM = struct.Struct("@PiffPPPq0q").pack
_NORM_SHAPE = struct.Struct("@qqiiff0q").pack
_LAYER_SHAPE = struct.Struct("@qqqiiiii0dd").pack


def declare(lib):
    """Argument types of the training entry points (called once by load_library). The shape
    structs are passed as bytes."""
    P, SZ = ctypes.c_void_p, ctypes.c_size_t
    lib.moe_grouped_matmul.argtypes = [P] * 8 + [SZ, P]
    lib.moe_grouped_matmul_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
    lib.moe_swiglu_backward.argtypes = [P] * 13
    lib.moe_route_backward_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
    lib.moe_route_backward.argtypes = [P] * 13 + [SZ, P]
    lib.moe_block_norm.argtypes = [P] * 11
    lib.moe_block_norm_backward_workspace_size.argtypes = [P, ctypes.POINTER(SZ)]
    lib.moe_block_norm_backward.argtypes = [P] * 16 + [SZ, P]
    for name in ("moe_grouped_matmul", "moe_grouped_matmul_workspace_size", "moe_swiglu_backward", "moe_route_backward_workspace_size",
                 "moe_route_backward", "moe_block_norm", "moe_block_norm_backward_workspace_size",
                 "moe_block_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int32


def _matrix(t, name, width="width"):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, {width}], got shape {tuple(t.shape)}")
    return t.shape


def _vector(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 1:
        raise ValueError(f"{name} must have one dimension, got shape {tuple(t.shape)}")
    return t.shape[0]


def _type(t) -> int:
    dt = _TYPES.get(t.dtype)
    return dt if dt is not None else _dtype_name(t)  # (raises)


def _pointers(tensors, dev):
    """Addresses of (tensor, name, shape, dtype) entries, None for None: every tensor of that
    shape and type, contiguous and on dev."""
    out = []
    index = dev.index
    for t, _, shape, dtype in tensors:
        if t is None:
            out.append(None)
        elif (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
              and t.get_device() == index and t.is_contiguous()):
            out.append(t.data_ptr())
        else:
            break
    else:
        if index is not None:  # (a host tensor has no index)
            return out
    for t, name, shape, _ in tensors:
        _shape_is(t, name, shape)
    for t, name, _, dtype in tensors:
        _need(t, name, dtype, dev)
    raise TypeError("tensors must be CUDA (HIP) tensors")


def _call(fn: str, dev: torch.device, *args):
    """One library call on dev's current stream, with dev the current device."""
    f = getattr(load_library(), fn)
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream  # (torch.cuda.current_stream builds an object)
    if torch.cuda.current_device() == index:
        st = f(*args, stream(index))
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream(index))
    if st:
        _check(fn, st)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(fn: str, shape: bytes) -> int:
    n = ctypes.c_size_t(0)
    _check(fn, getattr(load_library(), fn)(shape, ctypes.byref(n)))
    return n.value


def _scratch(fn: str, shape: bytes, dev, workspace):
    n = _workspace_bytes(fn, shape)
    if workspace is not None:
        _need(workspace, "workspace", dev=dev)
        if workspace.numel() * workspace.element_size() >= n:
            return workspace, workspace.numel() * workspace.element_size()
    n = max(n, 16)
    return torch.empty(n, dtype=torch.uint8, device=dev), n


def moe_grouped_matmul(a, b, offsets, *, form="nn", gather_a=None, gather_b=None, out_dtype=None,
                       accumulate=False, out=None, workspace=None) -> torch.Tensor:
    """Products of rows grouped by expert: group e is rows [offsets[e], offsets[e+1]).

    form "nn": out[r] = a[r] @ b[e], b [E,K,N]; "nt": out[r] = a[r] @ b[e].T, b [E,N,K];
    "tn": out[e] = a[group].T @ b[group], b [R,N], out [E,K,N]. a is [R,K], or any rows with
    gather_a [R] int32 (row r of the problem is a[gather_a[r]]); gather_b likewise for b in
    "tn". Sums are fp32; out_dtype (a's by default) is fp32 or, for bf16 inputs, bf16.
    accumulate adds to the given fp32 out. "nn" and "nt" leave rows in no group, before offsets[0]
    and at and past offsets[E], as they are (in a new `out`: unset)."""
    if form not in MATMUL_FORMS:
        raise ValueError(f"form must be one of {sorted(MATMUL_FORMS)}, got {form!r}")
    rows_a, K = _matrix(a, "a")
    E = _vector(offsets, "offsets") - 1
    if E < 1:
        raise ValueError("offsets must be [E + 1] with E >= 1")
    R = rows_a if gather_a is None else _vector(gather_a, "gather_a")
    rows_b = 0
    if form == "tn":
        rows_b, N = b_shape = _matrix(b, "b")
        Rb = rows_b if gather_b is None else _vector(gather_b, "gather_b")
        if Rb != R:
            raise ValueError(f"a and b give {R} and {Rb} rows")
        shape = (E, K, N)
    else:
        if gather_b is not None:
            raise ValueError("gather_b is for form 'tn'")
        if not isinstance(b, torch.Tensor) or b.dim() != 3:
            raise ValueError("b must be [E, K, N] ('nn') or [E, N, K] ('nt')")
        if form == "nn":
            N = b.shape[2]
            b_shape = (E, K, N)
        else:
            N = b.shape[1]
            b_shape = (E, N, K)
        shape = (R, N)
    dt = _type(a)
    if out_dtype is None:
        out_dtype = a.dtype if out is None or not isinstance(out, torch.Tensor) else out.dtype
    if out_dtype not in _TYPES:
        raise TypeError(f"unsupported out_dtype {out_dtype}: bfloat16 or float32")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dev, dtype = a.device, a.dtype
    pa, pb, po, pga, pgb, pout = _pointers(
        ((a, "a", (rows_a, K), dtype), (b, "b", b_shape, dtype), (offsets, "offsets", (E + 1,), _I32),
         (gather_a, "gather_a", (R,), _I32), (gather_b, "gather_b", (R,), _I32),
         (out, "out", shape, out_dtype)), dev)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
        pout = out.data_ptr()
    s = _MATMUL_SHAPE(R, rows_a, rows_b, K, N, E, MATMUL_FORMS[form], dt, _TYPES[out_dtype],
                      1 if accumulate else 0)
    ws = pws = None
    ws_bytes = _workspace_bytes("moe_grouped_matmul_workspace_size", s)
    if ws_bytes:
        ws, ws_bytes = _scratch("moe_grouped_matmul_workspace_size", s, dev, workspace)
        pws = ws.data_ptr()
    _call("moe_grouped_matmul", dev, s, pa, pb, po, pga, pgb, pout, pws, ws_bytes)
    return out


def moe_swiglu_backward(g, u, dh, w=None, *, src=None, pos=None, offsets=None, inplace=False) -> dict:
    """Gradient of h = silu(g) * u, with the rows' gate weights: dg, du, h (times w) and dw
    [R] fp32 = sum over the row of dh * silu(g) * u. dh is the unweighted dy W_down^T. w is
    [R] by row, or [T,k] by slot with src [R] and pos [T,k] (the routing of the forward's
    workspace). Rows before offsets[0] and at and past offsets[E] are left alone. inplace writes
    dg, du and h over g, u and dh."""
    R, f = rows = _matrix(g, "g")
    T = k = E = 0
    if (src is None) != (pos is None):
        raise ValueError("src and pos come together")
    w_shape = (R,)
    if pos is not None:
        T, k = w_shape = _matrix(pos, "pos", "k")
        if w is None:
            raise ValueError("src and pos need w")
    if offsets is not None:
        E = _vector(offsets, "offsets") - 1
    dt, dev, dtype = _type(g), g.device, g.dtype
    pg, pu, pdh, pw, ps, pp, po = _pointers(
        ((g, "g", rows, dtype), (u, "u", rows, dtype), (dh, "dh", rows, dtype), (w, "w", w_shape, _F32),
         (src, "src", (R,), _I32), (pos, "pos", w_shape, _I32), (offsets, "offsets", (E + 1,), _I32)), dev)
    if inplace:
        if R and len({pg, pu, pdh}) < 3:
            raise ValueError("inplace needs g, u and dh to be three tensors")
        dg, du, h = g, u, dh
    else:
        dg, du, h = torch.empty_like(g), torch.empty_like(u), torch.empty_like(dh)
    dw = torch.empty(R, dtype=_F32, device=dev)
    _call("moe_swiglu_backward", dev, _SWIGLU_SHAPE(R, f, T, k, E, dt), pg, pu, pdh, pw, ps, pp, po,
          dg.data_ptr(), du.data_ptr(), h.data_ptr(), dw.data_ptr())
    return {"dg": dg, "du": du, "h": h, "dw": dw}


def moe_route_backward(x, W_g, probs, idx, w, dw=None, *, b_g=None, f=None, loss_grad=0.0,
                       z_loss_grad=0.0, renormalize=True, rows=None, pos=None, want_dx=True,
                       want_dW=True, workspace=None) -> dict:
    """Gradient of the token-choice router (with or without an expert capacity; no training
    noise): dx [T,d], dW_g [d,E] (x's type), db_g [E] and dlogits [T,E] (fp32).

    probs, idx, w are the forward's outputs; dw is the gradient of w, [T,k] by slot or [R] by
    routed row (with pos). loss_grad and z_loss_grad are the gradients of the load-balancing
    loss (with the forward's f) and the z-loss. rows [R,d] with pos [T,k] adds each token's
    routed-row gradients to dx."""
    T, d = x_shape = _matrix(x, "x", "d_model")
    E = _matrix(W_g, "W_g", "E")[1]
    k = _matrix(idx, "idx", "k")[1]
    slots = (T, k)
    R = _matrix(rows, "rows", "d_model")[0] if rows is not None else 0
    by_row = isinstance(dw, torch.Tensor) and dw.dim() == 1
    if by_row:
        if rows is not None and dw.shape[0] != R:
            raise ValueError(f"dw has {dw.shape[0]} rows, rows {R}")
        R = dw.shape[0]
    if pos is None and (by_row or rows is not None):
        raise ValueError("rows, and dw by row, need pos")
    if loss_grad != 0 and f is None:
        raise ValueError("loss_grad needs f")
    dt, dev, dtype = _type(x), x.device, x.dtype
    px, pW, pb, pp, pi, pw, pdw, pf, prows, ppos = _pointers(
        ((x, "x", x_shape, dtype), (W_g, "W_g", (d, E), dtype), (b_g, "b_g", (E,), _F32),
         (probs, "probs", (T, E), _F32), (idx, "idx", slots, _I32), (w, "w", slots, _F32),
         (dw, "dw", (R,) if by_row else slots, _F32), (f, "f", (E,), _F32),
         (rows, "rows", (R, d), dtype), (pos, "pos", slots, _I32)), dev)
    shape = _LAYER_SHAPE(T, d, 64, E, k, MOE_TOKEN_CHOICE, dt, 1 if renormalize else 0, 1.0)
    ws, ws_bytes = _scratch("moe_route_backward_workspace_size", shape, dev, workspace)
    dx = torch.empty_like(x) if want_dx else None
    dW = torch.empty_like(W_g) if want_dW else None
    db = torch.empty(E, dtype=_F32, device=dev) if want_dW else None
    ds = torch.empty_like(probs)
    up = _ROUTE_UPSTREAM(pdw or 0, 1 if by_row else 0, loss_grad, z_loss_grad, pf or 0, prows or 0,
                         ppos or 0, R)
    _call("moe_route_backward", dev, shape, px, pW, pb, pp, pi, pw, up,
          None if dx is None else dx.data_ptr(), None if dW is None else dW.data_ptr(),
          None if db is None else db.data_ptr(), ds.data_ptr(), ws.data_ptr(), ws_bytes)
    return {"dx": dx, "dW_g": dW, "db_g": db, "dlogits": ds}


def _gate_kind(gate, y, T, d):
    if gate is None:
        return GATE_NONE
    if y is None:
        raise ValueError("gate belongs to the norm after the block: it needs y")
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a tensor")
    if gate.shape == (d,):
        return GATE_CHANNEL
    if gate.shape == (T, 1):
        return GATE_TOKEN
    raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {(d,)} or {(T, 1)}")


def moe_block_norm(x, *, gamma=None, y=None, gamma_post=None, gate=None, residual_scale=1.0,
                   eps=1e-6, want_rstd=True) -> dict:
    """RMS norms after a block (y given) and before the next one (gamma given), in one pass:

    out = residual_scale * x + gate * (y / rms(y) * gamma_post)   (x itself without y)
    u = out / rms(out) * gamma,   rms(v) = sqrt(mean(v^2) + eps) over the row

    x [T,d] bf16 or fp32; y [T,d] fp32, moe_forward's output; gamma, gamma_post [d] fp32; gate
    fp32, [d] per channel or [T,1] per token. Returns out and u (x's type; None where the part
    did not run) and, for the gradient, rstd = 1 / rms(out) and rstd_post = 1 / rms(y), [T]."""
    T, d = rows = _matrix(x, "x", "d")
    if y is None and gamma is None:
        raise ValueError("moe_block_norm needs y (the norm after) or gamma (the norm before)")
    if (y is None) != (gamma_post is None):
        raise ValueError("y and gamma_post come together")
    kind = _gate_kind(gate, y, T, d)
    dev = x.device
    s = _NORM_SHAPE(T, d, _type(x), kind, eps, residual_scale)
    px, py, pgp, pgate, pg = _pointers(
        ((x, "x", rows, x.dtype), (y, "y", rows, _F32), (gamma_post, "gamma_post", (d,), _F32),
         (gate, "gate", (d,) if kind == GATE_CHANNEL else (T, 1), _F32), (gamma, "gamma", (d,), _F32)), dev)
    out = u = rstd = rstd_post = pout = pu = prp = pr = None
    if y is not None:
        out = torch.empty_like(x)
        pout = out.data_ptr()
        if want_rstd:
            rstd_post = torch.empty(T, dtype=_F32, device=dev)
            prp = rstd_post.data_ptr()
    if gamma is not None:
        u = torch.empty_like(x)
        pu = u.data_ptr()
        if want_rstd:
            rstd = torch.empty(T, dtype=_F32, device=dev)
            pr = rstd.data_ptr()
    _call("moe_block_norm", dev, s, px, py, pgp, pgate, pg, pout, pu, prp, pr)
    return {"out": x if y is None else out, "u": u, "rstd": rstd, "rstd_post": rstd_post}


def moe_block_norm_backward(out, *, d_out=None, d_u=None, rstd=None, gamma=None, y=None,
                            rstd_post=None, gamma_post=None, gate=None, residual_scale=1.0,
                            workspace=None) -> dict:
    """Gradient of moe_block_norm. out is the forward's `out` (x where it had no y); d_out and
    d_u are the gradients of out and u (either may be None, u's part needs rstd and gamma).
    Returns dx and dy (out's type) and dgamma, dgamma_post, dgate (fp32, their inputs'
    shapes); None where the part did not run."""
    T, d = rows = _matrix(out, "out", "d")
    if d_out is None and d_u is None:
        raise ValueError("moe_block_norm_backward needs d_out or d_u")
    if d_u is not None and (rstd is None or gamma is None):
        raise ValueError("d_u needs rstd and gamma")
    if (y is None) != (rstd_post is None) or (y is None) != (gamma_post is None):
        raise ValueError("y, rstd_post and gamma_post come together")
    kind = _gate_kind(gate, y, T, d)
    dev, dtype = out.device, out.dtype
    s = _NORM_SHAPE(T, d, _type(out), kind, 1.0, residual_scale)
    pdo, pdu, po, pr, pg, py, prp, pgp, pgate = _pointers(
        ((d_out, "d_out", rows, dtype), (d_u, "d_u", rows, dtype), (out, "out", rows, dtype),
         (rstd, "rstd", (T,), _F32), (gamma, "gamma", (d,), _F32), (y, "y", rows, _F32),
         (rstd_post, "rstd_post", (T,), _F32), (gamma_post, "gamma_post", (d,), _F32),
         (gate, "gate", (d,) if kind == GATE_CHANNEL else (T, 1), _F32)), dev)
    ws, ws_bytes = _scratch("moe_block_norm_backward_workspace_size", s, dev, workspace)
    dx = torch.empty_like(out)
    dy = dgamma = dgamma_post = dgate = pdy = pdg = pdgp = pdgate = None
    if y is not None:
        dy, dgamma_post = torch.empty_like(out), torch.empty_like(gamma_post)
        pdy, pdgp = dy.data_ptr(), dgamma_post.data_ptr()
        if gate is not None:
            dgate = torch.empty_like(gate)
            pdgate = dgate.data_ptr()
    if d_u is not None:
        dgamma = torch.empty_like(gamma)
        pdg = dgamma.data_ptr()
    _call("moe_block_norm_backward", dev, s, pdo, pdu, po, pr, pg, py, prp, pgp, pgate, dx.data_ptr(),
          pdy, pdg, pdgp, pdgate, ws.data_ptr(), ws_bytes)
    return {"dx": dx, "dy": dy, "dgamma": dgamma, "dgamma_post": dgamma_post, "dgate": dgate}
