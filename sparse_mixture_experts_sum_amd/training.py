"""The layer's training operators: products grouped by expert, the experts' and the router's
gradients, and the norms around the layer with their gradient.

Bindings of the entry points in the "Training" section of ``include/moe.h``; like the
forward's, they check tensor metadata, allocate outputs and workspaces with torch and pass
pointers and the current HIP stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

MATMUL_FORMS = {"nn": 0, "nt": 1, "tn": 2}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2


class MoeMatmulShape(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("rows_a", ctypes.c_int64), ("rows_b", ctypes.c_int64),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("E", ctypes.c_int32),
                ("form", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class MoeSwigluShape(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("f", ctypes.c_int64), ("T", ctypes.c_int64),
                ("k", ctypes.c_int32), ("E", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MoeRouteUpstream(ctypes.Structure):
    _fields_ = [("dw", ctypes.c_void_p), ("dw_by_row", ctypes.c_int32),
                ("loss_grad", ctypes.c_float), ("z_loss_grad", ctypes.c_float),
                ("f", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("R", ctypes.c_int64)]


class MoeNormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float)]


def declare(lib, shape_p):
    """Argument types of the training entry points (called once by load_library)."""
    P, SZ, B = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    lib.moe_grouped_matmul.argtypes = [B(MoeMatmulShape)] + [P] * 7
    lib.moe_swiglu_backward.argtypes = [B(MoeSwigluShape)] + [P] * 12
    lib.moe_route_backward_workspace_size.argtypes = [shape_p, B(SZ)]
    lib.moe_route_backward.argtypes = [shape_p] + [P] * 6 + [B(MoeRouteUpstream)] + [P] * 5 + [SZ, P]
    lib.moe_block_norm.argtypes = [B(MoeNormShape)] + [P] * 10
    lib.moe_block_norm_backward_workspace_size.argtypes = [B(MoeNormShape), B(SZ)]
    lib.moe_block_norm_backward.argtypes = [B(MoeNormShape)] + [P] * 15 + [SZ, P]
    for name in ("moe_grouped_matmul", "moe_swiglu_backward", "moe_route_backward_workspace_size",
                 "moe_route_backward", "moe_block_norm", "moe_block_norm_backward_workspace_size",
                 "moe_block_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int32


from . import (MOE_BF16, MOE_FP32, _check, _dtype_name, _need, _shape_is,  # noqa: E402
               load_library, make_shape)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dt(t) -> int:
    return MOE_BF16 if _dtype_name(t) == "bf16" else MOE_FP32


def _matrix(t, name, cols=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [rows, {cols or 'width'}], got shape {tuple(t.shape)}")
    return t.shape


def _vector(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 1:
        raise ValueError(f"{name} must have one dimension, got shape {tuple(t.shape)}")
    return t.shape[0]


def _call(fn: str, dev: torch.device, *args):
    """One library call on dev's current stream, with dev the current device."""
    lib = load_library()
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        st = getattr(lib, fn)(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = getattr(lib, fn)(*args, stream)
    if st:
        _check(fn, st)


def _scratch(fn: str, shape, dev, workspace):
    n = ctypes.c_size_t(0)
    _check(fn, getattr(load_library(), fn)(ctypes.byref(shape), ctypes.byref(n)))
    if workspace is not None:
        _need(workspace, "workspace", dev=dev)
        if workspace.numel() * workspace.element_size() >= n.value:
            return workspace
    return torch.empty(max(n.value, 16), dtype=torch.uint8, device=dev)


def moe_grouped_matmul(a, b, offsets, *, form="nn", gather_a=None, gather_b=None, out_dtype=None,
                       accumulate=False, out=None) -> torch.Tensor:
    """Products of rows grouped by expert: group e is rows [offsets[e], offsets[e+1]).

    form "nn": out[r] = a[r] @ b[e], b [E,K,N]; "nt": out[r] = a[r] @ b[e].T, b [E,N,K];
    "tn": out[e] = a[group].T @ b[group], b [R,N], out [E,K,N]. a is [R,K], or any rows with
    gather_a [R] int32 (row r of the problem is a[gather_a[r]]); gather_b likewise for b in
    "tn". Sums are fp32; out_dtype (a's by default) is fp32 or, for bf16 inputs, bf16.
    accumulate adds to the given fp32 out. "nn" and "nt" leave rows at and past offsets[E] as
    they are (in a new `out`: unset)."""
    if form not in MATMUL_FORMS:
        raise ValueError(f"form must be one of {sorted(MATMUL_FORMS)}, got {form!r}")
    rows_a, K = _matrix(a, "a")
    E = _vector(offsets, "offsets") - 1
    if E < 1:
        raise ValueError("offsets must be [E + 1] with E >= 1")
    R = rows_a if gather_a is None else _vector(gather_a, "gather_a")
    rows_b = 0
    if form == "tn":
        rows_b, N = _matrix(b, "b")
        Rb = rows_b if gather_b is None else _vector(gather_b, "gather_b")
        if Rb != R:
            raise ValueError(f"a and b give {R} and {Rb} rows")
        shape = (E, K, N)
    else:
        if gather_b is not None:
            raise ValueError("gather_b is for form 'tn'")
        if not isinstance(b, torch.Tensor) or b.dim() != 3:
            raise ValueError("b must be [E, K, N] ('nn') or [E, N, K] ('nt')")
        N = b.shape[2] if form == "nn" else b.shape[1]
        _shape_is(b, "b", (E, K, N) if form == "nn" else (E, N, K))
        shape = (R, N)
    _shape_is(out, "out", shape)
    dt = _dt(a)
    if out_dtype is None:
        out_dtype = a.dtype if out is None else out.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported out_dtype {out_dtype}: bfloat16 or float32")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dev = a.device
    _need(a, "a", dev=dev)
    _need(b, "b", a.dtype, dev)
    _need(offsets, "offsets", torch.int32, dev)
    _need(gather_a, "gather_a", torch.int32, dev)
    _need(gather_b, "gather_b", torch.int32, dev)
    _need(out, "out", out_dtype, dev)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    s = MoeMatmulShape(R, rows_a, rows_b, K, N, E, MATMUL_FORMS[form], dt,
                       MOE_BF16 if out_dtype == torch.bfloat16 else MOE_FP32, 1 if accumulate else 0)
    _call("moe_grouped_matmul", dev, ctypes.byref(s), _p(a), _p(b), _p(offsets), _p(gather_a),
          _p(gather_b), _p(out))
    return out


def moe_swiglu_backward(g, u, dh, w=None, *, src=None, pos=None, offsets=None, inplace=False) -> dict:
    """Gradient of h = silu(g) * u, with the rows' gate weights: dg, du, h (times w) and dw
    [R] fp32 = sum over the row of dh * silu(g) * u. dh is the unweighted dy W_down^T. w is
    [R] by row, or [T,k] by slot with src [R] and pos [T,k] (the routing of the forward's
    workspace). Rows at and past offsets[E] are left alone. inplace writes dg, du and h over
    g, u and dh."""
    R, f = _matrix(g, "g")
    _shape_is(u, "u", (R, f))
    _shape_is(dh, "dh", (R, f))
    dev = g.device
    T = k = 0
    if (src is None) != (pos is None):
        raise ValueError("src and pos come together")
    if pos is not None:
        T, k = _matrix(pos, "pos")
        if w is None:
            raise ValueError("src and pos need w")
        _shape_is(w, "w", (T, k))
        _shape_is(src, "src", (R,))
    else:
        _shape_is(w, "w", (R,))
    E = 0
    if offsets is not None:
        E = _vector(offsets, "offsets") - 1
    dt = _dt(g)
    _need(g, "g", dev=dev)
    _need(u, "u", g.dtype, dev)
    _need(dh, "dh", g.dtype, dev)
    _need(w, "w", torch.float32, dev)
    _need(src, "src", torch.int32, dev)
    _need(pos, "pos", torch.int32, dev)
    _need(offsets, "offsets", torch.int32, dev)
    if inplace:
        dg, du, h = g, u, dh
    else:
        dg, du, h = torch.empty_like(g), torch.empty_like(u), torch.empty_like(dh)
    dw = torch.empty(R, dtype=torch.float32, device=dev)
    s = MoeSwigluShape(R, f, T, k, E, dt)
    _call("moe_swiglu_backward", dev, ctypes.byref(s), _p(g), _p(u), _p(dh), _p(w), _p(src),
          _p(pos), _p(offsets), _p(dg), _p(du), _p(h), _p(dw))
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
    T, d = _matrix(x, "x")
    E = _matrix(W_g, "W_g")[1]
    _shape_is(W_g, "W_g", (d, E))
    _shape_is(b_g, "b_g", (E,))
    _shape_is(probs, "probs", (T, E))
    k = _matrix(idx, "idx")[1]
    _shape_is(idx, "idx", (T, k))
    _shape_is(w, "w", (T, k))
    _shape_is(f, "f", (E,))
    _shape_is(pos, "pos", (T, k))
    R = 0
    if rows is not None:
        R = _matrix(rows, "rows", d)[0]
    by_row = isinstance(dw, torch.Tensor) and dw.dim() == 1
    if by_row:
        if rows is not None and dw.shape[0] != R:
            raise ValueError(f"dw has {dw.shape[0]} rows, rows {R}")
        R = dw.shape[0]
    else:
        _shape_is(dw, "dw", (T, k))
    if pos is None and (by_row or rows is not None):
        raise ValueError("rows, and dw by row, need pos")
    if loss_grad != 0 and f is None:
        raise ValueError("loss_grad needs f")
    dev = x.device
    _dtype_name(x)
    _need(x, "x", dev=dev)
    _need(W_g, "W_g", x.dtype, dev)
    for t, n in ((b_g, "b_g"), (probs, "probs"), (w, "w"), (dw, "dw"), (f, "f")):
        _need(t, n, torch.float32, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(pos, "pos", torch.int32, dev)
    _need(rows, "rows", x.dtype, dev)
    shape = make_shape(T, d, 64, E, k, "tc", _dtype_name(x), renormalize)
    ws = _scratch("moe_route_backward_workspace_size", shape, dev, workspace)
    dx = torch.empty_like(x) if want_dx else None
    dW = torch.empty_like(W_g) if want_dW else None
    db = torch.empty(E, dtype=torch.float32, device=dev) if want_dW else None
    ds = torch.empty(T, E, dtype=torch.float32, device=dev)
    up = MoeRouteUpstream(_p(dw), 1 if by_row else 0, float(loss_grad), float(z_loss_grad), _p(f),
                          _p(rows), _p(pos), R)
    _call("moe_route_backward", dev, ctypes.byref(shape), _p(x), _p(W_g), _p(b_g), _p(probs),
          _p(idx), _p(w), ctypes.byref(up), _p(dx), _p(dW), _p(db), _p(ds), _p(ws),
          ws.numel() * ws.element_size())
    return {"dx": dx, "dW_g": dW, "db_g": db, "dlogits": ds}


def _norm_shape(T, d, dt, y, gate, eps, scale):
    kind = GATE_NONE
    if gate is not None:
        if y is None:
            raise ValueError("gate belongs to the norm after the block: it needs y")
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a tensor")
        if tuple(gate.shape) == (d,):
            kind = GATE_CHANNEL
        elif tuple(gate.shape) == (T, 1):
            kind = GATE_TOKEN
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {(d,)} or {(T, 1)}")
    return MoeNormShape(T, d, dt, kind, float(eps), float(scale))


def moe_block_norm(x, *, gamma=None, y=None, gamma_post=None, gate=None, residual_scale=1.0,
                   eps=1e-6, want_rstd=True) -> dict:
    """RMS norms after a block (y given) and before the next one (gamma given), in one pass:

    out = residual_scale * x + gate * (y / rms(y) * gamma_post)   (x itself without y)
    u = out / rms(out) * gamma,   rms(v) = sqrt(mean(v^2) + eps) over the row

    x [T,d] bf16 or fp32; y [T,d] fp32, moe_forward's output; gamma, gamma_post [d] fp32; gate
    fp32, [d] per channel or [T,1] per token. Returns out and u (x's type; None where the part
    did not run) and, for the gradient, rstd = 1 / rms(out) and rstd_post = 1 / rms(y), [T]."""
    T, d = _matrix(x, "x")
    if y is None and gamma is None:
        raise ValueError("moe_block_norm needs y (the norm after) or gamma (the norm before)")
    _shape_is(y, "y", (T, d))
    _shape_is(gamma, "gamma", (d,))
    _shape_is(gamma_post, "gamma_post", (d,))
    if (y is None) != (gamma_post is None):
        raise ValueError("y and gamma_post come together")
    dt = _dt(x)
    s = _norm_shape(T, d, dt, y, gate, eps, residual_scale)
    dev = x.device
    _need(x, "x", dev=dev)
    for t, n in ((y, "y"), (gamma, "gamma"), (gamma_post, "gamma_post"), (gate, "gate")):
        _need(t, n, torch.float32, dev)
    out = u = rstd = rstd_post = None
    if y is not None:
        out = torch.empty_like(x)
        if want_rstd:
            rstd_post = torch.empty(T, dtype=torch.float32, device=dev)
    if gamma is not None:
        u = torch.empty_like(x)
        if want_rstd:
            rstd = torch.empty(T, dtype=torch.float32, device=dev)
    _call("moe_block_norm", dev, ctypes.byref(s), _p(x), _p(y), _p(gamma_post), _p(gate),
          _p(gamma), _p(out), _p(u), _p(rstd_post), _p(rstd))
    return {"out": x if y is None else out, "u": u, "rstd": rstd, "rstd_post": rstd_post}


def moe_block_norm_backward(out, *, d_out=None, d_u=None, rstd=None, gamma=None, y=None,
                            rstd_post=None, gamma_post=None, gate=None, residual_scale=1.0,
                            workspace=None) -> dict:
    """Gradient of moe_block_norm. out is the forward's `out` (x where it had no y); d_out and
    d_u are the gradients of out and u (either may be None, u's part needs rstd and gamma).
    Returns dx and dy (out's type) and dgamma, dgamma_post, dgate (fp32, their inputs'
    shapes); None where the part did not run."""
    T, d = _matrix(out, "out")
    if d_out is None and d_u is None:
        raise ValueError("moe_block_norm_backward needs d_out or d_u")
    for t, n in ((d_out, "d_out"), (d_u, "d_u"), (y, "y")):
        _shape_is(t, n, (T, d))
    _shape_is(gamma, "gamma", (d,))
    _shape_is(gamma_post, "gamma_post", (d,))
    _shape_is(rstd, "rstd", (T,))
    _shape_is(rstd_post, "rstd_post", (T,))
    if d_u is not None and (rstd is None or gamma is None):
        raise ValueError("d_u needs rstd and gamma")
    if (y is None) != (rstd_post is None) or (y is None) != (gamma_post is None):
        raise ValueError("y, rstd_post and gamma_post come together")
    s = _norm_shape(T, d, _dt(out), y, gate, 1.0, residual_scale)
    dev = out.device
    _need(out, "out", dev=dev)
    _need(d_out, "d_out", out.dtype, dev)
    _need(d_u, "d_u", out.dtype, dev)
    for t, n in ((rstd, "rstd"), (gamma, "gamma"), (y, "y"), (rstd_post, "rstd_post"),
                 (gamma_post, "gamma_post"), (gate, "gate")):
        _need(t, n, torch.float32, dev)
    ws = _scratch("moe_block_norm_backward_workspace_size", s, dev, workspace)
    dx = torch.empty_like(out)
    dy = dgamma = dgamma_post = dgate = None
    if y is not None:
        dy = torch.empty_like(out)
        dgamma_post = torch.empty_like(gamma_post)
        dgate = None if gate is None else torch.empty_like(gate)
    if d_u is not None:
        dgamma = torch.empty_like(gamma)
    _call("moe_block_norm_backward", dev, ctypes.byref(s), _p(d_out), _p(d_u), _p(out), _p(rstd),
          _p(gamma), _p(y), _p(rstd_post), _p(gamma_post), _p(gate), _p(dx), _p(dy), _p(dgamma),
          _p(dgamma_post), _p(dgate), _p(ws), ws.numel() * ws.element_size())
    return {"dx": dx, "dy": dy, "dgamma": dgamma, "dgamma_post": dgamma_post, "dgate": dgate}
