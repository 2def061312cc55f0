"""Refusals of the training operators, on the CPU: the binding's shape and type checks come
before its device checks, and the C entry points check every argument before any HIP call."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_sum_amd as M
from sparse_mixture_experts_sum_amd import training as TR

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(M.LIB_PATH):
        from sparse_mixture_experts_sum_amd import build
        build.build()
    return M.load_library()


def z(*s, dtype=BF16):
    return torch.zeros(*s, dtype=dtype)


# ---- the binding -----------------------------------------------------------------------
def matmul(a=None, b=None, offsets=None, **kw):
    return M.moe_grouped_matmul(z(10, 64) if a is None else a, z(4, 64, 128) if b is None else b,
                                z(5, dtype=I32) if offsets is None else offsets, **kw)


MATMUL_VALUE = {
    "form": dict(form="tt"),
    "a_3d": dict(a=z(1, 10, 64)),
    "b_2d": dict(b=z(64, 128)),
    "b_K": dict(b=z(4, 56, 128)),
    "b_E": dict(b=z(3, 64, 128)),
    "nt_b": dict(b=z(4, 64, 128), form="nt"),
    "offsets_2d": dict(offsets=z(1, 5, dtype=I32)),
    "no_groups": dict(offsets=z(1, dtype=I32)),
    "out": dict(out=z(9, 128)),
    "gather_b_nn": dict(gather_b=z(10, dtype=I32)),
    "tn_rows": dict(b=z(9, 128), form="tn"),
    "tn_gather": dict(b=z(10, 128), form="tn", gather_a=z(9, dtype=I32)),
    "accumulate": dict(accumulate=True),
}


@pytest.mark.parametrize("name", sorted(MATMUL_VALUE))
def test_matmul_refuses_shapes(name):
    with pytest.raises(ValueError):
        matmul(**MATMUL_VALUE[name])


def test_matmul_refuses_types_and_host_tensors():
    for kw in (dict(a=z(10, 64, dtype=torch.float16)), dict(out_dtype=torch.float16), dict(a=[1]),
               dict(offsets=[0, 1]), {}):
        with pytest.raises(TypeError):
            matmul(**kw)


NORM_VALUE = {
    "neither": dict(),
    "y_shape": dict(y=z(9, 64, dtype=F32), gamma_post=z(64, dtype=F32)),
    "gamma": dict(gamma=z(63, dtype=F32)),
    "no_gamma_post": dict(y=z(10, 64, dtype=F32)),
    "no_y": dict(gamma=z(64, dtype=F32), gamma_post=z(64, dtype=F32)),
    "gate_without_y": dict(gamma=z(64, dtype=F32), gate=z(64, dtype=F32)),
    "gate_shape": dict(y=z(10, 64, dtype=F32), gamma_post=z(64, dtype=F32), gate=z(10, dtype=F32)),
}


@pytest.mark.parametrize("name", sorted(NORM_VALUE))
def test_norm_refuses_shapes(name):
    with pytest.raises(ValueError):
        M.moe_block_norm(z(10, 64), **NORM_VALUE[name])


def test_norm_backward_refuses():
    out, v, t = z(10, 64), z(64, dtype=F32), z(10, dtype=F32)
    for kw in ({}, dict(d_u=out), dict(d_u=out, rstd=t), dict(d_out=z(9, 64)),
               dict(d_out=out, y=z(10, 64, dtype=F32)), dict(d_out=out, rstd_post=t),
               dict(d_out=out, gate=v), dict(d_u=out, rstd=z(9, dtype=F32), gamma=v)):
        with pytest.raises(ValueError):
            M.moe_block_norm_backward(out, **kw)
    with pytest.raises(TypeError):
        M.moe_block_norm_backward(out, d_out=out)  # a host tensor


def test_swiglu_and_route_refuse():
    g = z(6, 64)
    for kw in (dict(u=z(6, 56)), dict(dh=z(5, 64)), dict(w=z(5, dtype=F32)), dict(src=z(6, dtype=I32)),
               dict(src=z(6, dtype=I32), pos=z(3, 2, dtype=I32)),
               dict(src=z(5, dtype=I32), pos=z(3, 2, dtype=I32), w=z(3, 2, dtype=F32))):
        args = dict(g=g, u=g, dh=g)
        args.update(kw)
        with pytest.raises(ValueError):
            first = [args.pop(n, None) for n in ("g", "u", "dh", "w")]
            M.moe_swiglu_backward(*first, **args)
    with pytest.raises(TypeError):
        M.moe_swiglu_backward(g, g, g)
    x, W, p, i, w = z(5, 64), z(64, 8), z(5, 8, dtype=F32), z(5, 2, dtype=I32), z(5, 2, dtype=F32)
    for kw in (dict(W=z(56, 8)), dict(p=z(5, 7, dtype=F32)), dict(w=z(5, 1, dtype=F32)), dict(dw=z(4, 2, dtype=F32)),
               dict(rows=z(10, 64)), dict(dw=z(10, dtype=F32)), dict(loss_grad=1.0),
               dict(rows=z(10, 64), dw=z(9, dtype=F32), pos=i), dict(b_g=z(7, dtype=F32)),
               dict(rows=z(10, 56), pos=i)):
        args = dict(x=x, W=W, p=p, i=i, w=w, dw=None)
        args.update(kw)
        with pytest.raises(ValueError):
            first = [args.pop(n) for n in ("x", "W", "p", "i", "w", "dw")]
            M.moe_route_backward(*first, **args)
    with pytest.raises(TypeError):
        M.moe_route_backward(x, W, p, i, w)


def test_layer_refuses():
    with pytest.raises(ValueError):
        M.SparseMoE(None, None, None, None, gate=z(64, dtype=F32))
    with pytest.raises(ValueError):
        M.SparseMoE(None, None, None, None).backward(z(1, 64))


# ---- the C entry points ----------------------------------------------------------------
P = 4096  # an aligned address that nothing reads: every call below is refused first
NULL_ARG, BAD_SHAPE, UNSUPPORTED, SMALL, MISALIGNED = 1, 2, 3, 4, 5


def call_matmul(lib, shape=(), a=P, b=P, off=P, ga=None, gb=None, out=P, ws=None, ws_bytes=0, **kw):
    s = dict(R=10, rows_a=10, rows_b=0, K=64, N=128, E=4, form=0, dtype=1, out_dtype=1, accumulate=0)
    s.update(kw)
    return lib.moe_grouped_matmul(TR._MATMUL_SHAPE(*s.values()), a, b, off, ga, gb, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), NULL_ARG), (dict(off=None), NULL_ARG), (dict(out=None), NULL_ARG),
    (dict(R=-1), BAD_SHAPE), (dict(R=1 << 31, rows_a=1 << 31), BAD_SHAPE),
    (dict(R=(1 << 31) - 65535, rows_a=(1 << 31) - 65535), BAD_SHAPE), (dict(rows_a=9), BAD_SHAPE),
    (dict(E=0), BAD_SHAPE), (dict(E=65), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(N=4), UNSUPPORTED),
    (dict(K=0), BAD_SHAPE), (dict(N=(1 << 20) + 8), BAD_SHAPE), (dict(form=3), BAD_SHAPE),
    (dict(dtype=2), BAD_SHAPE), (dict(accumulate=2), BAD_SHAPE), (dict(accumulate=1), UNSUPPORTED),
    (dict(dtype=0), UNSUPPORTED), (dict(gb=P), UNSUPPORTED), (dict(a=P + 8), MISALIGNED),
    (dict(out=P + 4), MISALIGNED), (dict(form=2, rows_b=9), BAD_SHAPE),
    (dict(ga=P, rows_a=0), BAD_SHAPE), (dict(form=2, gb=P, rows_b=0), BAD_SHAPE),
    # a long sum of few tiles needs its workspace
    (dict(form=2, R=1 << 16, rows_a=1 << 16, rows_b=1 << 16, E=1), NULL_ARG),
    (dict(form=2, R=1 << 16, rows_a=1 << 16, rows_b=1 << 16, E=1, ws=P, ws_bytes=64), SMALL),
])
def test_matmul_statuses(lib, kw, status):
    assert call_matmul(lib, **kw) == status


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(7)
    f = lib.moe_grouped_matmul_workspace_size
    assert f(TR._MATMUL_SHAPE(1 << 16, 1 << 16, 0, 1024, 4096, 8, 0, 1, 1, 0), ctypes.byref(n)) == 0 and n.value == 0
    assert f(TR._MATMUL_SHAPE(1 << 16, 1 << 16, 1 << 16, 64, 64, 1, 2, 1, 1, 0), ctypes.byref(n)) == 0
    assert n.value > 0 and n.value % (64 * 64 * 4) == 0
    assert f(TR._MATMUL_SHAPE(0, 0, 0, 64, 64, 1, 2, 1, 1, 0), ctypes.byref(n)) == 0 and n.value == 0
    assert f(None, ctypes.byref(n)) == NULL_ARG and f(TR._MATMUL_SHAPE(*[0] * 10), None) == NULL_ARG
    s = M.make_shape(1000, 256, 64, 8, 2)
    assert lib.moe_route_backward_workspace_size(bytes(s), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.moe_block_norm_backward_workspace_size(TR._NORM_SHAPE(100, 64, 1, 0, 1.0, 1.0), ctypes.byref(n)) == 0
    # partial sums of three kinds per workgroup, at least one workgroup
    assert n.value >= 3 * 64 * 4 and n.value % (3 * 64 * 4) == 0


def test_swiglu_statuses(lib):
    def call(g=P, w=None, src=None, pos=None, off=None, dg=P, **kw):
        s = dict(R=10, f=64, T=0, k=0, E=0, dtype=1)
        s.update(kw)
        return lib.moe_swiglu_backward(TR._SWIGLU_SHAPE(*s.values()), g, P, P, w, src, pos, off, dg, P, P, P, None)

    assert call(g=None) == NULL_ARG and call(R=-1) == BAD_SHAPE and call(f=60) == UNSUPPORTED
    assert call(f=0) == BAD_SHAPE and call(dtype=5) == BAD_SHAPE and call(dg=P + 2) == MISALIGNED
    assert call(off=P) == BAD_SHAPE and call(off=P, E=65) == UNSUPPORTED
    assert call(pos=P, T=5, k=2) == NULL_ARG and call(pos=P, w=P, src=P, T=5, k=9) == UNSUPPORTED
    assert call(pos=P, w=P, src=P, T=0, k=2) == BAD_SHAPE
    assert lib.moe_swiglu_backward(None, *[P] * 11, None) == NULL_ARG


def test_route_statuses(lib):
    need = ctypes.c_size_t(0)
    lib.moe_route_backward_workspace_size(bytes(M.make_shape(10, 64, 64, 8, 2)), ctypes.byref(need))

    def call(x=P, idx=P, ds=P, ws=P, ws_bytes=None, up=(0, 0, 0.0, 0.0, 0, 0, 0, 0), dx=P, **kw):
        s = dict(T=10, d_model=64, d_ff=64, E=8, k=2)
        s.update(kw)
        return lib.moe_route_backward(
            bytes(M.make_shape(**s)), x, P, None, P, idx, P, None if up is None else TR._ROUTE_UPSTREAM(*up), dx, P,
            P, ds, ws, need.value if ws_bytes is None else ws_bytes, None)

    assert call(x=None) == NULL_ARG and call(idx=None) == NULL_ARG and call(ds=None) == NULL_ARG
    assert call(ws=None) == NULL_ARG and call(up=None) == NULL_ARG and call(dx=P + 8) == MISALIGNED
    assert call(ws_bytes=need.value - 1) == SMALL and call(mode="ec") == UNSUPPORTED
    assert call(d_model=60) == UNSUPPORTED and call(E=65) == UNSUPPORTED and call(k=9, E=16) == UNSUPPORTED
    assert call(k=9) == BAD_SHAPE and call(T=-1) == BAD_SHAPE
    assert call(up=(P, 0, 1.0, 0.0, 0, 0, 0, 0)) == NULL_ARG             # loss_grad without f
    assert call(up=(P, 1, 0.0, 0.0, 0, 0, 0, 9)) == NULL_ARG             # by row without pos
    assert call(up=(0, 0, 0.0, 0.0, 0, P, 0, 9)) == NULL_ARG             # rows without pos
    assert call(up=(P, 2, 0.0, 0.0, 0, 0, 0, 0)) == BAD_SHAPE
    assert call(up=(P, 0, float("nan"), 0.0, 0, 0, 0, 0)) == BAD_SHAPE
    assert call(up=(P, 0, 0.0, float("inf"), 0, 0, 0, 0)) == BAD_SHAPE
    assert call(up=(P, 0, 0.0, 0.0, 0, 0, 0, -1)) == BAD_SHAPE
    assert call(up=(0, 0, 0.0, 0.0, 0, P + 8, P, 9)) == MISALIGNED


def test_norm_statuses(lib):
    def fwd(x=P, y=None, gp=None, gate=None, g=P, out=None, u=P, rp=None, r=None, **kw):
        s = dict(T=10, d=64, dtype=1, gate_kind=0, eps=1e-6, scale=1.0)
        s.update(kw)
        return lib.moe_block_norm(TR._NORM_SHAPE(*s.values()), x, y, gp, gate, g, out, u, rp, r, None)

    post = dict(y=P, gp=P, out=P)
    assert fwd(x=None) == NULL_ARG and fwd(g=None, u=None) == NULL_ARG and fwd(u=None) == NULL_ARG
    assert fwd(g=None) == BAD_SHAPE and fwd(out=P) == BAD_SHAPE and fwd(gp=P) == BAD_SHAPE
    assert fwd(**dict(post, gp=None)) == NULL_ARG and fwd(**dict(post, out=None)) == NULL_ARG
    assert fwd(gate_kind=1, **post) == BAD_SHAPE and fwd(gate=P, **post) == BAD_SHAPE
    assert fwd(gate_kind=1) == BAD_SHAPE and fwd(gate_kind=3, **post) == BAD_SHAPE
    assert fwd(d=60) == UNSUPPORTED and fwd(d=16392) == UNSUPPORTED and fwd(d=0) == BAD_SHAPE
    assert fwd(T=-1) == BAD_SHAPE and fwd(eps=0.0) == BAD_SHAPE and fwd(eps=float("nan")) == BAD_SHAPE
    assert fwd(scale=float("inf")) == BAD_SHAPE and fwd(dtype=7) == BAD_SHAPE
    assert fwd(u=P + 8) == MISALIGNED and fwd(gate_kind=1, gate=P + 4, **post) == MISALIGNED

    def bwd(d_out=P, d_u=None, out=P, r=None, g=None, y=None, rp=None, gp=None, gate=None, dx=P, dy=None, dg=None,
            dgp=None, dgate=None, ws=P, ws_bytes=1 << 20, **kw):
        s = dict(T=10, d=64, dtype=1, gate_kind=0, eps=1e-6, scale=1.0)
        s.update(kw)
        return lib.moe_block_norm_backward(TR._NORM_SHAPE(*s.values()), d_out, d_u, out, r, g, y, rp, gp, gate, dx,
                                           dy, dg, dgp, dgate, ws, ws_bytes, None)

    assert bwd(d_out=None) == NULL_ARG and bwd(d_u=P) == NULL_ARG and bwd(d_u=P, r=P) == NULL_ARG
    assert bwd(y=P) == NULL_ARG and bwd(y=P, rp=P) == NULL_ARG and bwd(dy=P) == BAD_SHAPE
    assert bwd(dgate=P) == BAD_SHAPE and bwd(y=P, rp=P, gp=P, dgate=P) == BAD_SHAPE
    assert bwd(y=P, rp=P, gp=P, gate_kind=2) == BAD_SHAPE and bwd(ws=None) == NULL_ARG
    assert bwd(ws_bytes=100) == SMALL and bwd(dx=P + 8) == MISALIGNED and bwd(dg=P) == BAD_SHAPE
