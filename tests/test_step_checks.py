"""Refusals of the layer norms and the update step, on the CPU: the binding's shape and type
checks come before its device checks, and the C entry points check every argument before any
HIP call."""
import ctypes
import os

import pytest
import torch

import sparse_mixture_experts_sum_amd as M
from sparse_mixture_experts_sum_amd import step as ST

BF16, F32 = torch.bfloat16, torch.float32
OK, NULL_ARG, BAD_SHAPE, UNSUPPORTED, TOO_SMALL, MISALIGNED = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from sparse_mixture_experts_sum_amd import build
        build.build()
    return M.load_library()


def z(*s, dtype=BF16):
    return torch.zeros(*s, dtype=dtype)


def v(n=64):
    return z(n, dtype=F32)


# ---- the binding -----------------------------------------------------------------------
NORM_VALUE = {
    "x_3d": dict(x=z(1, 10, 64)),
    "no_gamma": dict(gamma=None),
    "gamma": dict(gamma=v(63)),
    "beta": dict(beta=v(65)),
    "y_shape": dict(y=z(9, 64, dtype=F32)),
    "scale_without_y": dict(residual_scale=0.5),
    "strided": dict(x=z(10, 128)[:, ::2]),
}


@pytest.mark.parametrize("name", sorted(NORM_VALUE))
def test_layer_norm_refuses(name):
    kw = dict(x=z(10, 64), gamma=v())
    kw.update(NORM_VALUE[name])
    with pytest.raises((ValueError, TypeError)):  # (a stride is found with the device)
        M.moe_layer_norm(kw.pop("x"), kw.pop("gamma"), kw.pop("beta", None), **kw)


def test_layer_norm_refuses_types():
    for x, kw in ((z(10, 64, dtype=torch.float16), {}), ([1], {}), (z(10, 64), dict(y=z(10, 64))), (z(10, 64), {})):
        with pytest.raises(TypeError):
            M.moe_layer_norm(x, v(), **kw)


@pytest.mark.parametrize("kw", [dict(out=z(64)), dict(d_u=z(9, 64)), dict(mean=v(9)), dict(rstd=None), dict(gamma=v(8)),
                                dict(d_out=z(10, 32)), dict(d_u=None)])
def test_layer_norm_backward_refuses(kw):
    a = dict(out=z(10, 64), d_u=z(10, 64), mean=v(10), rstd=v(10), gamma=v())
    a.update(kw)
    with pytest.raises(ValueError):
        M.moe_layer_norm_backward(**a)


ORTH_VALUE = {
    "vector": dict(g=z(64)),
    "4d": dict(g=z(1, 1, 8, 8)),
    "empty": dict(g=z(0, 8, 8)),
    "no_rows": dict(g=z(0, 8)),
    "steps_0": dict(steps=0),
    "steps_float": dict(steps=2.5),
    "two_coefficients": dict(coefficients=(1, 2)),
    "nan": dict(coefficients=(1.0, float("nan"), 0.0)),
    "eps": dict(eps=-1.0),
    "eps_inf": dict(eps=float("inf")),
    "out": dict(out=z(8, 16)),
}


@pytest.mark.parametrize("name", sorted(ORTH_VALUE))
def test_orthogonalize_refuses(name):
    kw = dict(g=z(8, 8))
    kw.update(ORTH_VALUE[name])
    with pytest.raises(ValueError):
        M.moe_orthogonalize(kw.pop("g"), **kw)


def test_orthogonalize_refuses_types():
    for g, kw in ((z(8, 8, dtype=torch.float16), {}), (None, {}), (z(8, 8), {})):
        with pytest.raises(TypeError):
            M.moe_orthogonalize(g, **kw)


MUON_VALUE = {
    "g": dict(g=z(8, 9)),
    "no_g": dict(g=None),
    "no_m": dict(m=None),
    "m": dict(m=z(9, 8, dtype=F32)),
    "lr": dict(lr=float("inf")),
    "momentum": dict(momentum=float("nan")),
    "decay": dict(weight_decay=float("nan")),
    "scale": dict(scale=float("inf")),
}


@pytest.mark.parametrize("name", sorted(MUON_VALUE))
def test_muon_refuses(name):
    kw = dict(g=z(8, 8), m=z(8, 8, dtype=F32), lr=0.1)
    kw.update(MUON_VALUE[name])
    with pytest.raises(ValueError):
        M.moe_muon_update(z(8, 8), kw.pop("g"), kw.pop("m"), **kw)


def test_muon_refuses_types():
    w = z(8, 8)
    for g, m in ((z(8, 8, dtype=F32), z(8, 8, dtype=F32)), (w, z(8, 8)), (z(8, 8), z(8, 8, dtype=F32))):
        with pytest.raises(TypeError):
            M.moe_muon_update(w, g, m, lr=0.1)


def test_layer_with_norms_refuses():
    W = (z(64, 4), z(4, 64, 64), z(4, 64, 64), z(4, 64, 64))
    for kw in (dict(norm="batch"), dict(norm="layer", post_gamma=v(), gate=v()), dict(pre_gamma=v(), pre_beta=v()),
               dict(norm="layer", pre_beta=v()), dict(norm="layer", post_beta=v(), pre_gamma=v())):
        with pytest.raises(ValueError):
            M.SparseMoE(*W, **kw)


# ---- the C entry points (aligned made-up addresses: nothing is launched) -----------------
A, B, C, D, U = (0x10000 * (i + 1) for i in range(5))


def norm_shape(**kw):
    s = dict(T=100, d=64, dtype=1, eps=1e-5, scale=1.0)
    s.update(kw)
    return ST._NORM_SHAPE(*s.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), BAD_SHAPE), (dict(T=-1), BAD_SHAPE), (dict(T=1 << 31), BAD_SHAPE), (dict(d=0), BAD_SHAPE),
    (dict(d=(1 << 20) + 8), BAD_SHAPE), (dict(eps=0.0), BAD_SHAPE), (dict(eps=float("nan")), BAD_SHAPE),
    (dict(scale=float("inf")), BAD_SHAPE), (dict(d=12), UNSUPPORTED), (dict(d=16392), UNSUPPORTED)])
def test_c_layer_norm_shapes(lib, kw, status):
    n = ctypes.c_size_t(0)
    s = norm_shape(**kw)
    assert lib.moe_layer_norm(s, A, None, B, None, None, C, None, None, None) == status
    assert lib.moe_layer_norm_backward_workspace_size(s, ctypes.byref(n)) == status
    assert lib.moe_layer_norm_backward(s, A, A, None, A, A, A, B, None, None, None, C, 1 << 40, None) == status


def test_c_layer_norm_arguments(lib):
    def fwd(x=A, y=None, gamma=B, beta=None, out=None, u=C, T=100):
        return lib.moe_layer_norm(norm_shape(T=T), x, y, gamma, beta, out, u, None, None, None)
    assert lib.moe_layer_norm(None, A, None, B, None, None, C, None, None, None) == NULL_ARG
    assert fwd(x=None) == fwd(gamma=None) == fwd(u=None) == fwd(y=D) == NULL_ARG
    assert fwd(out=D) == BAD_SHAPE
    assert fwd(x=A + 8) == fwd(beta=B + 4) == fwd(u=C + 2) == MISALIGNED
    assert fwd(T=0, x=None, u=None, gamma=None) == OK

    n = ctypes.c_size_t(0)
    assert lib.moe_layer_norm_backward_workspace_size(norm_shape(T=10000), ctypes.byref(n)) == OK and n.value >= 2 * 64 * 4
    assert lib.moe_layer_norm_backward_workspace_size(norm_shape(), None) == NULL_ARG

    def bwd(out=A, d_u=B, mean=C, rstd=C, gamma=D, dx=U, ws=U, ws_bytes=n.value):
        return lib.moe_layer_norm_backward(norm_shape(T=10000), out, d_u, None, mean, rstd, gamma, dx, None, None, None, ws,
                                           ws_bytes, None)
    assert bwd(out=None) == bwd(d_u=None) == bwd(mean=None) == bwd(rstd=None) == bwd(gamma=None) == bwd(ws=None) == NULL_ARG
    assert bwd(dx=U + 8) == MISALIGNED
    assert bwd(ws_bytes=n.value - 1) == TOO_SMALL


def orth_shape(**kw):
    s = dict(m=64, n=96, E=2, dtype=1, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7)
    s.update(kw)
    return ST._ORTH_SHAPE(*s.values())


PARAMS = ST._MUON_PARAMS(0.1, 0.9, 0.0, 1.0, 1)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), BAD_SHAPE), (dict(m=0), BAD_SHAPE), (dict(n=-1), BAD_SHAPE), (dict(E=0), BAD_SHAPE),
    (dict(steps=0), BAD_SHAPE), (dict(a=float("nan")), BAD_SHAPE), (dict(c=float("inf")), BAD_SHAPE),
    (dict(eps=-1e-9), BAD_SHAPE), (dict(E=65), UNSUPPORTED), (dict(steps=65), UNSUPPORTED),
    (dict(m=(1 << 18) + 1), UNSUPPORTED), (dict(m=16385, n=16385), UNSUPPORTED)])
def test_c_orthogonalize_shapes(lib, kw, status):
    n = ctypes.c_size_t(0)
    s = orth_shape(**kw)
    assert lib.moe_orthogonalize_workspace_size(s, ctypes.byref(n)) == status
    assert lib.moe_orthogonalize(s, A, B, C, 1 << 50, None) == status
    assert lib.moe_muon_update(s, PARAMS, A, B, C, D, 1 << 50, None) == status


def test_c_orthogonalize_arguments(lib):
    n = ctypes.c_size_t(0)
    s = orth_shape()
    assert lib.moe_orthogonalize_workspace_size(None, ctypes.byref(n)) == NULL_ARG
    assert lib.moe_orthogonalize_workspace_size(s, None) == NULL_ARG
    assert lib.moe_orthogonalize_workspace_size(s, ctypes.byref(n)) == OK and n.value > 0
    # the largest sizes that are supported have a workspace of a size
    assert lib.moe_orthogonalize_workspace_size(orth_shape(m=16384, n=1 << 18, E=64, dtype=0), ctypes.byref(n)) == OK
    assert n.value > 64 * 16384 * (1 << 18) * 8
    assert lib.moe_orthogonalize_workspace_size(s, ctypes.byref(n)) == OK

    def orth(g=A, out=B, ws=C, ws_bytes=n.value):
        return lib.moe_orthogonalize(s, g, out, ws, ws_bytes, None)
    assert orth(g=None) == orth(out=None) == orth(ws=None) == NULL_ARG
    assert orth(g=A + 1) == orth(out=B + 1) == orth(ws=C + 128) == MISALIGNED
    assert orth(ws_bytes=n.value - 1) == TOO_SMALL

    def muon(p=PARAMS, w=A, g=B, m=D, ws=C, ws_bytes=n.value):
        return lib.moe_muon_update(s, p, w, g, m, ws, ws_bytes, None)
    assert muon(p=None) == muon(w=None) == muon(g=None) == muon(m=None) == muon(ws=None) == NULL_ARG
    assert muon(m=D + 2) == muon(w=A + 1) == MISALIGNED
    assert muon(ws_bytes=n.value - 1) == TOO_SMALL
    for bad in ((float("nan"), 0.9, 0.0, 1.0, 1), (0.1, float("inf"), 0.0, 1.0, 1), (0.1, 0.9, float("nan"), 1.0, 1),
                (0.1, 0.9, 0.0, float("inf"), 1), (0.1, 0.9, 0.0, 1.0, 2)):
        assert muon(p=ST._MUON_PARAMS(*bad)) == BAD_SHAPE


# ---- the layer's update ------------------------------------------------------------------
@pytest.mark.parametrize("kw,error", [
    (dict(dW_gate=None), ValueError), (dict(dW_gate=z(4, 64, 95)), ValueError), (dict(), TypeError),
    (dict(dW_up=z(4, 64, 96, dtype=F32)), TypeError), (dict(lr=float("nan")), ValueError), (dict(steps=0), ValueError),
    (dict(drop="dW_down"), KeyError), (dict(scale=2.0), TypeError)])
def test_refused_update_of_a_layer_keeps_no_momentum(kw, error):
    block = M.SparseMoE(z(64, 4), z(4, 64, 96), z(4, 64, 96), z(4, 96, 64))
    grads = {"d" + n: torch.ones_like(getattr(block, n)) for n in ("W_gate", "W_up", "W_down")}
    drop, args = kw.get("drop"), dict(lr=0.1)
    for n, t in kw.items():
        (grads if n.startswith("dW") else args)[n] = t
    args.pop("drop", None)
    grads.pop(drop, None)
    with pytest.raises(error):
        block.muon_update(grads, **args)
    assert block.momentum == {} and block._update_ws is None
