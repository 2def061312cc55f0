"""The layer norms with their gradient, the orthogonalised update and the update step, against
their definitions in 64 bits.

Tolerances of the norms are the arithmetic's: half a step of the output's type (2^-8 of the value
in bf16, 2^-24 in fp32) plus, for fp32 sums of n terms in any order, (n + c) 2^-24 times the sum
of the terms' magnitudes, c counting the roundings of each term.

The orthogonalisation's error is not bounded usefully element by element: a step multiplies
small singular values, and what was rounded before it, by up to 3.4. Its tolerance is what the
documented roundings themselves give: the same iteration in 64 bits with fp16 rounding (of one term
or two) where the operator keeps its matrices (`rounded`), and what the plain iteration in fp32
gives (`plain32`), both against the exact one, are doubled; the output's own rounding is added.
"""
from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: U}
NS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1234)


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_sum_amd as M
    M.load_library()
    return M


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def draw(g, *shape, std=1.0, dtype=FP32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def close(got, ref, mag, terms, what=""):
    """|got - ref| <= half a step of got's type + terms * 2^-24 * mag, element by element;
    non-finite values agree."""
    torch.cuda.synchronize()
    tol = HALF[got.dtype] * ref.abs() * (1 + 2.0 ** -7) + terms * U * mag + 1e-37
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), what
    bad = ((g - ref).abs() > tol) & fine
    assert not bool(bad.any()), (what, int(bad.sum()), float(((g - ref).abs() / tol)[fine].max()))


# ---- layer norm --------------------------------------------------------------------------
def norm_inputs(T, d, dt, y, beta, seed=0):
    g = gen(seed + 1000 * d + T)
    x = (draw(g, T, d) * torch.exp(draw(g, d, std=0.5)) + 2 * draw(g, T, 1)).to(dt)
    return (x, draw(g, d, std=0.3) + 1, draw(g, d, std=0.3) if beta else None, draw(g, T, d) if y else None,
            draw(g, T, d).to(dt), draw(g, T, d).to(dt))


def check_norm(got, x, gamma, beta, y, scale, eps, d):
    """Every output of the forward, each from what the one before it stored."""
    if y is not None:
        sx, sy = scale * x.double(), y.double()
        close(got["out"], sx + sy, sx.abs() + sy.abs(), 2, "out")
    s = got["out"].double().cpu()
    mean, size = s.mean(1), s.abs().mean(1)
    close(got["mean"], mean, size, d + 4, "mean")
    var = ((s - mean[:, None]) ** 2).mean(1)
    r = (var + eps).rsqrt()
    # the squares' sum is off by (d + 8) roundings of itself, and by the square of the mean's own error
    close(got["rstd"], r, r + r ** 3 * ((d + 4) * size) ** 2 * U, d / 2 + 8, "rstd")
    z = (s - mean[:, None]) * r[:, None]
    u = z * gamma.double() + (beta.double() if beta is not None else 0)
    mag = gamma.double().abs() * (z.abs() + (r * size)[:, None]) + u.abs()
    close(got["u"], u, mag, d + 16, "u")


def check_norm_grad(res, s, d_u, d_out, mean, rstd, gamma, scale, T, d):
    s, du, mean, r, gm = (t.double().cpu() for t in (s, d_u, mean, rstd, gamma))
    do = d_out.double().cpu() if d_out is not None else torch.zeros_like(du)
    mean, r = mean[:, None], r[:, None]
    z = (s - mean) * r
    dz = du * gm
    D = do + r * (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True))
    mag = do.abs() + r.abs() * (dz.abs() + dz.abs().mean(1, keepdim=True) + z.abs() * (dz * z).abs().mean(1, keepdim=True))
    close(res["dx"], scale * D, abs(scale) * mag, d + 16, "dx")
    if res["dy"] is not None:
        close(res["dy"], D, mag, d + 16, "dy")
    close(res["dgamma"], (du * z).sum(0), (du * z).abs().sum(0), T + 8, "dgamma")
    close(res["dbeta"], du.sum(0), du.abs().sum(0), T + 8, "dbeta")


# widths on both sides of every split of a row over threads, and rows that leave a workgroup's last ones empty
WIDTHS = [8, 64, 120, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_layer_norm_and_gradient(moe, d, dt):
    for T, y, beta in ((1, True, True), (37, False, False), (512, True, True), (533, True, True)):
        say("layer norm", T, d, dt)
        x, gm, bt, yy, du, do = norm_inputs(T, d, dt, y, beta)
        scale, eps = (0.75 if y else 1.0), 1e-5
        dev = [None if t is None else t.cuda() for t in (x, gm, bt, yy, du, do)]
        got = moe.moe_layer_norm(dev[0], dev[1], dev[2], y=dev[3], residual_scale=scale, eps=eps)
        check_norm(got, x, gm, bt, yy, scale, eps, d)
        res = moe.moe_layer_norm_backward(got["out"], dev[4], got["mean"], got["rstd"], dev[1],
                                          d_out=dev[5] if y else None, residual_scale=scale, want_dy=y)
        check_norm_grad(res, got["out"], du, do if y else None, got["mean"], got["rstd"], gm, scale, T, d)


def test_layer_norm_rows_past_the_grid(moe):
    """More rows than workgroups: rows in strides, in both passes, and the last ones."""
    T, d = (1 << 20) * 16 + 21, 8
    x = torch.randn(T, d, device="cuda", dtype=BF16)
    gm, du = torch.ones(d, device="cuda"), torch.randn(T, d, device="cuda", dtype=BF16)
    got = moe.moe_layer_norm(x, gm)
    at = torch.cat([torch.arange(50), torch.arange(T - 50, T), torch.arange(T // 2 - 40, T // 2 + 40)])
    pick = {n: got[n][at.cuda()] if got[n] is not None else None for n in ("out", "u", "mean", "rstd")}
    check_norm(pick, x[at.cuda()].cpu(), gm.cpu(), None, None, 1.0, 1e-5, d)
    res = moe.moe_layer_norm_backward(x, du, got["mean"], got["rstd"], gm)
    ref = du.double().sum(0)
    assert float((res["dbeta"].double() - ref).abs().max()) <= (T ** 0.5 + 8) * 8 * U * float(du.double().abs().sum(0).max())
    z = (x.double() - got["mean"].double()[:, None]) * got["rstd"].double()[:, None]
    ref = (du.double() * z).sum(0)
    assert float((res["dgamma"].double() - ref).abs().max()) <= (T ** 0.5 + 8) * 8 * U * float((du * z).abs().sum(0).max())


def test_layer_norm_past_2_31_elements(moe):
    T, d = (1 << 18) + 3, 8192
    x = torch.randn(T, d, device="cuda", dtype=BF16)
    gm, bt = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    got = moe.moe_layer_norm(x, gm, bt)
    at = torch.tensor([0, 1, (1 << 18) - 1, 1 << 18, T - 1], device="cuda")
    check_norm({n: got[n][at] for n in ("out", "u", "mean", "rstd")}, x[at].cpu(), gm.cpu(), bt.cpu(), None, 1.0, 1e-5, d)
    res = moe.moe_layer_norm_backward(x, got["u"], got["mean"], got["rstd"], gm)
    s, du, m, r = x[at].double(), got["u"][at].double(), got["mean"][at].double()[:, None], got["rstd"][at].double()[:, None]
    z, dz = (s - m) * r, du * gm.double()
    D = r * (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True))
    mag = r * (dz.abs() + dz.abs().mean(1, keepdim=True) + z.abs() * (dz * z).abs().mean(1, keepdim=True))
    close(res["dx"][at], D.cpu(), mag.cpu(), d + 16, "dx")


@pytest.mark.parametrize("d", [64, 1024, 4096])
def test_layer_norm_gradient_by_differences(moe, d):
    """<d_u, u> along a direction of x, gamma and beta: the gradient's against the definition's
    central difference in 64 bits (step h: off by h^2 times a third derivative of order 1)."""
    g = gen(d)
    T, eps, h = 19, 1e-5, 1e-4
    x, gm, bt, du = draw(g, T, d), draw(g, d), draw(g, d), draw(g, T, d)
    vx, vg, vb = (torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (x, gm, bt))

    def value(k):
        s, gg, b = x.double() + k * vx, gm.double() + k * vg, bt.double() + k * vb
        s = s - s.mean(1, keepdim=True)
        return (((s / ((s * s).mean(1, keepdim=True) + eps).sqrt()) * gg + b) * du.double()).sum()
    want = float(value(h) - value(-h)) / (2 * h)
    f = moe.moe_layer_norm(x.cuda(), gm.cuda(), bt.cuda(), eps=eps)
    r = moe.moe_layer_norm_backward(x.cuda(), du.cuda(), f["mean"], f["rstd"], gm.cuda())
    parts = [(r[n].double().cpu() * t) for n, t in (("dx", vx), ("dgamma", vg), ("dbeta", vb))]
    got, size = sum(float(p.sum()) for p in parts), sum(float(p.abs().sum()) for p in parts)
    assert abs(got - want) <= size * ((d + 16) * U + 1e-6), (got, want, size)


def test_layer_norm_special_rows(moe):
    """A constant row's variance is 0, a far mean cancels, a row that is not finite is alone."""
    d = 2048
    x = torch.randn(6, d)
    x[1] = 3.0                                   # variance 0: u = beta
    x[2] = 1e4 + torch.arange(d).float() / 64    # mean 1e4, spread 10
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    x[5] = 0
    gm, bt = torch.randn(d).cuda(), torch.randn(d).cuda()
    got = moe.moe_layer_norm(x.cuda(), gm, bt)
    check_norm({n: got[n][[0, 1, 2, 5]] for n in ("out", "u", "mean", "rstd")}, x[[0, 1, 2, 5]], gm.cpu(), bt.cpu(), None, 1.0,
               1e-5, d)
    assert torch.equal(got["u"][1], bt) and torch.equal(got["u"][5], bt)
    assert bool(torch.isnan(got["u"][3]).any()) and bool(torch.isnan(got["u"][4]).all())
    r = moe.moe_layer_norm_backward(x.cuda(), torch.ones(6, d).cuda(), got["mean"], got["rstd"], gm)
    assert bool(torch.isfinite(r["dx"][[0, 1, 2, 5]]).all())


def test_layer_norm_without_rows(moe):
    x, gm = torch.empty(0, 64, device="cuda", dtype=BF16), torch.ones(64, device="cuda")
    f = moe.moe_layer_norm(x, gm)
    assert f["u"].shape == (0, 64) and f["mean"].shape == (0,)
    r = moe.moe_layer_norm_backward(x, x, f["mean"], f["rstd"], gm)
    assert float(r["dgamma"].abs().sum()) == 0 and float(r["dbeta"].abs().sum()) == 0


def test_layer_norm_sum_and_norm_are_two_calls(moe):
    """One call with y gives the bits of the sum and then the norm of it; the same bits twice."""
    x, gm, bt, y, du, do = (t.cuda() for t in norm_inputs(300, 1408, BF16, True, True))
    a = moe.moe_layer_norm(x, gm, bt, y=y, residual_scale=0.5)
    b = moe.moe_layer_norm(a["out"], gm, bt)
    assert all(torch.equal(a[n], b[n]) for n in ("u", "mean", "rstd"))
    g = [moe.moe_layer_norm_backward(x, du, b["mean"], b["rstd"], gm, d_out=do, want_dy=True) for _ in range(2)]
    assert all(torch.equal(g[0][n], g[1][n]) for n in g[0])
    assert torch.equal(g[0]["dx"], g[0]["dy"])
    assert moe.moe_layer_norm(x, gm, want_stats=False)["mean"] is None


@pytest.mark.parametrize("T", [77, 601])
def test_layer_norm_c_outputs_left_out_and_in_place(moe, T):
    from sparse_mixture_experts_sum_amd import step as ST
    x, gm, bt, y, du, do = (t.cuda() for t in norm_inputs(T, 520, BF16, True, True))
    ref = moe.moe_layer_norm(x, gm, bt, y=y, residual_scale=0.5)
    shape = ST._NORM_SHAPE(T, 520, 1, 1e-5, 0.5)
    xx, u = x.clone(), torch.empty_like(x)
    ST._call("moe_layer_norm", x.device, shape, xx.data_ptr(), y.data_ptr(), gm.data_ptr(), bt.data_ptr(), xx.data_ptr(),
             u.data_ptr(), None, None)
    assert torch.equal(xx, ref["out"]) and torch.equal(u, ref["u"])
    args = (ref["out"], du, ref["mean"], ref["rstd"], gm)
    full = moe.moe_layer_norm_backward(*args, d_out=do, residual_scale=0.5, want_dy=True)
    names = ("dx", "dy", "dgamma", "dbeta")
    from sparse_mixture_experts_sum_amd.training import _scratch
    for keep in names + ("none",):
        outs = {n: torch.full_like(full[n], 7) for n in names}
        ws, n = _scratch("moe_layer_norm_backward_workspace_size", shape, x.device, None)
        ST._call("moe_layer_norm_backward", x.device, shape, args[0].data_ptr(), du.data_ptr(), do.data_ptr(),
                 *(t.data_ptr() for t in args[2:]), *(outs[k].data_ptr() if k == keep else None for k in names),
                 ws.data_ptr(), n)
        for k in names:
            assert torch.equal(outs[k], full[k] if k == keep else torch.full_like(full[k], 7)), (keep, k)
    for over in (du, do):  # dx over either gradient
        a, b = du.clone(), do.clone()
        to = a if over is du else b
        ws, n = _scratch("moe_layer_norm_backward_workspace_size", shape, x.device, None)
        ST._call("moe_layer_norm_backward", x.device, shape, args[0].data_ptr(), a.data_ptr(), b.data_ptr(),
                 *(t.data_ptr() for t in args[2:]), to.data_ptr(), None, None, None, ws.data_ptr(), n)
        assert torch.equal(to, full["dx"])


@pytest.mark.parametrize("T,d", [(1, 64), (300, 1024), (512, 8200), (513, 1024)])
def test_layer_norm_gradient_over_its_inputs(moe, T, d):
    """Every output, dx or dy over d_u or d_out: the column sums are those of the d_u that was given."""
    from sparse_mixture_experts_sum_amd import step as ST
    from sparse_mixture_experts_sum_amd.training import _scratch
    x, gm, _, _, du, do = (t.cuda() if t is not None else None for t in norm_inputs(T, d, BF16, False, False))
    f = moe.moe_layer_norm(x, gm)
    want = moe.moe_layer_norm_backward(x, du, f["mean"], f["rstd"], gm, d_out=do, residual_scale=0.5, want_dy=True)
    shape = ST._NORM_SHAPE(T, d, 1, 1e-5, 0.5)
    ws, n = _scratch("moe_layer_norm_backward_workspace_size", shape, x.device, None)
    for over in ("dx", "dy", "both"):
        a, b = du.clone(), do.clone()
        dx, dy = (a, b) if over == "both" else (a, torch.empty_like(a)) if over == "dx" else (torch.empty_like(a), a)
        dg, db = torch.empty_like(gm), torch.empty_like(gm)
        ST._call("moe_layer_norm_backward", x.device, shape, x.data_ptr(), a.data_ptr(), b.data_ptr(), f["mean"].data_ptr(),
                 f["rstd"].data_ptr(), gm.data_ptr(), dx.data_ptr(), dy.data_ptr(), dg.data_ptr(), db.data_ptr(),
                 ws.data_ptr(), n)
        for k, v in zip(("dx", "dy", "dgamma", "dbeta"), (dx, dy, dg, db)):
            assert torch.equal(v, want[k]), (over, k)


# ---- orthogonalisation ---------------------------------------------------------------------
def plain(g, steps, co=NS, eps=1e-7, dtype=torch.float64):
    """The definition, matrix by matrix of the last two dimensions."""
    a, b, c = co
    n = g.double().pow(2).sum((1, 2), keepdim=True).sqrt() + eps
    x = (g.double() / n).to(dtype)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(steps):
        A = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.transpose(1, 2) if tall else x


def in_strips(E, s, l, terms):
    """Whether a matrix's steps are two launches each: none share a Gram matrix."""
    return 128 < s <= 256 and 8 * E * -(-l // 128) * terms <= 256


def rounded(g, steps, terms, co=NS, eps=1e-7):
    """The iteration as the operator takes it, in 64 bits but for the roundings of what it keeps."""
    a, b, c = co
    g = g.double()
    if g.shape[1] > g.shape[2]:
        return rounded(g.transpose(1, 2).contiguous(), steps, terms, co, eps).transpose(1, 2)

    def keep(t):
        t = t.float()
        hi = t.half().float()
        return (hi if terms == 1 else hi + ((t - hi) * 2048).half().float() / 2048).double()

    n = g.pow(2).sum((1, 2), keepdim=True).sqrt() + eps
    scale = 2.0 ** math.ceil(math.log2(math.sqrt(g.shape[2])))
    p = torch.exp2(torch.floor(torch.log2(scale / n)))
    x, unit = keep(g * p), 1 / (n * p)
    eye = torch.eye(g.shape[1], dtype=torch.float64, device=g.device)
    done = 0
    while done < steps:
        left = steps - done
        few = terms == 2 and g.shape[1] <= 24
        two = left >= 2 and not in_strips(*g.shape, terms) and not (few and (left % 2 or g.shape[2] <= 384)) and (terms == 2 or done == 0 or (g.shape[2] >= 2 * g.shape[1] and left % 2 == 0))
        A = keep(unit ** 2 * (x @ x.transpose(1, 2).contiguous()))
        P = keep(a * eye + b * A + c * (A @ A))
        if two:
            A = keep(P @ keep(P @ A))
            P = keep(keep(a * eye + b * A + c * (A @ A)) @ P)
        done += 2 if two else 1
        x = unit * (P @ x)
        if done < steps:
            x = keep(scale * x)
            unit = torch.full_like(unit, 1 / scale)
    return x


def norm(t):
    return t.double().pow(2).sum((1, 2)).sqrt()


def check_orth(got, g, steps, terms, co=NS, eps=1e-7):
    """Each matrix's error by its norm, and each value's by 8 times the typical one, or by its
    own share: the last product is M X, and a rounding of M's diagonal, which is most of M, is off by
    as much of the value in every place. (Where the values are even, as in a gradient's matrix, the
    first covers that; in an outer product single values are 15 times the typical one and more.)"""
    E = plain(g, steps, co, eps)
    slack = 2 * (norm(rounded(g, steps, terms, co, eps) - E) + norm(plain(g, steps, co, eps, FP32) - E)) + 1e-6 * norm(E)
    off = got.double() - E
    half = HALF[got.dtype]
    size = math.sqrt(E.shape[1] * E.shape[2])
    assert bool((norm(off) <= slack + half * norm(E)).all()), (norm(off) / norm(E), slack / norm(E))
    most = 8 * slack[:, None, None] / size + (half * (1 + 2 ** -7) + 2 * (slack / norm(E))[:, None, None]) * E.abs()
    # (a matrix of one row or column has the error of a factor: it lies where the values lie)
    if min(E.shape[1:]) > 8:
        assert bool((off.abs() <= most).all()), float((off.abs() / most).max())


def stack(E, m, n, dt, seed=0, std=1e-3):
    """Gradients: a few shared directions of falling weight, and noise."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * m + n)
    r = max(1, min(m, n) // 8)
    w = torch.arange(1, r + 1, device="cuda").float().rsqrt()
    a = torch.randn(E, m, r, generator=g, device="cuda") * w
    x = a @ torch.randn(E, r, n, generator=g, device="cuda").contiguous()
    return ((x + torch.randn(E, m, n, generator=g, device="cuda")) * std).to(dt)


def terms_of(m, n, dt):
    return 1 if dt is BF16 and min(m, n) > 128 else 2


SIZES = [(1, 1, 1), (2, 1, 300), (3, 300, 1), (2, 16, 16), (5, 31, 33), (8, 64, 128), (3, 128, 64), (1, 127, 129),
         (2, 129, 1000), (5, 201, 333), (1, 250, 4090), (1, 1500, 200), (3, 256, 256), (2, 200, 333), (2, 333, 200), (1, 512, 513), (1, 513, 640), (2, 640, 520), (1, 520, 2056),
         (1, 2056, 520), (64, 24, 40), (3, 64, 384), (2, 64, 385), (2, 17, 1000), (16, 16, 680), (3, 1531, 33), (1, 64, 12288), (1, 9, 12289)]


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_orthogonalize(moe, size, dt):
    E, m, n = size
    g = stack(E, m, n, dt)
    for steps in (1, 2, 3, 5):
        say("orthogonalize", size, dt, steps)
        check_orth(moe.moe_orthogonalize(g, steps=steps), g, steps, terms_of(m, n, dt))


@pytest.mark.parametrize("size", [(8, 1024, 2048), (8, 2048, 1024), (13, 1408, 1536), (13, 1536, 1408), (3, 2100, 2300)],
                         ids=lambda s: "x".join(map(str, s)))
def test_orthogonalize_large_tiles(moe, size):
    """Products of more than a round of 256-row tiles, whose last ones are half empty."""
    E, m, n = size
    g = stack(E, m, n, BF16)
    say("orthogonalize", size)
    check_orth(moe.moe_orthogonalize(g), g, 5, 1)


def test_orthogonalize_converges_to_the_polar_factor(moe):
    """With coefficients that drive the singular values to 1, the result is U V^T of the SVD."""
    g = stack(2, 96, 160, FP32)
    o = moe.moe_orthogonalize(g, steps=20, coefficients=(1.5, -0.5, 0.0)).double()
    u, s, vt = torch.linalg.svd(g.double().cpu(), full_matrices=False)
    assert float(s.min() / s.max()) > 0.01  # 20 steps are enough
    assert float((o.cpu() - u @ vt).abs().max()) < 2e-5
    assert float((o @ o.transpose(1, 2) - torch.eye(96, device="cuda")).abs().max()) < 2e-5


def test_orthogonalize_rank_one(moe):
    """An outer product: bf16 kept in one term is off by its roundings, times what the steps
    multiply the rest by; kept in two it is as in fp32."""
    r = torch.Generator(device="cuda").manual_seed(3)
    a, b = torch.randn(1, 700, 1, generator=r, device="cuda"), torch.randn(1, 1, 800, generator=r, device="cuda")
    for dt, m in ((FP32, 700), (BF16, 700), (BF16, 300), (BF16, 100)):
        g = (a[:, :m] * b).to(dt)
        check_orth(moe.moe_orthogonalize(g), g, 5, terms_of(m, 800, dt))


def test_orthogonalize_scales_exactly(moe):
    """A power of two in front of the matrix changes no bit, down to and up to fp32's limits. (At
    2^-120 the values below 2^-6 are no multiples of fp32's last step, 2^-149, any more where they have
    24 bits: another matrix, by half of that step at most, which is held to the definition.)"""
    g = torch.randn(2, 100, 170, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    ref = moe.moe_orthogonalize(g, eps=0.0)
    for p in (-120, -60, 60, 124):
        scaled = g * 2.0 ** p
        same = torch.equal(scaled.double() * 2.0 ** -p, g.double())
        assert same == (p != -120)
        got = moe.moe_orthogonalize(scaled, eps=0.0)
        if same:
            assert torch.equal(got, ref), p
        else:
            check_orth(got, scaled, 5, 2, eps=0.0)
    small = moe.moe_orthogonalize(g * 2.0 ** -40)  # eps counts beside the norm
    check_orth(small, g * 2.0 ** -40, 5, 2)


@pytest.mark.parametrize("m,n,dt", [(262144, 8200, BF16), (8200, 262144, FP32)])
def test_orthogonalize_past_2_31_values(moe, m, n, dt):
    """One step of a matrix with the longest side there is and more than 2^31 values, 256 of its long side
    at a time against P X with P in 64 bits. Four directions hold four fifths of it (singular values of
    0.45: P is far from a I). Tolerance, of each of these parts' norm: half a step of the result; where one term is
    kept 2^-9 for P's rounding of 2^-11 and the products, and A's in fp16's last steps (values of
    1 / s lie among them), 2^-25 s of its norm at most, times |b| + 2 |c|."""
    tall, s, l = m > n, min(m, n), max(m, n)
    g = torch.empty(m, n, device="cuda", dtype=dt)
    side = (lambda t, i, w: t[i:i + w].t()) if tall else (lambda t, i, w: t[:, i:i + w])
    r = torch.Generator(device="cuda").manual_seed(11)
    u = torch.randn(s, 4, device="cuda", generator=r)
    for i in range(0, l, 8192):
        x = torch.randn(s, 8192, device="cuda", generator=r) + u @ torch.randn(4, 8192, device="cuda", generator=r)
        side(g, i, 8192).copy_(x)
    got = moe.moe_orthogonalize(g, steps=1)
    A = torch.zeros(s, s, device="cuda")
    for i in range(0, l, 8192):  # (sums of 8192 fp32 terms, and of 32 of these)
        x = side(g, i, 8192).float().contiguous()
        A += x @ x.t()
    t = A.diagonal().double().sum().sqrt() + 1e-7  # the norm
    A = A.double() / t ** 2
    for i in (0, 128, 131072 - 64, l - 512, l - 256):
        x = side(g, i, 256).double().contiguous() / t
        Ax = A @ x
        want = NS[0] * x + NS[1] * Ax + NS[2] * (A @ Ax)
        off = side(got, i, 256).double() - want
        tol = HALF[dt] + (2.0 ** -9 + 2.0 ** -25 * s * (abs(NS[1]) + 2 * abs(NS[2])) if dt is BF16 else 1e-5)
        assert float(off.norm() / want.norm()) <= tol, i


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_orthogonalize_special_matrices(moe, dt):
    """Zeros give zeros; a value that is not finite spoils its own matrix and no other."""
    for m, n in ((72, 200), (600, 530), (140, 200)):
        g = stack(5, m, n, dt)
        ref = moe.moe_orthogonalize(g)
        bad = g.clone()
        bad[1] = 0
        bad[2, 3, 4] = float("nan")
        bad[4, m - 1, n - 1] = float("inf")
        got = moe.moe_orthogonalize(bad)
        assert float(got[1].float().abs().max()) == 0
        assert not bool(torch.isfinite(got[2]).any()) and not bool(torch.isfinite(got[4]).any())
        assert torch.equal(got[0], ref[0]) and torch.equal(got[3], ref[3])
        assert float(moe.moe_orthogonalize(torch.zeros_like(g), eps=0.0).float().abs().max()) == 0


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_orthogonalize_buffers(moe, dt):
    """In place, a workspace full of garbage or larger than needed, matrices at odd addresses,
    one matrix without its stack's dimension."""
    for m, n in ((70, 201), (530, 640), (201, 130)):
        g = stack(3, m, n, dt)
        ref = moe.moe_orthogonalize(g)
        same = g.clone()
        assert moe.moe_orthogonalize(same, out=same) is same and torch.equal(same, ref)
        ws = torch.full((200 << 20,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(moe.moe_orthogonalize(g, workspace=ws), ref)
        buf, out = torch.full((g.numel() + 9,), 5.0, dtype=dt, device="cuda"), torch.full((g.numel() + 9,), 5.0, dtype=dt, device="cuda")
        at, to = buf[1:1 + g.numel()].view(g.shape), out[3:3 + g.numel()].view(g.shape)
        at.copy_(g)
        moe.moe_orthogonalize(at, out=to)
        assert torch.equal(to, ref)
        assert float((out[:3] - 5).abs().sum() + (out[3 + g.numel():] - 5).abs().sum()) == 0
        assert torch.equal(moe.moe_orthogonalize(g[1]), moe.moe_orthogonalize(g[1:2])[0])


def test_orthogonalize_is_reproducible_and_captured(moe):
    """The same bits again; captured and replayed on new values, with eager work between."""
    for m, n, dt in ((90, 130, FP32), (640, 700, BF16), (150, 260, FP32)):
        g = stack(2, m, n, dt)
        others = [stack(2, m, n, dt, seed=s) for s in (1, 2, 3)]
        want = [moe.moe_orthogonalize(t) for t in others]
        assert torch.equal(moe.moe_orthogonalize(g), moe.moe_orthogonalize(g))
        x, out = g.clone(), torch.empty_like(g)
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            moe.moe_orthogonalize(x, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_orthogonalize(x, out=out, workspace=ws)
        for t, w in zip(others, want):
            x.copy_(t)
            graph.replay()
            moe.moe_orthogonalize(g)  # eager work, on a workspace of its own
            torch.cuda.synchronize()
            assert torch.equal(out, w)


def test_orthogonalize_on_two_streams(moe):
    a, b = stack(2, 300, 400, BF16, seed=1), stack(4, 600, 520, BF16, seed=2)
    wa, wb = moe.moe_orthogonalize(a), moe.moe_orthogonalize(b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s):
            oa = moe.moe_orthogonalize(a)
        with torch.cuda.stream(t):
            ob = moe.moe_orthogonalize(b)
        got.append((oa, ob))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_shared_memory_is_refused(moe):
    buf = torch.randn(4, 40, 72, device="cuda")
    a, b, c = buf[:2], buf[1:3], buf[2:]
    with pytest.raises(ValueError, match="apart"):
        moe.moe_orthogonalize(a, out=b)
    assert torch.equal(moe.moe_orthogonalize(a, out=c), moe.moe_orthogonalize(a))
    m = torch.zeros(2, 40, 72, device="cuda")
    for w, g, mom in ((a, a, m), (a, b, m), (a, m, b), (m, a, a), (m, b, a)):
        with pytest.raises(ValueError, match="share no memory"):
            moe.moe_muon_update(w, g, mom, lr=0.1)


# ---- the update step -------------------------------------------------------------------------
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("size,dt", [((3, 70, 201), FP32), ((3, 70, 201), BF16), ((2, 640, 536), BF16), ((2, 536, 640), BF16),
                                     ((5, 201, 333), FP32), ((2, 200, 1501), BF16), ((2, 1501, 200), BF16), ((1, 1, 9), FP32)])
def test_muon_update(moe, size, dt, nesterov):
    E, m, n = size
    say("muon", size, dt, nesterov)
    g, w = stack(E, m, n, dt), (torch.randn(size, device="cuda") * 0.02).to(dt)
    mom = torch.randn(size, device="cuda") * 1e-3
    lr, mu, wd, scale = 0.05, 0.9, 0.1, 1.5
    w1, m1 = w.clone(), mom.clone()
    moe.moe_muon_update(w1, g, m1, lr=lr, momentum=mu, nesterov=nesterov, weight_decay=wd, scale=scale)
    f = lambda v: torch.tensor(v, dtype=FP32).double().item()  # noqa: E731  (what the library is given)
    kept = f(mu) * mom.double()
    m_ref = kept + g.double()
    close(m1, m_ref.cpu(), (kept.abs() + m_ref.abs()).cpu(), 2, "m")
    u = f(mu) * m1.double() + g.double() if nesterov else m1.double()
    terms = terms_of(m, n, dt)
    O = plain(u, 5)
    slack = 2 * (norm(rounded(u, 5, terms) - O) + norm(plain(u, 5, dtype=FP32) - O)) + 1e-6 * norm(O)
    keep, rate = 1 - f(lr) * f(wd), f(lr) * f(scale)
    ref = keep * w.double() - rate * O
    off = (w1.double() - ref).abs()
    most = HALF[dt] * ref.abs() * (1 + 2 ** -7) + rate * (8 * slack / math.sqrt(m * n))[:, None, None] + \
        8 * U * (w.double().abs() + rate * O.abs())
    if min(m, n) > 8:
        assert bool((off <= most).all()), float((off / most).max())
    else:
        assert bool((off <= most + rate * slack[:, None, None]).all())


def test_muon_update_without_steps_of_size(moe):
    """lr 0 leaves the weights' bits, momentum 0 takes the gradient, zero gradients move nothing."""
    g, w = stack(2, 40, 72, BF16), (torch.randn(2, 40, 72, device="cuda") * 0.02).to(BF16)
    w1, m1 = w.clone(), torch.randn(2, 40, 72, device="cuda")
    moe.moe_muon_update(w1, g, m1, lr=0.0, momentum=0.0)
    assert torch.equal(w1, w) and torch.equal(m1, g.float())
    moe.moe_muon_update(w1, torch.zeros_like(g), torch.zeros_like(m1), lr=0.1)
    assert torch.equal(w1, w)


# ---- together, as a training step -------------------------------------------------------------
def layer(moe, dt, T=96, d=128, f=192, E=4, seed=0, **kw):
    g = gen(seed)
    W = [draw(g, d, E, std=0.3).to(dt), draw(g, E, d, f, std=0.1).to(dt), draw(g, E, d, f, std=0.1).to(dt),
         draw(g, E, f, d, std=0.1).to(dt)]
    gb = [1 + draw(g, d, std=0.2), draw(g, d, std=0.2), 1 + draw(g, d, std=0.2), draw(g, d, std=0.2)]
    x = (draw(g, T, d) + 0.5).to(dt)
    dev = [t.cuda() for t in W + gb]
    block = moe.SparseMoE(*dev[:4], k=2, norm="layer", pre_gamma=dev[4], pre_beta=dev[5], post_gamma=dev[6], post_beta=dev[7],
                          residual_scale=0.75, norm_eps=1e-5, **kw)
    return block, W, gb, x


def reference_block(x, W, gb, idx, eps=1e-5):
    """The block in 64 bits on the device's choice of experts."""
    W_g, W_gate, W_up, W_down = W
    ln = torch.nn.functional.layer_norm
    u = ln(x, x.shape[1:], gb[0], gb[1], eps)
    p = torch.softmax(u @ W_g, 1)
    w = p.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(W_gate.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(u[t] @ W_gate[e]) * (u[t] @ W_up[e])
        y = y.index_add(0, t, w[t, j, None] * (h @ W_down[e]))
    return ln(0.75 * x + y, x.shape[1:], gb[2], gb[3], eps)


def test_block_with_layer_norms_in_fp32(moe):
    """Output and every gradient of norm, layer, norm in fp32 against 64-bit automatic
    differentiation. Tolerance: sums of at most 192 fp32 terms, ten roundings deep in a chain of
    seven products and norms whose factors are of order 1: 3e-5 of each tensor's largest value."""
    block, W, gb, x = layer(moe, FP32)
    out = block(x.cuda())
    idx = block.last["idx"].long().cpu()
    leaves = [t.double().requires_grad_() for t in [x] + W + gb]
    ref = reference_block(leaves[0], leaves[1:5], leaves[5:], idx)
    d_out = draw(gen(5), *x.shape)
    want = torch.autograd.grad(ref, leaves, d_out.double())
    got = block.backward(d_out.cuda())
    names = ("dx", "dW_g", "dW_gate", "dW_up", "dW_down", "d_pre_gamma", "d_pre_beta", "d_post_gamma", "d_post_beta")
    torch.cuda.synchronize()
    ref = ref.detach()
    assert float((out.double().cpu() - ref).abs().max()) <= 3e-5 * float(ref.abs().max())
    for n, w in zip(names, want):
        assert float((got[n].double().cpu() - w).abs().max()) <= 3e-5 * float(w.abs().max()), n
    assert set(got) == set(names)


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_training_steps(moe, dt):
    """Three steps of norm, layer, gradients and update: each update is what the entry points give
    by themselves from the same gradients, with the factor of each matrix's shape."""
    block, W, gb, x = layer(moe, dt)
    names = ("W_gate", "W_up", "W_down")
    mom = {n: torch.zeros_like(getattr(block, n), dtype=FP32) for n in names}
    for i in range(3):
        block(x.cuda())
        grads = block.backward(draw(gen(i), *x.shape).cuda())
        want = {}
        for n in names:
            want[n] = getattr(block, n).clone()
            r, c = want[n].shape[1:]
            moe.moe_muon_update(want[n], grads["d" + n], mom[n], lr=0.02, weight_decay=0.01, scale=max(1.0, c / r) ** 0.5)
        before = {n: getattr(block, n).clone() for n in names}
        block.muon_update(grads, lr=0.02, weight_decay=0.01)
        for n in names:
            assert torch.equal(getattr(block, n), want[n]) and torch.equal(block.momentum[n], mom[n])
            assert not torch.equal(before[n], want[n])
    assert bool(torch.isfinite(block(x.cuda()).float()).all())


def test_training_step_captured(moe):
    """The whole step in a graph, replayed on new rows, against the same steps run eagerly."""
    eager, _, _, x = layer(moe, BF16)
    held, _, _, _ = layer(moe, BF16)
    rows = [draw(gen(20 + i), *x.shape).to(BF16).cuda() for i in range(4)]
    d_out = draw(gen(30), *x.shape).to(BF16).cuda()
    want = []
    for r in rows:
        want.append(eager(r).clone())
        eager.muon_update(eager.backward(d_out), lr=0.02)
    buf = rows[0].clone()
    held(buf)
    held.backward(d_out)
    for n in ("W_gate", "W_up", "W_down"):  # (the first step's momentum and workspace, before the capture)
        held.momentum[n] = torch.zeros_like(getattr(held, n), dtype=FP32)
    held._update_ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = held(buf)
        held.muon_update(held.backward(d_out), lr=0.02)
    for r, w in zip(rows, want):
        buf.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    for n in ("W_gate", "W_up", "W_down"):
        assert torch.equal(getattr(held, n), getattr(eager, n)) and torch.equal(held.momentum[n], eager.momentum[n])


def test_first_update_in_a_capture_is_refused(moe):
    """A momentum made by the captured call would be zeroed again by every replay."""
    block, _, _, x = layer(moe, BF16)
    block(x.cuda())
    grads = block.backward(draw(gen(1), *x.shape).cuda())
    before = block.W_up.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="before the capture"):
            block.muon_update(grads, lr=0.02)
    assert not block.momentum and torch.equal(block.W_up, before)
    block.muon_update(grads, lr=0.02)
    assert not torch.equal(block.W_up, before)


def test_layer_with_one_norm_of_the_two(moe):
    """Only the norm before, or only the one after: what the block gives is what the entry points give."""
    block, W, gb, x = layer(moe, BF16)
    xx = x.cuda()
    pre = moe.SparseMoE(block.W_g, block.W_gate, block.W_up, block.W_down, norm="layer", pre_gamma=block.pre_gamma)
    y = pre(xx)
    u = moe.moe_layer_norm(xx, block.pre_gamma, eps=1e-6)["u"]
    assert torch.equal(y, moe.moe_forward(u, block.W_g, None, block.W_gate, block.W_up, block.W_down, k=2)["y"])
    g = pre.backward(torch.ones_like(y))
    assert "d_pre_gamma" in g and "d_pre_beta" not in g and "d_post_gamma" not in g
    post = moe.SparseMoE(block.W_g, block.W_gate, block.W_up, block.W_down, norm="layer", post_gamma=block.post_gamma,
                         post_beta=block.post_beta)
    o = post(xx)
    y = moe.moe_forward(xx, block.W_g, None, block.W_gate, block.W_up, block.W_down, k=2)["y"]
    assert torch.equal(o, moe.moe_layer_norm(xx, block.post_gamma, block.post_beta, y=y, eps=1e-6)["u"])
    g = post.backward(torch.ones_like(o))
    assert "d_post_beta" in g and "d_pre_gamma" not in g and g["dx"].dtype is BF16
