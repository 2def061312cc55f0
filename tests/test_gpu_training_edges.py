"""The training operators where their sums cancel, where groups start behind row 0, and in the
variants that only larger or other sizes reach, against their definitions in 64 bits.

Tolerances as in test_gpu_training.py: half a step of the output's type plus, for fp32 sums,
2^-24 of the terms' magnitudes for each rounding on the way.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_sum_amd as M
from sparse_mixture_experts_sum_amd import training as TR
from tests.test_gpu_training import (BF16, FP32, close, cuda, draw, gen, layer_inputs, matmul_ref,  # noqa: F401
                                     moe, offsets_of, route_inputs, route_ref, say, swiglu_ref)

pytestmark = pytest.mark.gpu


# ---- router gradient -------------------------------------------------------------------
def _route_alone(moe, T, E, k, dt, d=64, seed=0, **given):
    """dx and dW_g of given weights, probabilities and dw (no losses), and the ds they are of."""
    r = gen(seed)
    t = dict(x=draw(r, T, d, dtype=dt), W=draw(r, d, E, dtype=dt), probs=torch.zeros(T, E),
             idx=torch.arange(k).repeat(T, 1).int(), w=torch.ones(T, k), dw=draw(r, T, k))
    t.update(given)
    out = moe.moe_route_backward(*cuda(*(t[n] for n in ("x", "W", "probs", "idx", "w", "dw"))), renormalize=False)
    return t, out, out["dlogits"].double().cpu()


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("E", [4, 64])
def test_route_dx_where_ds_cancels(moe, dt, E):
    # ds sums to zero over a token's experts, so that dx keeps 1e-5 of its terms here: the
    # terms have to be ds in 32 bits. One rounding per added expert, and one of each product
    # (ds as a sum of narrower terms: those of the smaller ones are some 2^-8 of it more).
    say("route dx cancels", dt, E)
    T, k = 64, 2
    logits = draw(gen(1), T, E)
    logits[:, -1] = -10.0
    probs = torch.softmax(logits, 1)
    idx = torch.topk(probs[:, :-1], k).indices
    W = torch.ones(64, E, dtype=dt)
    W[:, -1] = 0.0
    t, out, ds = _route_alone(moe, T, E, k, dt, W=W, probs=probs, idx=idx.int(), w=probs.gather(1, idx))
    ref, mag = ds @ W.double().t(), ds.abs() @ W.double().abs().t()
    assert float((ref.abs() / mag).max()) < 1e-3
    close(out["dx"], ref, mag, E + 2, "dx")


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("E", [8, 40])
def test_route_weight_gradient_where_tokens_cancel(moe, dt, E):
    # two tokens x and -x whose ds differ by 2^-12 of themselves: one addition
    say("route dW cancels", dt, E)
    k, r = 8, gen(2)
    x = draw(r, 1, 64, dtype=dt)
    for e0 in range(0, E, k):
        dw = draw(r, 1, k)
        t, out, ds = _route_alone(moe, 2, E, k, dt, x=torch.cat([x, -x]), dw=torch.cat([dw, dw * (1 + 2.0 ** -12)]),
                                  idx=torch.arange(e0, e0 + k).repeat(2, 1).int())
        X = t["x"].double()
        ref, mag = X.t() @ ds, X.abs().t() @ ds.abs()
        close(out["dW_g"], ref, mag, 4, "dW_g")


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_route_products_of_the_largest_and_non_finite_ds(moe, dt):
    # a ds past the largest bf16 value, one that overflowed and NaN: dx is what one product in
    # fp32 gives, and no other token's changes
    say("route non-finite", dt)
    E, inf, nan = 4, float("inf"), float("nan")
    w = torch.tensor([[0.5, 0.5], [1.0, 1.0], [0.1, 0.9], [0.1, 0.9], [0.5, 0.5], [0.5, 0.5]])
    dw = torch.tensor([[1.0, 2.0], [0.0, -3.4e38], [3.4e38, -3.4e38], [-3.4e38, 3.4e38], [nan, 1.0], [3.0, 1.0]])
    T, W = w.shape[0], torch.full((64, E), 0.25, dtype=dt)
    idx = torch.tensor([[0, 1]] * T, dtype=torch.int32)
    out = moe.moe_route_backward(*cuda(draw(gen(3), T, 64, dtype=dt), W, torch.zeros(T, E), idx, w, dw))
    ds = out["dlogits"].double().cpu()
    assert ds[1, 0] > 3.39e38 and ds[2, 0] == inf and ds[3, 0] == -inf
    assert bool(torch.isnan(ds[4, :2]).all())
    want = 0.25 * ds.sum(1, keepdim=True).expand(T, 64)
    got = out["dx"].double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    over = torch.isinf(want)
    assert torch.equal(got[over], want[over])
    close(out["dx"], want, 0.25 * ds.abs().sum(1, keepdim=True).expand(T, 64), E + 2, "dx")


# ---- rows in front of the first group --------------------------------------------------
@pytest.mark.parametrize("form,c,K,N", [("nn", [3], 4104, 136), ("nt", [1, 0, 2], 8200, 72), ("nn", [0, 40, 0], 4096, 64),
                                        ("nt", [300], 2056, 136), ("nn", [70, 9], 64, 136), ("nt", [0, 130], 72, 200)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_leaves_rows_before_the_first_group(moe, form, c, K, N, dt):
    # a slice of a table of bounds with its experts' weights, into the whole table's out: rows of
    # the other groups stay, whether the sum is in parts (the long ones here) or not
    say("before", form, c, K, N, dt)
    first, last, E, g = 7, 7 + sum(c), len(c), gen(K)
    R = last + 5
    a = draw(g, R, K, dtype=dt)
    a[:first] = a[last:] = float("nan")
    b = draw(g, E, *((K, N) if form == "nn" else (N, K)), dtype=dt)
    ref, mag = matmul_ref(form, a[first:last], b, c)
    da, db, do = cuda(a, b, first + offsets_of(c))
    ws = torch.full((1 << 23,), float("nan"), device="cuda")
    for out in {dt, FP32}:
        for accumulate in (False, True) if out is FP32 else (False,):
            o = torch.full((R, N), 2.5, dtype=out, device="cuda")
            moe.moe_grouped_matmul(da, db, do, form=form, out=o, accumulate=accumulate, workspace=ws)
            close(o[first:last], ref + 2.5 * accumulate, mag + 2.5 * accumulate, K + 18)
            assert bool((o[:first] == 2.5).all()) and bool((o[last:] == 2.5).all())


def test_matmul_tn_takes_no_rows_before_the_first_group(moe):
    say("tn before")
    for c, K, N in (([40, 0, 30], 72, 136), ([5000], 72, 136)):
        first, g = 9, gen(K)
        R = first + sum(c) + 3
        a, b = draw(g, R, K, dtype=BF16), draw(g, R, N, dtype=BF16)
        ref, mag = matmul_ref("tn", a[first:], b[first:], c)
        a[:first] = float("nan")
        got = moe.moe_grouped_matmul(*cuda(a, b, first + offsets_of(c)), form="tn", out_dtype=FP32)
        close(got, ref, mag, max(c) + 18)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("f", [72, 4104])
@pytest.mark.parametrize("inplace", [False, True])
def test_swiglu_leaves_rows_before_the_first_group(moe, dt, f, inplace):
    # two slices of one table of bounds, in place: every row's gradient is taken once
    say("swiglu before", dt, f, inplace)
    R, r = 40, gen(f)
    g, u, dh = (draw(r, R, f, dtype=dt) for _ in range(3))
    w, off = torch.rand(R, generator=r), torch.tensor([0, 5, 17, 17, 33], dtype=torch.int32)
    ref, mag = swiglu_ref(g, u, dh, w)
    dg, du, ddh, dw, doff = cuda(g, u, dh, w, off)
    parts = [moe.moe_swiglu_backward(dg, du, ddh, dw, offsets=doff[e:e + 3].contiguous(), inplace=inplace) for e in (2, 0)]
    for (lo, hi), got in zip(((17, 33), (0, 17)), parts):
        for n in ref:
            close(got[n][lo:hi], ref[n][lo:hi], mag[n][lo:hi], 16 + (f if n == "dw" else 0), n)
    if inplace:
        assert torch.equal(dg[33:].cpu(), g[33:]) and torch.equal(ddh[33:].cpu(), dh[33:])


# ---- SwiGLU gradient -------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_swiglu_gate_weight_gradient_of_far_gates(moe, dt):
    # dw is fp32 for bf16 rows too. Far below 0, s is e^g: an exponent of |g| rounded in 32 bits
    # would move it by |g| 2^-24. Of each term: exp (one step: 2), the sum and the division
    # (1 each), three products, and seven additions to the row's sum
    say("swiglu far gates", dt)
    R, f, r = 512, 8, gen(1)
    g = (-20 - 64 * torch.rand(R, 1, generator=r)).expand(R, f).to(dt)
    u, dh = draw(r, R, f, dtype=dt), draw(r, R, f, dtype=dt)
    s = 1 / (1 + torch.exp(-g.double()))
    v = dh.double() * g.double() * s * u.double()
    got = moe.moe_swiglu_backward(*cuda(g.contiguous(), u, dh))
    close(got["dw"], v.sum(1), v.abs().sum(1), 2 + 1 + 1 + 3 + 7, "dw")


# ---- grouped products: tiles and addresses that larger sizes take --------------------------
@pytest.mark.parametrize("form,K,N", [("nn", 1024, 1032), ("nt", 1032, 1024)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_128_row_tiles(moe, form, K, N, dt):
    # groups of many rows with too few tiles for the 256-row ones, stored and accumulated
    say("128-row tiles", form, K, N, dt)
    c, g = [1399, 1, 700], gen(K)
    a = draw(g, sum(c), K, dtype=dt)
    b = draw(g, 3, *((K, N) if form == "nn" else (N, K)), dtype=dt)
    ref, mag = matmul_ref(form, a, b, c)
    da, db, do = cuda(a, b, offsets_of(c))
    out = moe.moe_grouped_matmul(da, db, do, form=form, out_dtype=FP32)
    close(out, ref, mag, K + 2)
    moe.moe_grouped_matmul(da, db, do, form=form, out=out, accumulate=True)
    close(out, 2 * ref, 2 * mag, K + 4)


@pytest.mark.parametrize("form", ["nn", "nt"])
def test_matmul_fp32_weights_past_the_last_level_cache(moe, form):
    say("far weights fp32", form)
    c, K, N = [(7 * i * i + i) % 9 for i in range(40)], 520, 3400
    c[39] = 0
    R, E, g = sum(c), len(c), gen(6)
    a = draw(g, R + 3, K)
    b = draw(g, E, *((K, N) if form == "nn" else (N, K)))
    ref, mag = matmul_ref(form, a[:R], b, c)
    da, db, do = cuda(a, b, offsets_of(c))
    o = torch.full((R + 3, N), 2.5, device="cuda")
    moe.moe_grouped_matmul(da, db, do, form=form, out=o)
    close(o[:R], ref, mag, K + 2)
    assert bool((o[R:] == 2.5).all())
    moe.moe_grouped_matmul(da, db, do, form=form, out=o, accumulate=True)
    close(o[:R], 2 * ref, 2 * mag, K + 4)


def test_matmul_inputs_past_2_31_elements(moe):
    # a of more than 2^31 elements without a gather, and gathered rows that lie there (TN)
    say("far a")
    K, N, few = 4096, 72, 512
    R = 2 ** 31 // K + 1000
    g = gen(14)
    rows = draw(g, few, K, dtype=BF16)
    a = torch.zeros(R, K, dtype=BF16, device="cuda")
    a[R - few:] = rows.cuda()
    b = draw(g, 2, K, N, dtype=BF16)
    ref, mag = matmul_ref("nn", rows, b[1:], [few])
    out = moe.moe_grouped_matmul(a, b.cuda(), torch.tensor([0, R - few, R], dtype=torch.int32, device="cuda"))
    close(out[R - few:], ref, mag, K + 2)
    assert not bool(out[:R - few].any())
    src = torch.arange(R - few, R).int()
    cols = draw(g, few, N, dtype=BF16)
    ref, mag = matmul_ref("tn", rows, cols, [200, few - 200])
    got = moe.moe_grouped_matmul(a, cols.cuda(), offsets_of([200, few - 200]).cuda(), form="tn", gather_a=src.cuda())
    close(got, ref, mag, few + 2)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
def test_matmul_weights_past_2_31_elements(moe, form):
    # b (TN: out) of more than 2^31 elements: the last experts' matrices
    say("far b", form)
    E, K, N, g = 33, 8192, 8200, gen(15)
    c = [0] * 30 + [3, 0, 40]
    R = sum(c)
    a = draw(g, R, K, dtype=BF16)
    if form == "tn":
        b = draw(g, R, N, dtype=BF16)
        out = moe.moe_grouped_matmul(*cuda(a, b, offsets_of(c)), form=form)
        ref, mag = matmul_ref(form, a[:, -256:], b, c[30:])
        close(out[30:, -256:], ref, mag, R + 2)
        assert not bool(out[:30].any())
        return
    b = torch.zeros(E, *((K, N) if form == "nn" else (N, K)), dtype=BF16, device="cuda")
    last = draw(g, *b.shape[1:], std=0.1, dtype=BF16)
    b[30], b[32] = last.cuda(), last.cuda()
    out = moe.moe_grouped_matmul(a.cuda(), b, offsets_of(c).cuda(), form=form)
    ref, mag = matmul_ref(form, a, last[None], [R])
    close(out, ref, mag, K + 18)


# ---- router gradient: several tiles a chunk, W_g in memory, more slots ------------------
@pytest.mark.parametrize("T,d,E,k,dt", [(2100, 128, 8, 2, BF16), (2100, 192, 40, 5, BF16), (2100, 128, 33, 3, FP32),
                                        (8300, 64, 8, 2, BF16), (8300, 64, 5, 1, FP32), (4200, 64, 64, 8, BF16),
                                        (300, 1024, 64, 4, BF16), (300, 512, 64, 8, FP32), (9, 2048, 17, 2, FP32)])
def test_route_of_many_tokens_and_wide_rows(moe, T, d, E, k, dt):
    # tokens past 2048: chunks of several tiles; past 8192: groups that come back for more;
    # W_g past 64 KB: transposed in memory for the z-loss
    say("route sizes", T, d, E, k, dt)
    for renorm, drop in ((True, 0.3), (False, 0.0)):
        lg, zg = 0.1 * T, 0.05 * T
        s = route_inputs(T, d, E, k, dt, renorm, T + E, drop)
        ref, mag = route_ref(s, k, renorm, lg, zg)
        x, W, p, idx, w, dw, b, f = cuda(*(s[n] for n in ("x", "W", "probs", "idx", "w", "dw", "b", "f")))
        out = moe.moe_route_backward(x, W, p, idx, w, dw, b_g=b, f=f, loss_grad=lg, z_loss_grad=zg,
                                     renormalize=renorm)
        for n in ref:
            close(out[n], ref[n], mag[n], {"dx": E, "dW_g": T, "db_g": T, "dlogits": 0}[n] + 16, (n, drop))
        for want in (dict(want_dx=False), dict(want_dW=False), dict(want_dx=False, want_dW=False)):
            some = moe.moe_route_backward(x, W, p, idx, w, dw, b_g=b, f=f, loss_grad=lg, z_loss_grad=zg,
                                          renormalize=renorm, **want)
            for n in ref:
                skipped = (n == "dx" and "want_dx" in want) or (n in ("dW_g", "db_g") and "want_dW" in want)
                assert some[n] is None if skipped else torch.equal(some[n], out[n]), (n, want)


@pytest.mark.parametrize("T,d,E,k", [(300, 192, 8, 3), (100, 320, 64, 4), (70, 64, 33, 5), (257, 128, 64, 8), (33, 64, 1, 1)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_route_adds_rows_of_any_number_of_slots(moe, T, d, E, k, dt):
    say("route slots", T, d, E, k, dt)
    s = route_inputs(T, d, E, k, dt, True, 5, drop=0.2)
    r = gen(6)
    order = torch.randperm(T * k, generator=r).int().view(T, k)
    pos = torch.where(s["kept"], order, torch.full_like(order, -1))
    rows = draw(r, T * k, d, dtype=dt)
    ref, mag = route_ref(s, k, True, 0.0, 0.0, rows, pos)
    s["dw"][~s["kept"]] = float("nan")
    x, W, p, idx, w, dw, dpos, drows = cuda(*(s[n] for n in ("x", "W", "probs", "idx", "w", "dw")), pos, rows)
    out = moe.moe_route_backward(x, W, p, idx, w, dw, rows=drows, pos=dpos)
    for n in ref:
        close(out[n], ref[n], mag[n], {"dx": E + k, "dW_g": T, "db_g": T, "dlogits": 0}[n] + 16, n)


@pytest.mark.parametrize("k,T", [(2, 17001), (8, 4601)])
@pytest.mark.parametrize("E", [8, 40])
def test_route_adds_rows_past_half_the_last_level_cache_of_any_number_of_slots(moe, k, T, E):
    # (dw is None: dx is the rows' sums)
    say("route many rows", k, T, E)
    d, g = 2048, torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(T * k, d, device="cuda", generator=g).to(BF16)
    pos = torch.randperm(T * k, device="cuda", generator=g).int().view(T, k)
    pos[5] = -1
    pos[6, 1] = T * k
    x, W = torch.zeros(T, d, dtype=BF16, device="cuda"), torch.zeros(d, E, dtype=BF16, device="cuda")
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(T, 1)
    out = moe.moe_route_backward(x, W, torch.full((T, E), 1 / E, device="cuda"), idx,
                                 torch.full((T, k), 1 / k, device="cuda"), None, rows=rows, pos=pos)
    some = torch.cat([torch.arange(0, 200), torch.arange(T - 300, T)])
    at = pos.cpu()[some].long()
    ok = ((at >= 0) & (at < T * k))[..., None]
    v = torch.where(ok, rows.cpu().double()[at.clamp(0, T * k - 1)], 0.0)
    close(out["dx"][some.cuda()], v.sum(1), v.abs().sum(1), k)


# ---- norms: several rows per workgroup at every width --------------------------------------
@pytest.mark.parametrize("d,T", [(256, 8209), (1024, 4099), (1032, 2051), (2048, 2051), (4096, 1027), (8192, 515), (16384, 515)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_norm_gradient_of_many_rows(moe, d, T, gate, dt):
    # more rows than workgroups, an uneven last round: column sums carried over rows
    say("norm rows", d, T, gate, dt)
    r, eps, scale = torch.Generator(device="cuda").manual_seed(d), 1e-5, 0.7
    rn = lambda *s, std=1.0, t=FP32: (torch.randn(*s, device="cuda", generator=r) * std).to(t)  # noqa: E731
    x, y, d_out, d_u = rn(T, d, t=dt), rn(T, d, std=2.0), rn(T, d, t=dt), rn(T, d, t=dt)
    gp, gm = 1 + rn(d, std=0.2), 1 + rn(d, std=0.2)
    gt = {"none": None, "channel": rn(d), "token": rn(T, 1)}[gate]
    f = moe.moe_block_norm(x, gamma=gm, y=y, gamma_post=gp, gate=gt, residual_scale=scale, eps=eps)
    res = moe.moe_block_norm_backward(f["out"], d_out=d_out, d_u=d_u, rstd=f["rstd"], gamma=gm, y=y,
                                      rstd_post=f["rstd_post"], gamma_post=gp, gate=gt, residual_scale=scale)
    q, rstd = f["rstd_post"].double()[:, None], f["rstd"].double()[:, None]
    z, dz = f["out"].double() * rstd, d_u.double() * gm.double()
    D = d_out.double() + rstd * (dz - z * (dz * z).mean(1, keepdim=True))
    Dm = d_out.double().abs() + rstd * (dz.abs() + z.abs() * (dz * z).abs().mean(1, keepdim=True))
    n = y.double() * q
    g = torch.ones(1, dtype=torch.float64, device="cuda") if gt is None else gt.double()
    dn, dnm = g * D * gp.double(), (g * gp.double()).abs() * Dm
    v, vm = D * n * gp.double(), Dm * (n * gp.double()).abs()
    want = {"dx": (scale * D, Dm, d + 12),
            "dy": (q * (dn - n * (dn * n).mean(1, keepdim=True)),
                   q * (dnm + n.abs() * (dnm * n.abs()).mean(1, keepdim=True)), 2 * d + 24),
            "dgamma": ((d_u.double() * z).sum(0), (d_u.double() * z).abs().sum(0), T + 8),
            "dgamma_post": ((g * D * n).sum(0), (g.abs() * Dm * n.abs()).sum(0), T + d + 24)}
    if gt is not None:
        dim = 0 if gate == "channel" else 1
        want["dgate"] = v.sum(dim).view(gt.shape), vm.sum(dim).view(gt.shape), T + 2 * d + 24
    for name, (ref, mag, terms) in want.items():
        close(res[name], ref.cpu(), mag.cpu(), terms, name)


# ---- outputs that the C entry points skip ----------------------------------------------
def _p(t):
    return None if t is None else t.data_ptr()


def _each_output_alone(call, shapes):
    """call(outputs) with all outputs, then with each one alone and with each one left out: the
    same bits. shapes: name -> (shape, type)."""
    def fresh(names):
        return {n: torch.full(shapes[n][0], 7.0, dtype=shapes[n][1], device="cuda") if n in names else None for n in shapes}
    full = fresh(shapes)
    call(full)
    for n in shapes:
        for names in ({n}, set(shapes) - {n}):
            got = fresh(names)
            call(got)
            for m in names:
                assert torch.equal(got[m], full[m]), (m, sorted(names))


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_swiglu_skips_outputs(moe, dt):
    say("swiglu skips", dt)
    R, f, r = 37, 264, gen(1)
    g, u, dh, w = cuda(draw(r, R, f, dtype=dt), draw(r, R, f, dtype=dt), draw(r, R, f, dtype=dt), torch.rand(R, generator=r))
    shape = TR._SWIGLU_SHAPE(R, f, 0, 0, 0, TR._TYPES[dt])

    def call(o):
        TR._call("moe_swiglu_backward", g.device, shape, _p(g), _p(u), _p(dh), _p(w), None, None, None, _p(o["dg"]),
                 _p(o["du"]), _p(o["hw"]), _p(o["dw"]))
    _each_output_alone(call, dict(dg=((R, f), dt), du=((R, f), dt), hw=((R, f), dt), dw=((R,), FP32)))


@pytest.mark.parametrize("T,d", [(70, 512), (70, 2048), (5, 4096), (9, 8200)])
@pytest.mark.parametrize("kind", [TR.GATE_NONE, TR.GATE_CHANNEL, TR.GATE_TOKEN])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_norms_skip_outputs(moe, T, d, kind, dt):
    say("norm skips", T, d, kind, dt)
    r = gen(d)
    x, d_out, d_u, y = cuda(*(draw(r, T, d, dtype=t) for t in (dt, dt, dt, FP32)))
    gp, gm = cuda(draw(r, d), draw(r, d))
    gate = {TR.GATE_NONE: None, TR.GATE_CHANNEL: draw(r, d).cuda(), TR.GATE_TOKEN: draw(r, T).cuda()}[kind]
    shape = TR._NORM_SHAPE(T, d, TR._TYPES[dt], kind, 1e-5, 0.7)
    rows, cols, tok = ((T, d), dt), ((d,), FP32), ((T,), FP32)
    keep = {}

    def forward(o):
        out, u = torch.empty_like(x), torch.empty_like(x)
        TR._call("moe_block_norm", x.device, shape, _p(x), _p(y), _p(gp), _p(gate), _p(gm), _p(out), _p(u),
                 _p(o["rstd_post"]), _p(o["rstd"]))
        for n, v in (("out", out), ("u", u)):
            assert torch.equal(keep.setdefault(n, v), v), n
    _each_output_alone(forward, dict(rstd_post=tok, rstd=tok))
    rstd, rstd_post = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    forward(dict(rstd=rstd, rstd_post=rstd_post))
    n = TR._workspace_bytes("moe_block_norm_backward_workspace_size", shape)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def backward(o):
        ws.fill_(255)
        TR._call("moe_block_norm_backward", x.device, shape, _p(d_out), _p(d_u), _p(keep["out"]), _p(rstd), _p(gm), _p(y),
                 _p(rstd_post), _p(gp), _p(gate), _p(o["dx"]), _p(o["dy"]), _p(o["dgamma"]), _p(o["dgamma_post"]),
                 _p(o.get("dgate")), _p(ws), n)
    shapes = dict(dx=rows, dy=rows, dgamma=cols, dgamma_post=cols)
    if gate is not None:
        shapes["dgate"] = cols if kind == TR.GATE_CHANNEL else tok
    _each_output_alone(backward, shapes)


@pytest.mark.parametrize("E,d", [(8, 128), (64, 1024)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_route_skips_outputs(moe, E, d, dt):
    say("route skips", E, d, dt)
    T, k = 2100, 2
    s = route_inputs(T, d, E, k, dt, True, 3)
    x, W, b, p, idx, w, dw, f = cuda(*(s[n] for n in ("x", "W", "b", "probs", "idx", "w", "dw", "f")))
    shape = TR._LAYER_SHAPE(T, d, 64, E, k, M.MOE_TOKEN_CHOICE, TR._TYPES[dt], 1, 1.0)
    up = TR._ROUTE_UPSTREAM(_p(dw), 0, 2.0, 3.0, _p(f), 0, 0, 0)
    n = TR._workspace_bytes("moe_route_backward_workspace_size", shape)
    ws, keep = torch.full((n,), 255, dtype=torch.uint8, device="cuda"), {}

    def call(o):
        ws.fill_(255)
        ds = torch.empty(T, E, device="cuda")
        TR._call("moe_route_backward", x.device, shape, _p(x), _p(W), _p(b), _p(p), _p(idx), _p(w), up, _p(o["dx"]),
                 _p(o["dW_g"]), _p(o["db_g"]), _p(ds), _p(ws), n)
        assert torch.equal(keep.setdefault("ds", ds), ds)
    _each_output_alone(call, dict(dx=((T, d), dt), dW_g=((d, E), dt), db_g=((E,), FP32)))


# ---- together: a layer's training step with either norm, and of the largest tiles --------
def _layer_ref(t, idx, kept, pre, post, gate, scale, lg, zg, eps):
    """As layer_ref, with each norm and the gate on its own; renormalised weights."""
    p = {n: v.double().requires_grad_() for n, v in t.items() if n != "d_out"}
    x, E = p["x"], p["W_g"].shape[1]
    T, k = idx.shape
    rms = lambda v: (v.square().mean(1, keepdim=True) + eps).sqrt()  # noqa: E731
    u = x / rms(x) * p["pre_gamma"] if pre else x
    logits = u @ p["W_g"] + p["b_g"]
    prob = torch.softmax(logits, 1)
    sel = prob.gather(1, idx) * kept
    w = sel / sel.sum(1, keepdim=True).clamp_min(1e-300)
    y = torch.zeros_like(x)
    for e in range(E):
        tok, slot = torch.nonzero((idx == e) & kept, as_tuple=True)
        g = u[tok] @ p["W_gate"][e]
        h = g / (1 + torch.exp(-g)) * (u[tok] @ p["W_up"][e])
        y = y.index_add(0, tok, (h @ p["W_down"][e]) * w[tok, slot][:, None])
    out = y
    if post:
        out = scale * x + y / rms(y) * p["post_gamma"] * (p["gate"] if gate else 1.0)
    f = torch.bincount(idx.reshape(-1), minlength=E).double() / T
    total = (out * t["d_out"].double()).sum() + lg * E * (f / k * prob.mean(0)).sum() \
        + zg * torch.logsumexp(logits, 1).square().mean()
    total.backward()
    names = {"pre_gamma": "d_pre_gamma", "post_gamma": "d_post_gamma", "gate": "d_gate"}
    return {names.get(n, "d" + n): v.grad for n, v in p.items() if v.grad is not None}


@pytest.mark.parametrize("pre,post,gate", [(True, False, False), (False, True, True), (False, True, False),
                                           (True, True, False)])
@pytest.mark.parametrize("T,d,f,E,dt", [(173, 128, 192, 8, BF16), (173, 128, 192, 8, FP32), (4200, 1088, 1152, 4, BF16),
                                        (8209, 128, 192, 8, BF16)])
def test_layer_backward_with_either_norm(moe, pre, post, gate, T, d, f, E, dt):
    say("layer norms", pre, post, gate, T, d, f, E, dt)
    k, eps, scale = 2, 1e-5, 0.7
    t = {n: v.cuda() for n, v in layer_inputs(T, d, f, E, dt, 22).items()}
    layer = moe.SparseMoE(t["W_g"], t["W_gate"], t["W_up"], t["W_down"], t["b_g"], k=k, mode="tc_capacity",
                          capacity_factor=0.9, pre_gamma=t["pre_gamma"] if pre else None,
                          post_gamma=t["post_gamma"] if post else None, gate=t["gate"] if gate else None,
                          residual_scale=scale, norm_eps=eps)
    lg, zg = 0.02 * T, 0.01 * T
    layer(t["x"])
    got = layer.backward(t["d_out"], loss_grad=lg, z_loss_grad=zg)
    last = layer.last
    ref = _layer_ref(t, last["idx"].long(), last["w"] != 0, pre, post, gate, scale, lg, zg, eps)
    assert set(got) == set(ref), (sorted(got), sorted(ref))
    # Of each gradient's size, in the 2-norm. bf16: at most nine values on the way are rounded (u,
    # the two products, dy, dh, the hidden gradient, the rows, the residual's gradient or u's, the
    # result), half a step of 2^-8 each. fp32: the longest chain of sums has d + f + d terms and T more.
    tol = 9 * 2.0 ** -8 if dt == BF16 else (2 * d + f + T) * 2.0 ** -24 * 8
    for n in ref:
        assert got[n].shape == ref[n].shape, n
        err = float((got[n].double() - ref[n]).norm() / ref[n].norm())
        assert err <= tol, (n, err)
