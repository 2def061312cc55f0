"""The layer norm's statistics and column sums against bounds from the kernels' real summation depths, in which a
variance by a difference of squares, a lost or doubled block of rows or a skipped value would show; on the CPU, that they would.

A row's sum: a thread adds its 8 values of each chunk, a wave its lanes by halves, the row its waves: D roundings deep,
not d. All bounds are per row, with U = 2^-24:
  a mean (a wave's, the row's) is off by at most delta = D U max|out|;
  squares around a wave's own mean add up to M2_w (1 + (D + 6) U) + n_w delta^2, and the waves are joined by
  n_w (mean_w - mean)^2, which is off by 2 |mean_w - mean| 2 delta + 4 delta^2: the variance by at most
  (D + 6) U var + 4 sqrt(var) delta + 5 delta^2 (the waves' means lie within sqrt(var), on the average of their squares);
  rstd by half of that relative to var + eps, and three roundings;
  u by |gamma| (rstd delta + |z| (rstd's relative bound + 3 U)), the sum's rounding and the result's own.
"""
from __future__ import annotations

import math

import pytest
import torch

BF16, FP32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: U}
EPS = 1e-5
WIDTHS = [8, 64, 120, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


def depth(d):
    """Roundings of a value on its way into a row's sum: chunks of 8 per thread, lanes, waves, and four more."""
    threads, chunks = next(v for most, v in ((128, (16, 1)), (256, (32, 1)), (512, (64, 1)), (1024, (64, 2)), (2048, (256, 1)),
                                             (4096, (512, 1)), (8192, (512, 2)), (16384, (1024, 2))) if d <= most)
    return 8 * chunks + int(math.log2(min(threads, 64))) + max(threads // 64, 1) + 4


def rows_of(d, dt, seed=0):
    """Rows whose statistics are hard: ordinary, far means (random, rising, in halves apart), constant, one value far out."""
    g = torch.Generator().manual_seed(seed + d)
    x = torch.randn(12, d, generator=g, dtype=torch.float64)
    x[1] = x[1] * 2 + 3
    x[2] += 100
    x[3] += 1e4
    x[4] = 1e4 + torch.arange(d) * (20 / d)
    x[5] = -1e4 + torch.arange(d).flip(0) * (20 / d)
    x[6] = 1e3 + 10 * (torch.arange(d) >= d // 2)
    x[7] = 3.0
    x[8, d // 3] = 1e4
    x[9] *= 1e-3
    x[10] = x[10] * 1e3 + 1e5
    x[11] = x[11].abs() + 7
    return x.to(dt)


def check_stats(got, x, gamma, beta, d):
    """mean, rstd and u of rows x (as they are stored), on the CPU."""
    s, D = x.double(), depth(d)
    mean = s.mean(1)
    var = ((s - mean[:, None]) ** 2).mean(1)
    r = 1 / (var + EPS).sqrt()
    delta = D * U * s.abs().amax(1)
    bad = []
    if not bool(((got["mean"].double() - mean).abs() <= delta).all()):
        bad.append("mean")
    rel = 0.5 * ((D + 6) * U * var + 4 * var.sqrt() * delta + 5 * delta ** 2) / (var + EPS) + 4 * U
    # (a variance may be off by as much as itself: then rstd lies between what the two ends give)
    low, high = r * (1 - 2 * rel).clamp(min=0), r * (1 + 2 * rel)
    if not bool(((got["rstd"].double() >= torch.where(rel < 0.05, r * (1 - 1.2 * rel), low)) &
                 (got["rstd"].double() <= torch.where(rel < 0.05, r * (1 + 1.2 * rel), high))).all()):
        bad.append("rstd")
    z = (s - mean[:, None]) * r[:, None]
    u = z * gamma.double() + beta.double()
    tol = gamma.double().abs() * (1.1 * (r * delta)[:, None] + z.abs() * (1.3 * rel + 3 * U)[:, None]) + \
        U * ((z * gamma.double()).abs() + beta.double().abs()) + HALF[got["u"].dtype] * u.abs() * (1 + 2.0 ** -7) + 1e-37
    fine = (rel < 0.05)[:, None]
    if not bool((((got["u"].double() - u).abs() <= tol) | ~fine).all()):
        bad.append("u")
    assert int(fine.sum()) >= 8  # the bounds say something
    return bad


def by(x, gamma, beta, variance):
    """Layer norm in fp32, its variance by `variance`."""
    mean = x.float().mean(1)
    r = 1 / (variance(x.float(), mean) + EPS).sqrt()
    return {"mean": mean, "rstd": r, "u": ((x.float() - mean[:, None]) * r[:, None] * gamma + beta).to(x.dtype)}


@pytest.mark.parametrize("d", [64, 1024, 2048, 8192])
def test_the_bounds_tell_variances_apart(d):
    x, g = rows_of(d, FP32), torch.Generator().manual_seed(1)
    gamma, beta = torch.randn(d, generator=g), torch.randn(d, generator=g)

    def around(v, m):
        return ((v - m[:, None]) ** 2).mean(1)

    def squares(v, m):
        return ((v * v).mean(1) - m * m).clamp(min=0)
    assert check_stats(by(x, gamma, beta, around), x, gamma, beta, d) == []
    assert "rstd" in check_stats(by(x, gamma, beta, squares), x, gamma, beta, d)
    good = by(x, gamma, beta, around)
    for k in (0.0, 0.99, 1.01, 2.0):
        assert "rstd" in check_stats({**good, "rstd": good["rstd"] * k}, x, gamma, beta, d)
    ordinary = slice(0, 2)  # one value left out of a row
    off = {n: t[ordinary] for n, t in by(torch.cat([x[:, 1:], x[:, 1:2]], 1), gamma, beta, around).items()}
    part = {n: t.clone() for n, t in good.items()}
    part["mean"][ordinary], part["rstd"][ordinary] = off["mean"], off["rstd"]
    assert {"mean", "rstd"} <= set(check_stats(part, x, gamma, beta, d))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_statistics_within_the_summation_depth(d, dt):
    import sparse_mixture_experts_sum_amd as moe
    g = torch.Generator().manual_seed(d)
    gamma, beta = torch.randn(d, generator=g), torch.randn(d, generator=g)
    for seed in range(4):
        x = rows_of(d, dt, seed)
        got = moe.moe_layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), eps=EPS)
        print("[case] statistics", d, dt, seed, flush=True)
        assert check_stats({n: got[n].cpu() for n in ("mean", "rstd", "u")}, x, gamma, beta, d) == []


# ---- column sums -------------------------------------------------------------------------
def whole_numbers(T, d, dt, seed=0):
    """out (with mean 0 and rstd 1 it is z), and d_u: small whole numbers of one sign, whose products' sums stay below
    2^24, so that every order of adding gives them exactly."""
    g = torch.Generator(device="cuda").manual_seed(seed + d)
    z = torch.randint(1, 3, (T, d), generator=g, device="cuda", dtype=torch.int8).to(dt)
    du = torch.randint(0, 2, (T, d), generator=g, device="cuda", dtype=torch.int8).to(dt)
    return z, du


def column_sums(z, du, rows=1 << 20):
    """dgamma and dbeta in 64 bits, some rows at a time."""
    rows = max(1, rows * 8 // z.shape[1])
    dg, db = torch.zeros(z.shape[1], dtype=torch.float64, device="cuda"), torch.zeros(z.shape[1], dtype=torch.float64, device="cuda")
    for i in range(0, z.shape[0], rows):
        b = du[i:i + rows].double()
        dg += (z[i:i + rows].double() * b).sum(0)
        db += b.sum(0)
    return dg, db


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("T,d", [((1 << 20) * 16 + 21, 8), (3000007, 64), (1000003, 136), (300001, 512), (100003, 1024), (50021, 2048),
                                 (20011, 4096), (9001, 8192), (5003, 16384), (513, 1024), (512, 2056), (1, 64), (4099, 1000)])
def test_column_sums_of_whole_numbers_are_exact(T, d, dt):
    import sparse_mixture_experts_sum_amd as moe
    print("[case] column sums", T, d, dt, flush=True)
    z, du = whole_numbers(T, d, dt)
    dg, db = column_sums(z, du)
    assert float(dg.max()) < 2 ** 24
    r = moe.moe_layer_norm_backward(z, du, torch.zeros(T, device="cuda"), torch.ones(T, device="cuda"), torch.ones(d, device="cuda"))
    assert torch.equal(r["dgamma"].double(), dg) and torch.equal(r["dbeta"].double(), db)


@pytest.mark.gpu
def test_column_sums_past_2_31_values_are_exact():
    import sparse_mixture_experts_sum_amd as moe
    T, d = (1 << 18) + 3, 8192
    print("[case] column sums", T, d, flush=True)
    z, du = whole_numbers(T, d, BF16)
    dg, db = column_sums(z, du)
    r = moe.moe_layer_norm_backward(z, du, torch.zeros(T, device="cuda"), torch.ones(T, device="cuda"), torch.ones(d, device="cuda"))
    assert torch.equal(r["dgamma"].double(), dg) and torch.equal(r["dbeta"].double(), db)
