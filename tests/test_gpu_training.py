"""The training operators (grouped products, SwiGLU gradient, router gradient, norms around
the layer) against their definitions in 64 bits on the CPU.

Every tolerance is the arithmetic's: half a step of the output's type (2^-8 of the value in
bf16, 2^-24 in fp32) plus, for fp32 sums of n terms in any order, (n + c) 2^-24 times the sum
of the terms' magnitudes, c counting the roundings of each term.
"""
from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: U}


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


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def offsets_of(counts):
    return torch.tensor([0] + list(counts)).cumsum(0).int()


# ---- grouped products ------------------------------------------------------------------
def matmul_ref(form, a, b, counts, ga=None, gb=None):
    """The product and the same of magnitudes, in 64 bits."""
    A = a.double() if ga is None else a.double()[ga.long()]
    outs = []
    for B, AA in ((b.double(), A), (b.double().abs(), A.abs())):
        if form == "tn" and gb is not None:
            B = B[gb.long()]
        parts, r = [], 0
        for e, n in enumerate(counts):
            rows = AA[r:r + n]
            if form == "tn":
                parts.append((rows.t() @ B[r:r + n])[None])
            else:
                parts.append(rows @ (B[e] if form == "nn" else B[e].t()))
            r += n
        outs.append(torch.cat(parts))
    return outs


COUNTS = {
    "one_row": [1],
    "one_group": [129],
    "empty_ends": [0, 5, 0, 0, 64, 65, 0],
    "ragged": [1, 63, 64, 200, 0, 257, 31, 33],
    "one_takes_all": [0, 0, 700, 0],
    "many": [(7 * i * i + i) % 23 for i in range(64)],
}


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (BF16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("K,N", [(64, 64), (8, 8), (136, 328), (520, 264)])
def test_matmul(moe, form, dt, out, counts, K, N):
    say("matmul", form, dt, out, counts, K, N)
    c = COUNTS[counts]
    R, E = sum(c), len(c)
    g = gen(R + K)
    a = draw(g, R, K, dtype=dt)
    b = draw(g, *{"nn": (E, K, N), "nt": (E, N, K), "tn": (R, N)}[form], dtype=dt)
    ref, mag = matmul_ref(form, a, b, c)
    da, db, do = cuda(a, b, offsets_of(c))
    got = moe.moe_grouped_matmul(da, db, do, form=form, out_dtype=out)
    close(got, ref, mag, (max(c) if form == "tn" else K) + 2)
    again = moe.moe_grouped_matmul(da, db, do, form=form, out_dtype=out)
    assert torch.equal(got, again)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_gathers_rows_any_number_of_times(moe, form, dt):
    say("gather", form, dt)
    c, K, N, rows = [3, 0, 130, 70], 72, 200, 41
    R, g = sum(c), gen(7)
    ga = torch.randint(0, rows, (R,), generator=g).int()
    ga[10:20] = 5
    a = draw(g, rows, K, dtype=dt)
    gb = None
    if form == "tn":
        b = draw(g, rows + 3, N, dtype=dt)
        gb = torch.randint(0, rows + 3, (R,), generator=g).int()
    else:
        b = draw(g, len(c), *((K, N) if form == "nn" else (N, K)), dtype=dt)
    ref, mag = matmul_ref(form, a, b, c, ga, gb)
    da, db, do, dga, dgb = cuda(a, b, offsets_of(c), ga, gb)
    got = moe.moe_grouped_matmul(da, db, do, form=form, gather_a=dga, gather_b=dgb, out_dtype=FP32)
    close(got, ref, mag, (max(c) if form == "tn" else K) + 2)
    # values outside the rows are taken for the nearest row
    far = dga.clone()
    far[0], far[1] = -7, 2 ** 31 - 1
    near = dga.clone()
    near[0], near[1] = 0, rows - 1
    x = moe.moe_grouped_matmul(da, db, do, form=form, gather_a=far, gather_b=dgb, out_dtype=FP32)
    y = moe.moe_grouped_matmul(da, db, do, form=form, gather_a=near, gather_b=dgb, out_dtype=FP32)
    assert torch.equal(x, y)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_accumulates(moe, form, dt):
    say("accumulate", form, dt)
    c, K, N = [0, 100, 3, 90], 128, 96
    R, g = sum(c), gen(8)
    a = draw(g, R, K, dtype=dt)
    b = draw(g, *{"nn": (4, K, N), "nt": (4, N, K), "tn": (R, N)}[form], dtype=dt)
    ref, mag = matmul_ref(form, a, b, c)
    first = draw(g, *ref.shape)
    da, db, do, out = cuda(a, b, offsets_of(c), first)
    got = moe.moe_grouped_matmul(da, db, do, form=form, out=out, accumulate=True)
    assert got is out
    close(got, ref + first.double(), mag + first.double().abs(), max(max(c), K) + 3)


@pytest.mark.parametrize("form", ["nn", "nt"])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_leaves_rows_behind_the_last_group(moe, form, dt):
    say("behind", form, dt)
    c, extra, K, N = [70, 0, 9], 60, 64, 136
    R, g = sum(c) + extra, gen(9)
    a = draw(g, R, K, dtype=dt)
    a[sum(c):] = float("nan")
    b = draw(g, 3, *((K, N) if form == "nn" else (N, K)), dtype=dt)
    ref, mag = matmul_ref(form, a[:sum(c)], b, c)
    da, db, do = cuda(a, b, offsets_of(c))
    out = torch.full((R, N), 3.5, dtype=dt, device="cuda")
    moe.moe_grouped_matmul(da, db, do, form=form, out=out)
    close(out[:sum(c)], ref, mag, K + 2)
    assert bool((out[sum(c):] == 3.5).all())


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_tn_keeps_groups_apart(moe, dt):
    # non-finite rows of one group, and behind the last one, reach no other group
    say("apart", dt)
    c, K, N = [33, 40, 1, 50, 0], 72, 64
    R, g = sum(c) + 20, gen(10)
    a, b = draw(g, R, K, dtype=dt), draw(g, R, N, dtype=dt)
    ref, mag = matmul_ref("tn", a, b, c)
    a[33:73] = float("nan")
    b[33:73] = float("inf")
    a[sum(c):] = float("nan")
    b[sum(c):] = float("inf")
    got = moe.moe_grouped_matmul(*cuda(a, b, offsets_of(c)), form="tn", out_dtype=FP32)
    keep = [0, 2, 3, 4]
    close(got[keep], ref[keep], mag[keep], 60)
    assert bool(torch.isnan(got[1]).all()) and bool((got[4] == 0).all())


@pytest.mark.parametrize("form", ["nn", "nt"])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_keeps_rows_and_columns_apart(moe, form, dt):
    # a non-finite row of a, or column of b, reaches its own row or column only, at widths
    # whose last tiles are partial
    say("rows apart", form, dt)
    c, K, N = [130, 20], 136, 72
    g = gen(11)
    a, b = draw(g, 150, K, dtype=dt), draw(g, 2, *((K, N) if form == "nn" else (N, K)), dtype=dt)
    ref, mag = matmul_ref(form, a, b, c)
    a[3] = float("inf")
    if form == "nn":
        b[1, :, 5] = float("nan")
    else:
        b[1, 5] = float("nan")
    got = moe.moe_grouped_matmul(*cuda(a, b, offsets_of(c)), form=form, out_dtype=FP32)
    fine = torch.ones(150, N, dtype=torch.bool)
    fine[3] = False
    fine[130:, 5] = False
    torch.cuda.synchronize()
    assert not bool(torch.isfinite(got.cpu()[~fine]).any())
    close(got.cpu()[fine].cuda(), ref[fine], mag[fine], K + 2)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
def test_matmul_takes_any_table_of_bounds(moe, form):
    # bounds that fall, lie below 0 or past R: each is the largest so far, within [0, R]
    say("bounds", form)
    R, K, N = 100, 64, 64
    g = gen(12)
    bad = torch.tensor([-5, 30, 10, 60, 1000, 70], dtype=torch.int32)
    good = torch.tensor([0, 30, 30, 60, 100, 100], dtype=torch.int32)
    a = draw(g, R, K, dtype=BF16)
    b = draw(g, *{"nn": (5, K, N), "nt": (5, N, K), "tn": (R, N)}[form], dtype=BF16)
    da, db, dbad, dgood = cuda(a, b, bad, good)
    x = moe.moe_grouped_matmul(da, db, dbad, form=form)
    y = moe.moe_grouped_matmul(da, db, dgood, form=form)
    assert torch.equal(x, y)


def test_matmul_without_rows(moe):
    say("no rows")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, b = torch.empty(0, 64, device="cuda"), torch.empty(3, 64, 8, device="cuda")
    assert moe.moe_grouped_matmul(a, b, off).shape == (0, 8)
    dW = moe.moe_grouped_matmul(a, torch.empty(0, 8, device="cuda"), off, form="tn")
    assert dW.shape == (3, 64, 8) and bool((dW == 0).all())
    # rows, but every group empty
    a = torch.full((5, 64), float("nan"), device="cuda")
    dW = moe.moe_grouped_matmul(a, torch.ones(5, 8, device="cuda"), off, form="tn")
    assert bool((dW == 0).all())


@pytest.mark.parametrize("form,R,E,K,N", [("nn", 2100, 3, 1024, 1032), ("nt", 2100, 3, 1032, 1024),
                                          ("tn", 2100, 3, 520, 1032), ("nn", 5, 4, 4096, 512),
                                          ("nt", 40, 2, 2056, 264), ("tn", 40, 2, 264, 2056)])
def test_matmul_larger(moe, form, R, E, K, N):
    say("larger", form, R, E, K, N)
    g = gen(R + N)
    c = [R // E + (R % E if e == 0 else 0) for e in range(E)]
    if E > 2:
        c[0], c[1] = c[0] + c[1] - 1, 1
    a = draw(g, R, K, dtype=BF16)
    b = draw(g, *{"nn": (E, K, N), "nt": (E, N, K), "tn": (R, N)}[form], dtype=BF16)
    ref, mag = matmul_ref(form, a, b, c)
    for out in (BF16, FP32):
        got = moe.moe_grouped_matmul(*cuda(a, b, offsets_of(c)), form=form, out_dtype=out)
        close(got, ref, mag, (max(c) if form == "tn" else K) + 2)


@pytest.mark.parametrize("form,c,K,N", [("tn", [5000], 72, 136), ("tn", [2100, 0, 1900], 64, 64),
                                        ("tn", [1, 4000, 33], 264, 8), ("nn", [3], 4104, 136),
                                        ("nt", [1, 0, 2], 8200, 72), ("nn", [0, 40, 0], 4096, 64)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_matmul_in_parts(moe, form, c, K, N, dt):
    # few output tiles and a long sum: the sum is taken in parts
    say("parts", form, c, K, N, dt)
    R, E, g = sum(c), len(c), gen(K)
    a = draw(g, R + 5, K, dtype=dt)
    b = draw(g, *{"nn": (E, K, N), "nt": (E, N, K), "tn": (R + 5, N)}[form], dtype=dt)
    a[R:] = float("nan")
    ref, mag = matmul_ref(form, a[:R], b[:R] if form == "tn" else b, c)
    da, db, do = cuda(a, b, offsets_of(c))
    for out in {dt, FP32}:
        o = torch.full((E, K, N) if form == "tn" else (R + 5, N), 2.5, dtype=out, device="cuda")
        moe.moe_grouped_matmul(da, db, do, form=form, out=o)
        close(o if form == "tn" else o[:R], ref, mag, (max(c) if form == "tn" else K) + 18)
        if form != "tn":
            assert bool((o[R:] == 2.5).all())
    acc = torch.full((E, K, N) if form == "tn" else (R + 5, N), 2.5, device="cuda")
    moe.moe_grouped_matmul(da, db, do, form=form, out=acc, accumulate=True)
    close(acc if form == "tn" else acc[:R], ref + 2.5, mag + 2.5, (max(c) if form == "tn" else K) + 18)


@pytest.mark.parametrize("c,K,N", [([3, 2500, 0, 70, 1], 136, 264), ([30000], 64, 64), ([800, 0, 5100, 769, 768], 72, 128),
                                   ([20, 60, 4000, 0, 33, 5, 1, 1500], 520, 1032)])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (BF16, FP32), (FP32, FP32)])
def test_matmul_tn_groups_in_parts_beside_whole_ones(moe, c, K, N, dt, out):
    # a long group's sum is taken in parts (32 at most), its neighbours' are not
    say("tn parts", c, K, N, dt, out)
    R, E, g = sum(c), len(c), gen(K)
    a, b = draw(g, 501, K, dtype=dt), draw(g, R + 5, N, dtype=dt)
    b[R:] = float("nan")
    ga = torch.randint(0, 501, (R + 5,), generator=g).int()
    gb = torch.arange(R + 5).int()
    ref, mag = matmul_ref("tn", a, b[:R], c, ga[:R], None)
    da, db, do, dga, dgb = cuda(a, b, offsets_of(c), ga, gb)
    terms = max(c) + 34
    got = moe.moe_grouped_matmul(da, db, do, form="tn", gather_a=dga, gather_b=dgb, out_dtype=out)
    close(got, ref, mag, terms)
    ws = torch.full((1 << 26,), float("nan"), device="cuda")
    again = moe.moe_grouped_matmul(da, db, do, form="tn", gather_a=dga, out_dtype=out, workspace=ws)
    assert torch.equal(got, again)
    if out is FP32:
        acc = torch.full((E, K, N), 2.5, device="cuda")
        moe.moe_grouped_matmul(da, db, do, form="tn", gather_a=dga, out=acc, accumulate=True)
        close(acc, ref + 2.5, mag + 2.5, terms + 2)
    # a table that is no table: bounds are taken as the running maximum, at most R
    bad = do.clone()
    bad[0], bad[-1] = -5, 2 ** 31 - 1
    if E > 3:
        bad[2] = 0
    good = torch.cummax(bad.cpu().clamp(0, R + 5), 0).values.cuda()
    x = moe.moe_grouped_matmul(da, db, bad, form="tn", gather_a=dga, out_dtype=out)
    y = moe.moe_grouped_matmul(da, db, good, form="tn", gather_a=dga, out_dtype=out)
    assert torch.equal(x.view(torch.int16 if out is BF16 else torch.int32),
                       y.view(torch.int16 if out is BF16 else torch.int32))


@pytest.mark.parametrize("form,c,K,N", [("nn", [1, 700, 0, 799], 1032, 5640), ("nt", [257, 1, 1242], 1160, 5512),
                                        ("tn", [33, 0, 300], 1000, 2832), ("tn", [1, 97, 64], 1288, 2056),
                                        ("tn", [0, 70, 130], 2312, 2568), ("tn", [150], 2568, 4360)])
@pytest.mark.parametrize("gathered", [False, True])
def test_matmul_many_tiles(moe, form, c, K, N, gathered):
    # more tiles than are resident at once: the largest tiles, several of them per workgroup
    say("many tiles", form, c, K, N, gathered)
    R, E, g = sum(c), len(c), gen(N)
    rows = 501 if gathered else R + 5
    a = draw(g, rows, K, dtype=BF16)
    ga = torch.randint(0, rows, (R,), generator=g).int() if gathered else None
    gb = None
    if form == "tn":
        b = draw(g, rows, N, dtype=BF16)
        gb = torch.randint(0, rows, (R,), generator=g).int() if gathered else None
    else:
        b = draw(g, E, *((K, N) if form == "nn" else (N, K)), dtype=BF16)
    if not gathered:
        a[R:] = float("nan")
    ref, mag = matmul_ref(form, a if gathered else a[:R], b if gathered or form != "tn" else b[:R], c, ga, gb)
    da, db, do, dga, dgb = cuda(a, b, offsets_of(c), ga, gb)
    terms = max(c) if form == "tn" else K
    for out in (BF16, FP32):
        o = torch.full((E, K, N) if form == "tn" else (R if gathered else R + 5, N), 2.5, dtype=out, device="cuda")
        moe.moe_grouped_matmul(da, db, do, form=form, gather_a=dga, gather_b=dgb, out=o)
        close(o if form == "tn" else o[:R], ref, mag, terms + 2)
        if form != "tn":
            assert bool((o[R:] == 2.5).all())
    moe.moe_grouped_matmul(da, db, do, form=form, gather_a=dga, gather_b=dgb, out=o, accumulate=True)
    close(o if form == "tn" else o[:R], 2 * ref, 2 * mag, terms + 4)


@pytest.mark.parametrize("form", ["nn", "nt"])
def test_matmul_weights_past_the_last_level_cache(moe, form):
    # few rows a group, weights of more than 256 MB
    c, K, N = [(7 * i * i + i) % 9 for i in range(40)], 1032, 3400
    c[3], c[39] = 45, 0
    R, E, g = sum(c), len(c), gen(5)
    say("far weights", form, R)
    a = draw(g, 77, K, dtype=BF16)
    b = torch.randn(E, *((K, N) if form == "nn" else (N, K)), dtype=BF16, generator=g)
    ga = torch.randint(0, 77, (R + 3,), generator=g).int()
    ref, mag = matmul_ref(form, a, b, c, ga[:R])
    da, db, do, dga = cuda(a, b, offsets_of(c), ga)
    for out in (BF16, FP32):
        o = torch.full((R + 3, N), 2.5, dtype=out, device="cuda")
        moe.moe_grouped_matmul(da, db, do, form=form, gather_a=dga, out=o)
        close(o[:R], ref, mag, K + 2)
        assert bool((o[R:] == 2.5).all())
    moe.moe_grouped_matmul(da, db, do, form=form, gather_a=dga, out=o, accumulate=True)
    close(o[:R], 2 * ref, 2 * mag, K + 4)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_matmul_captured_with_other_groups_at_each_replay(moe, form, accumulate):
    # the bounds are read when the graph runs: long and empty groups, whole sums and parts
    say("captured", form, accumulate)
    R, E, K, N = 3000, 4, 264, 136
    g = gen(21)
    a, b = draw(g, R, K, dtype=BF16), draw(g, *{"nn": (E, K, N), "nt": (E, N, K), "tn": (R, N)}[form], dtype=BF16)
    tables = [[0, 0, 3000, 0], [700, 800, 750, 750], [2990, 1, 0, 9], [0, 0, 0, 0], [1, 2, 3, 2000]]
    da, db, do = cuda(a, b, offsets_of(tables[1]))
    shape = (E, K, N) if form == "tn" else (R, N)
    out = torch.zeros(shape, device="cuda")
    moe.moe_grouped_matmul(da, db, do, form=form, out=out, accumulate=accumulate)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_grouped_matmul(da, db, do, form=form, out=out, accumulate=accumulate)
    for c in tables:
        do.copy_(offsets_of(c))
        out.fill_(1.5)
        want = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        moe.moe_grouped_matmul(da, db, do, form=form, out=want, accumulate=accumulate)
        assert torch.equal(out, want), c
        last = sum(c)
        rows = slice(None) if form == "tn" else slice(0, last)
        ref, mag = matmul_ref(form, a[:last], b[:last] if form == "tn" else b, c)
        close(out[rows], ref + 1.5 * accumulate, mag + 1.5 * accumulate, (max(c) if form == "tn" else K) + 34, c)
        if form != "tn":
            assert bool((out[last:] == 1.5).all())


def test_matmul_rows_past_2_31_elements(moe):
    # a and out of more than 2^31 elements: the last rows against the first ones' copies
    say("far rows")
    K, N, R = 2048, 1032, (2 ** 31) // 1032 + 4096
    g = gen(13)
    few = draw(g, 256, K, dtype=BF16).cuda()
    src = torch.arange(R, dtype=torch.int32, device="cuda") % 256
    b = draw(g, 2, K, N, std=0.1, dtype=BF16).cuda()
    off = torch.tensor([0, 1000, R], dtype=torch.int32, device="cuda")
    out = moe.moe_grouped_matmul(few, b, off, gather_a=src)
    ref, mag = matmul_ref("nn", few.cpu(), b[1:].cpu(), [256])
    last = out[-300:]
    want = src[-300:].long().cpu()
    close(last, ref[want], mag[want], K + 2)


# ---- SwiGLU gradient -------------------------------------------------------------------
def swiglu_ref(g, u, dh, w):
    g, u, dh, w = g.double(), u.double(), dh.double(), w.double()[:, None]
    s = 1 / (1 + torch.exp(-g))
    ref = {"dg": w * dh * u * s * (1 + g * (1 - s)), "du": w * dh * g * s, "h": w * g * s * u,
           "dw": (dh * g * s * u).sum(1)}
    # the exponent's rounding moves s by |g| 2^-24 of itself and more; 1 - s loses no more
    # than 2^-24 of 1 in absolute terms
    slope = 1 + g.abs()
    mag = {"dg": (w * dh * u).abs() * s * slope * (1 + g.abs()), "du": (w * dh * g).abs() * s * slope,
           "h": (w * g * u).abs() * s * slope, "dw": ((dh * g * u).abs() * s * slope).sum(1)}
    return ref, mag


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("R,f", [(1, 8), (37, 1408), (5, 2048), (130, 72), (9, 2056), (3, 14336)])
def test_swiglu(moe, dt, R, f):
    say("swiglu", dt, R, f)
    r = gen(R + f)
    g, u, dh = draw(r, R, f, std=3.0, dtype=dt), draw(r, R, f, dtype=dt), draw(r, R, f, dtype=dt)
    w = torch.rand(R, generator=r)
    g[0, :4] = torch.tensor([200.0, -200.0, 0.0, -30.0]).to(dt)
    ref, mag = swiglu_ref(g, u, dh, w)
    out = moe.moe_swiglu_backward(*cuda(g, u, dh, w))
    for n in ref:
        close(out[n], ref[n], mag[n], 16 + (f if n == "dw" else 0), n)
    # against differences of the definition, in 64 bits
    def h(gg):
        return (w.double()[:, None] * gg / (1 + torch.exp(-gg)) * u.double() * dh.double())
    step = 1e-4
    num = (h(g.double() + step) - h(g.double() - step)) / (2 * step)
    assert float((ref["dg"] - num).abs().max()) < 1e-5 * float(1 + num.abs().max())
    # in place: the same bits
    dev = cuda(g, u, dh, w)
    same = moe.moe_swiglu_backward(*dev, inplace=True)
    assert same["dg"] is dev[0] and same["h"] is dev[2]
    for n in ref:
        assert torch.equal(same[n], out[n]), n


def test_swiglu_weights_by_slot_and_rows_behind(moe):
    say("swiglu slots")
    T, k, f, r = 50, 3, 264, gen(3)
    slots = torch.randperm(T * k, generator=r)
    pos = torch.full((T, k), -1, dtype=torch.int32)
    used = T * k - 20  # 20 dropped slots; two more rows that no slot names
    src = torch.zeros(T * k, dtype=torch.int32)
    for row, slot in enumerate(slots[:used].tolist()):
        pos[slot // k, slot % k] = row
        src[row] = slot // k
    last = used + 2
    off = torch.tensor([0, 40, last], dtype=torch.int32)
    w = torch.rand(T, k, generator=r)
    g, u, dh = (draw(r, T * k, f, dtype=BF16) for _ in range(3))
    w_row = torch.zeros(T * k)
    w_row[:used] = w.reshape(-1)[slots[:used]]
    ref, mag = swiglu_ref(g, u, dh, w_row)
    dg, du, ddh, dw, dsrc, dpos, doff = cuda(g, u, dh, w, src, pos, off)
    out = moe.moe_swiglu_backward(dg, du, ddh, dw, src=dsrc, pos=dpos)
    for n in ref:
        close(out[n], ref[n], mag[n], 16 + (f if n == "dw" else 0), n)
    keep = dg.clone()
    out = moe.moe_swiglu_backward(dg, du, ddh, dw, src=dsrc, pos=dpos, offsets=doff, inplace=True)
    close(out["dg"][:last], ref["dg"][:last], mag["dg"][:last], 16)
    assert torch.equal(dg[last:], keep[last:])


def test_swiglu_in_place_of_one_tensor_is_refused(moe):
    g, dh = torch.ones(3, 8, device="cuda"), torch.ones(3, 8, device="cuda")
    with pytest.raises(ValueError, match="three tensors"):
        moe.moe_swiglu_backward(g, g, dh, inplace=True)
    assert bool((g == 1).all())


def test_swiglu_without_rows_or_weights(moe):
    say("swiglu none")
    e = torch.empty(0, 64, device="cuda")
    assert moe.moe_swiglu_backward(e, e, e)["dw"].shape == (0,)
    r = gen(4)
    g, u, dh = (draw(r, 6, 64, dtype=FP32) for _ in range(3))
    ref, mag = swiglu_ref(g, u, dh, torch.ones(6))
    out = moe.moe_swiglu_backward(*cuda(g, u, dh))
    for n in ref:
        close(out[n], ref[n], mag[n], 16 + (64 if n == "dw" else 0), n)


# ---- router gradient -------------------------------------------------------------------
def route_inputs(T, d, E, k, dt, renorm, seed, drop=0.0):
    r = gen(seed)
    x, W, b = draw(r, T, d, dtype=dt), draw(r, d, E, std=0.05, dtype=dt), draw(r, E, std=0.5)
    p = torch.softmax(x.double() @ W.double() + b.double(), 1)
    top = torch.topk(p, k)
    kept = torch.rand(T, k, generator=r) >= drop
    v = top.values * kept
    w = v / v.sum(1, keepdim=True).clamp_min(1e-300) if renorm else v
    f = torch.bincount(top.indices.reshape(-1), minlength=E).double() / max(T, 1)
    return dict(x=x, W=W, b=b, probs=p.float(), idx=top.indices.int(), w=w.float(), f=f.float(),
                kept=kept, dw=draw(r, T, k))


def route_ref(s, k, renorm, lg, zg, rows=None, pos=None):
    """Autograd of the definition in 64 bits, and magnitudes for the tolerances."""
    x, W, b = (s[n].double().requires_grad_() for n in ("x", "W", "b"))
    T, E = s["probs"].shape
    logits = x @ W + b
    logits.retain_grad()
    p = torch.softmax(logits, 1)
    sel = p.gather(1, s["idx"].long()) * s["kept"]
    w = sel / sel.sum(1, keepdim=True).clamp_min(1e-300) if renorm else sel
    dw = torch.where(s["kept"], s["dw"].double(), torch.zeros((), dtype=torch.float64))
    total = (w * dw).sum()
    if T:
        total = total + lg * E * (s["f"].double() / k * p.mean(0)).sum() \
            + zg * torch.logsumexp(logits, 1).square().mean()
    total.backward()
    ds = logits.grad
    lse = torch.logsumexp(logits.detach(), 1, keepdim=True)
    S = sel.detach().sum(1, keepdim=True)
    big = (dw.abs().max(1, keepdim=True).values + (dw * w.detach()).abs().sum(1, keepdim=True)) \
        / (S.clamp_min(1e-30) if renorm else 1) + abs(lg) * E / (k * max(T, 1)) * s["f"].double().max()
    # the z-loss term: s is a dot product of d terms, log p a rounding of p
    dot = x.detach().abs() @ W.detach().abs()
    zmag = abs(zg) * 2 / max(T, 1) * (lse.abs() + (x.shape[1] / 16) * dot.max(1, keepdim=True).values + 8)
    mag = p.detach() * (big * (E / 4 + 4) + zmag)
    dx, dxm = x.grad, mag @ W.detach().t().abs()
    if rows is not None:
        for j in range(k):
            ok = (pos[:, j] >= 0)[:, None]
            v = torch.where(ok, rows.double()[pos[:, j].clamp_min(0).long()], 0.0)
            dx, dxm = dx + v, dxm + v.abs()
    return ({"dx": dx, "dW_g": W.grad, "db_g": b.grad, "dlogits": ds},
            {"dx": dxm, "dW_g": x.detach().abs().t() @ mag, "db_g": mag.sum(0), "dlogits": mag})


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("T,d,E,k", [(1, 64, 1, 1), (3, 64, 5, 2), (100, 128, 8, 2), (257, 192, 64, 8),
                                     (1000, 256, 33, 3), (64, 1024, 16, 4)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(moe, dt, T, d, E, k, renorm):
    say("route", dt, T, d, E, k, renorm)
    for drop, lg, zg in ((0.0, 0.0, 0.0), (0.0, 0.3 * T, 0.0), (0.3, 0.1 * T, 0.05 * T), (1.0, 0.0, 0.0)):
        s = route_inputs(T, d, E, k, dt, renorm, T + E, drop)
        # what a dropped slot's gradient holds is not looked at
        s["dw"][~s["kept"]] = float("nan")
        ref, mag = route_ref(s, k, renorm, lg, zg)
        x, W, p, idx, w, dw, b, f = cuda(*(s[n] for n in ("x", "W", "probs", "idx", "w", "dw", "b", "f")))
        out = moe.moe_route_backward(x, W, p, idx, w, dw, b_g=b, f=f, loss_grad=lg, z_loss_grad=zg,
                                     renormalize=renorm)
        for n in ref:
            terms = {"dx": E, "dW_g": T, "db_g": T, "dlogits": 0}[n] + 16
            close(out[n], ref[n], mag[n], terms, (n, drop))
        again = moe.moe_route_backward(x, W, p, idx, w, dw, b_g=b, f=f, loss_grad=lg, z_loss_grad=zg,
                                       renormalize=renorm)
        for n in ref:
            assert torch.equal(out[n], again[n]), n


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_route_adds_rows_and_takes_dw_by_row(moe, dt):
    say("route rows", dt)
    T, d, E, k = 300, 128, 8, 2
    s = route_inputs(T, d, E, k, dt, True, 5, drop=0.2)
    r = gen(6)
    order = torch.randperm(T * k, generator=r).int().view(T, k)
    pos = torch.where(s["kept"], order, torch.full_like(order, -1))
    rows = draw(r, T * k, d, dtype=dt)
    ref, mag = route_ref(s, k, True, 0.0, 0.0, rows, pos)
    dw_row = torch.full((T * k,), float("nan"))
    dw_row[pos[s["kept"]].long()] = s["dw"][s["kept"]]
    x, W, p, idx, w, dpos, drows, ddw = cuda(s["x"], s["W"], s["probs"], s["idx"], s["w"], pos, rows, dw_row)
    out = moe.moe_route_backward(x, W, p, idx, w, ddw, rows=drows, pos=dpos)
    for n in ref:
        close(out[n], ref[n], mag[n], {"dx": E + k, "dW_g": T, "db_g": T, "dlogits": 0}[n] + 16, n)
    # rows alone: every gradient of the router's is zero
    out = moe.moe_route_backward(x, W, p, idx, w, None, rows=drows, pos=dpos)
    assert not bool(out["dlogits"].any()) and not bool(out["dW_g"].any())


@pytest.mark.parametrize("dt", [BF16, FP32])
def test_route_adds_rows_past_half_the_last_level_cache(moe, dt):
    # (only dx's sums of rows: dw is None, so every other gradient is zero)
    T, d, E, k = 9001, 2048, 8, 4
    say("route many rows", dt)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(T * k, d, device="cuda", generator=g).to(dt)
    pos = torch.randperm(T * k, device="cuda", generator=g).int().view(T, k)
    pos[5] = -1
    pos[6, 1] = T * k
    x, W = torch.zeros(T, d, dtype=dt, device="cuda"), torch.zeros(d, E, dtype=dt, device="cuda")
    p = torch.full((T, E), 1 / E, device="cuda")
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(T, 1)
    out = moe.moe_route_backward(x, W, p, idx, torch.full((T, k), 1 / k, device="cuda"), None, rows=rows, pos=pos)
    some = torch.cat([torch.arange(0, 200), torch.arange(T - 300, T)])
    at = pos.cpu()[some].long()
    ok = ((at >= 0) & (at < T * k))[..., None]
    v = torch.where(ok, rows.cpu().double()[at.clamp(0, T * k - 1)], 0.0)
    close(out["dx"][some.cuda()], v.sum(1), v.abs().sum(1), k)


def test_route_with_kept_slots_of_the_smallest_probabilities(moe):
    # the likely experts' slots were dropped by the capacity: S of the kept ones is a
    # denormal number, their weights are not. ds is w_j (dw_j - sum_i dw_i w_i) there, and
    # at most 1e-38 elsewhere
    say("route small S")
    T, d, E, k = 5, 64, 8, 3
    p = torch.zeros(T, E)
    p[:, 0] = 1.0
    p[:, 3], p[:, 5] = 1e-40, 3e-40
    idx = torch.tensor([[0, 5, 3]] * T, dtype=torch.int32)
    w = torch.tensor([[0.0, 0.75, 0.25]] * T)
    dw = draw(gen(3), T, k)
    x, W = draw(gen(4), T, d), draw(gen(5), d, E)
    out = moe.moe_route_backward(*cuda(x, W, p, idx, w, dw))
    g, wd = dw.double(), w.double()
    mean = (g * wd).sum(1, keepdim=True)
    ref, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    ref.scatter_(1, idx.long(), wd * (g - mean))
    mag.scatter_(1, idx.long(), wd * (g.abs() + (g.abs() * wd).sum(1, keepdim=True)))
    close(out["dlogits"], ref, mag, 4, "dlogits")  # (two products, their sum, a difference)


def test_route_without_tokens(moe):
    say("route none")
    z = lambda *s, dtype=FP32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    out = moe.moe_route_backward(z(0, 64), z(64, 8), z(0, 8), z(0, 2, dtype=torch.int32), z(0, 2), z(0, 2))
    assert out["dx"].shape == (0, 64) and not bool(out["dW_g"].any()) and not bool(out["db_g"].any())


def test_route_against_the_forward(moe):
    # its own forward's outputs, with a capacity that drops slots, against differences of
    # the forward's loss, z-loss and weights as 64-bit functions
    say("route forward")
    T, d, E, k = 200, 64, 8, 2
    r = gen(9)
    x, W, b = draw(r, T, d), draw(r, d, E, std=0.1), draw(r, E, std=0.5)
    dx_, dW_, db_ = cuda(x, W, b)
    fwd = moe.moe_route(dx_, dW_, db_, k=k, mode="tc_capacity", capacity_factor=0.8)
    w, idx = fwd["w"].cpu(), fwd["idx"].cpu()
    assert bool((w == 0).any())
    s = dict(x=x, W=W, b=b, probs=fwd["probs"].cpu(), idx=idx, w=w, kept=w != 0, dw=draw(r, T, k),
             f=fwd["counts"].cpu().float() / T)
    ref, mag = route_ref(s, k, True, 0.02 * T, 0.01 * T)
    out = moe.moe_route_backward(dx_, dW_, fwd["probs"], fwd["idx"], fwd["w"], s["dw"].cuda(), b_g=db_,
                                 f=s["f"].cuda(), loss_grad=0.02 * T, z_loss_grad=0.01 * T)
    for n in ref:
        # the forward's probabilities are fp32: d fp32 roundings in the logits reach p
        close(out[n], ref[n], mag[n], {"dx": E, "dW_g": T, "db_g": T, "dlogits": 0}[n] + 16 + d, n)


# ---- norms -----------------------------------------------------------------------------
def norm_ref(x, y, gp, gate, gamma, scale, eps, dt):
    out, r = x.double(), {}
    if y is not None:
        q = 1 / ((y.double() ** 2).mean(1, keepdim=True) + eps).sqrt()
        n = y.double() * q * gp.double() * (1 if gate is None else gate.double())
        r["rstd_post"] = (q[:, 0], q[:, 0])
        out = scale * out + n
        r["out"] = (out, (scale * x.double()).abs() + n.abs())
    return r, out


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("T,d", [(1, 8), (5, 72), (67, 512), (8, 520), (33, 2048), (3, 4096), (9, 4104),
                                 (2, 8200), (2, 16384)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm(moe, dt, T, d, gate):
    say("norm", dt, T, d, gate)
    r, eps, scale = gen(T + d), 1e-5, 0.7
    x, y = draw(r, T, d, dtype=dt), draw(r, T, d, std=2.0)
    gp, gm = 1 + draw(r, d, std=0.2), 1 + draw(r, d, std=0.2)
    gt = {"none": None, "channel": draw(r, d), "token": draw(r, T, 1)}[gate]
    dx_, dy_, dgp, dgm, dgt = cuda(x, y, gp, gm, gt)
    got = moe.moe_block_norm(dx_, gamma=dgm, y=dy_, gamma_post=dgp, gate=dgt, residual_scale=scale, eps=eps)
    ref, _ = norm_ref(x, y, gp, gt, gm, scale, eps, dt)
    for n in ref:
        close(got[n], ref[n][0], ref[n][1], d + 12, n)
    # the next norm reads the stored sum
    o = got["out"].double().cpu()
    rs = 1 / ((o ** 2).mean(1, keepdim=True) + eps).sqrt()
    close(got["rstd"], rs[:, 0], rs[:, 0], d + 4, "rstd")
    close(got["u"], o * rs * gm.double(), (o * rs * gm.double()).abs(), d + 8, "u")
    # each part alone gives the same bits
    after = moe.moe_block_norm(dx_, y=dy_, gamma_post=dgp, gate=dgt, residual_scale=scale, eps=eps)
    before = moe.moe_block_norm(after["out"], gamma=dgm, eps=eps)
    assert torch.equal(after["out"], got["out"]) and torch.equal(before["u"], got["u"])
    assert after["u"] is None and before["out"] is after["out"]

    # gradient, both parts and each alone
    d_out, d_u = draw(r, T, d, dtype=dt), draw(r, T, d, dtype=dt)
    q, rstd = got["rstd_post"].double().cpu()[:, None], got["rstd"].double().cpu()[:, None]
    for use_out, use_u, use_y in ((1, 1, 1), (1, 0, 1), (0, 1, 1), (0, 1, 0), (1, 1, 0)):
        kw = dict(d_out=d_out.cuda() if use_out else None, d_u=d_u.cuda() if use_u else None,
                  residual_scale=scale if use_y else 1.0)
        if use_u:
            kw.update(rstd=got["rstd"], gamma=dgm)
        if use_y:
            kw.update(y=dy_, rstd_post=got["rstd_post"], gamma_post=dgp, gate=dgt)
        res = moe.moe_block_norm_backward(got["out"], **kw)
        D = d_out.double() if use_out else torch.zeros(T, d, dtype=torch.float64)
        Dm = D.abs()
        if use_u:
            z, dz = o * rstd, d_u.double() * gm.double()
            mean, meanm = (dz * z).mean(1, keepdim=True), (dz * z).abs().mean(1, keepdim=True)
            D = D + rstd * (dz - z * mean)
            Dm = Dm + rstd * (dz.abs() + z.abs() * meanm)
            close(res["dgamma"], (d_u.double() * z).sum(0), (d_u.double() * z).abs().sum(0), T + 8, "dgamma")
        else:
            assert res["dgamma"] is None
        sc = scale if use_y else 1.0
        close(res["dx"], sc * D, Dm, d + 12, "dx")
        if not use_y:
            assert res["dy"] is None and res["dgate"] is None
            continue
        n = y.double() * q
        g = torch.ones(1, dtype=torch.float64) if gt is None else gt.double()
        dn, dnm = g * D * gp.double(), (g * gp.double()).abs() * Dm
        dy = q * (dn - n * (dn * n).mean(1, keepdim=True))
        dym = q * (dnm + n.abs() * (dnm * n.abs()).mean(1, keepdim=True))
        close(res["dy"], dy, dym, 2 * d + 24, "dy")
        close(res["dgamma_post"], (g * D * n).sum(0), (g.abs() * Dm * n.abs()).sum(0), T + d + 24, "dgamma_post")
        if gt is None:
            assert res["dgate"] is None
        else:
            v, vm = D * n * gp.double(), Dm * (n * gp.double()).abs()
            dim = 0 if gate == "channel" else 1
            want, wm = v.sum(dim), vm.sum(dim)
            close(res["dgate"].reshape(-1), want, wm, T + 2 * d + 24, "dgate")
            assert res["dgate"].shape == gt.shape


def test_norm_gradient_against_differences(moe):
    say("norm differences")
    T, d, r, eps = 3, 16, gen(1), 1e-3
    x, y, gp, gm, gate = (draw(r, *s).double() for s in ((T, d), (T, d), (d,), (d,), (d,)))
    d_out, d_u = draw(r, T, d).double(), draw(r, T, d).double()

    def loss(x, y, gp, gm, gate):
        out = 0.5 * x + gate * (y / ((y ** 2).mean(1, keepdim=True) + eps).sqrt() * gp)
        u = out / ((out ** 2).mean(1, keepdim=True) + eps).sqrt() * gm
        return ((out * d_out).sum() + (u * d_u).sum()).item()

    args = [x, y, gp, gm, gate]
    dx_, dy_, dgp, dgm, dgt = cuda(*(a.float() for a in args))
    fwd = moe.moe_block_norm(dx_, gamma=dgm, y=dy_, gamma_post=dgp, gate=dgt, residual_scale=0.5, eps=eps)
    got = moe.moe_block_norm_backward(fwd["out"], d_out=d_out.float().cuda(), d_u=d_u.float().cuda(),
                                      rstd=fwd["rstd"], gamma=dgm, y=dy_, rstd_post=fwd["rstd_post"],
                                      gamma_post=dgp, gate=dgt, residual_scale=0.5)
    for i, n in enumerate(("dx", "dy", "dgamma_post", "dgamma", "dgate")):
        num = torch.zeros_like(args[i]).reshape(-1)
        for j in range(num.numel()):
            for sign in (1, -1):
                moved = [a.clone() for a in args]
                moved[i].reshape(-1)[j] += sign * 1e-5
                num[j] += sign * loss(*moved) / 2e-5
        # fp32 inputs and sums against differences good to about 1e-9
        err = (got[n].double().cpu().reshape(-1) - num).abs().max() / num.abs().max()
        assert float(err) < 2e-5, n


def test_norm_zero_row_and_no_rows(moe):
    say("norm zero rows")
    d = 128
    x = torch.zeros(3, d, dtype=BF16, device="cuda")
    gm = torch.ones(d, device="cuda")
    got = moe.moe_block_norm(x, gamma=gm, eps=1e-6)
    assert not bool(got["u"].any()) and bool(torch.isfinite(got["rstd"]).all())
    e = torch.empty(0, d, dtype=BF16, device="cuda")
    got = moe.moe_block_norm(e, gamma=gm)
    assert got["u"].shape == (0, d)
    res = moe.moe_block_norm_backward(e, d_u=e, rstd=got["rstd"], gamma=gm)
    assert res["dx"].shape == (0, d) and not bool(res["dgamma"].any())


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norms_after_a_block_without_rows(moe, gate):
    say("norm no rows", gate)
    d = 128
    x, y = torch.empty(0, d, dtype=BF16, device="cuda"), torch.empty(0, d, device="cuda")
    gm = torch.ones(d, device="cuda")
    gt = {"none": None, "channel": gm, "token": torch.empty(0, 1, device="cuda")}[gate]
    got = moe.moe_block_norm(x, gamma=gm, y=y, gamma_post=gm, gate=gt)
    assert got["out"].shape == got["u"].shape == (0, d)
    res = moe.moe_block_norm_backward(got["out"], d_out=x, d_u=x, rstd=got["rstd"], gamma=gm, y=y,
                                      rstd_post=got["rstd_post"], gamma_post=gm, gate=gt)
    assert res["dx"].shape == res["dy"].shape == (0, d)
    assert not bool(res["dgamma"].any()) and not bool(res["dgamma_post"].any())
    if gate == "channel":
        assert not bool(res["dgate"].any())


def test_layer_block_without_tokens(moe):
    say("layer block none")
    t = {n: v.cuda() for n, v in layer_inputs(0, 64, 64, 4, BF16, 3).items()}
    ones = torch.ones(64, device="cuda")
    layer = moe.SparseMoE(t["W_g"], t["W_gate"], t["W_up"], t["W_down"], pre_gamma=ones, post_gamma=ones, gate=ones)
    assert layer(t["x"]).shape == (0, 64)
    got = layer.backward(t["d_out"].to(BF16))
    assert got["dx"].shape == (0, 64) and not any(bool(got[n].any()) for n in got if n != "dx")


def test_norm_many_rows(moe):
    # more rows than workgroups, an odd count: every row once, columns summed over all
    say("norm many rows")
    T, d, r = 5003, 256, gen(2)
    x, du = draw(r, T, d, dtype=BF16), draw(r, T, d, dtype=BF16)
    gm = 1 + draw(r, d, std=0.1)
    dx_, ddu, dgm = cuda(x, du, gm)
    f = moe.moe_block_norm(dx_, gamma=dgm)
    got = moe.moe_block_norm_backward(dx_, d_u=ddu, rstd=f["rstd"], gamma=dgm)
    z = x.double() * f["rstd"].double().cpu()[:, None]
    close(got["dgamma"], (du.double() * z).sum(0), (du.double() * z).abs().sum(0), T + 8)


# ---- together: one layer's training step -----------------------------------------------
def layer_inputs(T, d, f, E, dt, seed):
    r = gen(seed)
    return dict(x=draw(r, T, d, dtype=dt), W_g=draw(r, d, E, std=0.1, dtype=dt), b_g=draw(r, E, std=0.5),
                W_gate=draw(r, E, d, f, std=d ** -0.5, dtype=dt), W_up=draw(r, E, d, f, std=d ** -0.5, dtype=dt),
                W_down=draw(r, E, f, d, std=f ** -0.5, dtype=dt), pre_gamma=1 + draw(r, d, std=0.1),
                post_gamma=1 + draw(r, d, std=0.1), gate=draw(r, d), d_out=draw(r, T, d, dtype=dt))


def layer_ref(t, idx, kept, k, renorm, norms, lg, zg, eps):
    """Gradients by automatic differentiation of the layer's definition in 64 bits, with the
    forward's choice of experts and of kept slots."""
    p = {n: v.double().requires_grad_() for n, v in t.items() if n != "d_out"}
    x = p["x"]
    T, E = x.shape[0], p["W_g"].shape[1]
    rms = lambda v: (v.square().mean(1, keepdim=True) + eps).sqrt()  # noqa: E731
    u = x / rms(x) * p["pre_gamma"] if norms else x
    logits = u @ p["W_g"] + p["b_g"]
    prob = torch.softmax(logits, 1)
    sel = prob.gather(1, idx) * kept
    w = sel / sel.sum(1, keepdim=True).clamp_min(1e-300) if renorm else sel
    y = torch.zeros_like(x)
    for e in range(E):
        tok, slot = torch.nonzero((idx == e) & kept, as_tuple=True)
        g = u[tok] @ p["W_gate"][e]
        h = g / (1 + torch.exp(-g)) * (u[tok] @ p["W_up"][e])
        y = y.index_add(0, tok, (h @ p["W_down"][e]) * w[tok, slot][:, None])
    out = 0.5 * x + p["gate"] * (y / rms(y) * p["post_gamma"]) if norms else y
    f = torch.bincount(idx.reshape(-1), minlength=E).double() / T
    total = (out * t["d_out"].double()).sum() + lg * E * (f / k * prob.mean(0)).sum() \
        + zg * torch.logsumexp(logits, 1).square().mean()
    total.backward()
    return {"d" + n if not n.endswith(("gamma", "gate")) or n == "W_gate" else "d_" + n: v.grad
            for n, v in p.items() if v.grad is not None}


@pytest.mark.parametrize("mode", ["tc", "tc_capacity"])
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("norms,renorm", [(False, True), (True, True), (True, False)])
def test_layer_backward(moe, mode, dt, norms, renorm):
    say("layer", mode, dt, norms, renorm)
    T, d, f, E, k, eps = 173, 128, 192, 8, 2, 1e-5
    t = layer_inputs(T, d, f, E, dt, 21)
    dev = {n: v.cuda() for n, v in t.items()}
    kw = dict(pre_gamma=dev["pre_gamma"], post_gamma=dev["post_gamma"], gate=dev["gate"],
              residual_scale=0.5, norm_eps=eps) if norms else {}
    layer = moe.SparseMoE(dev["W_g"], dev["W_gate"], dev["W_up"], dev["W_down"], dev["b_g"], k=k, mode=mode,
                          capacity_factor=0.9, renormalize=renorm, **kw)
    lg, zg = 0.02 * T, 0.01 * T
    out = layer(dev["x"].view(1, T, d))
    assert out.shape == (1, T, d)
    got = layer.backward(dev["d_out"].view(1, T, d), loss_grad=lg, z_loss_grad=zg)
    kept = layer.last["w"].cpu() != 0
    assert mode == "tc" or not bool(kept.all())
    ref = layer_ref(t, layer.last["idx"].cpu().long(), kept, k, renorm, norms, lg, zg, eps)
    assert set(got) == set(ref), (sorted(got), sorted(ref))
    # Of each gradient's size, in the 2-norm. bf16: at most eight values on the way are
    # rounded (u, the two products, dy, dh, the hidden gradient, the rows, the result), half a
    # step of 2^-8 each. fp32: the longest chain of sums has d + f + d terms and T more.
    tol = 8 * 2.0 ** -8 if dt == BF16 else (2 * d + f + T) * U * 8
    for n in ref:
        assert got[n].shape == ref[n].shape, n
        err = float((got[n].double().cpu() - ref[n]).norm() / ref[n].norm())
        assert err <= tol, (n, err)
    # the same call again gives the same bits
    layer(dev["x"])
    again = layer.backward(dev["d_out"], loss_grad=lg, z_loss_grad=zg)
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_layer_backward_without_tokens_and_refusals(moe):
    say("layer none")
    t = {n: v.cuda() for n, v in layer_inputs(0, 64, 64, 4, BF16, 3).items()}
    layer = moe.SparseMoE(t["W_g"], t["W_gate"], t["W_up"], t["W_down"], t["b_g"])
    with pytest.raises(ValueError):
        layer.backward(t["d_out"])
    layer(t["x"])
    got = layer.backward(t["d_out"])
    assert got["dx"].shape == (0, 64) and not any(bool(got[n].any()) for n in got if n != "dx")
    x = torch.randn(32, 64, device="cuda").to(BF16)
    layer(x, eps=torch.randn(32, 4, device="cuda"))
    with pytest.raises(ValueError):
        layer.backward(x)
    layer(x, want_probs=False)
    with pytest.raises(ValueError):
        layer.backward(x)
    ec = moe.SparseMoE(t["W_g"], t["W_gate"], t["W_up"], t["W_down"], mode="ec")
    ec(x, want_stats=False)
    with pytest.raises(ValueError):
        ec.backward(x)


def test_layer_step_captured_in_a_graph(moe):
    # forward and backward of a block as one graph, replayed on new values with eager work of
    # the same operators, on the same shapes, between the replays
    say("graph")
    T, d, f, E = 300, 128, 128, 8
    t = {n: v.cuda() for n, v in layer_inputs(T, d, f, E, BF16, 5).items()}

    def make():
        return moe.SparseMoE(t["W_g"], t["W_gate"], t["W_up"], t["W_down"], t["b_g"], pre_gamma=t["pre_gamma"],
                             post_gamma=t["post_gamma"], gate=t["gate"])

    def step(layer, x, d_out):
        out = layer(x)
        return dict(layer.backward(d_out, loss_grad=1.0, z_loss_grad=0.5), out=out)

    layer, x, d_out = make(), t["x"].clone(), t["d_out"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer, x, d_out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step(layer, x, d_out)
    g = torch.Generator(device="cuda").manual_seed(7)
    for rep in range(4):
        x.copy_(torch.randn(T, d, device="cuda", generator=g))
        d_out.copy_(torch.randn(T, d, device="cuda", generator=g))
        eager = step(make(), x, d_out)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(cap[n], eager[n]), (rep, n)


def test_operators_run_on_the_current_stream(moe):
    # two streams at once, each with inputs made on it: nothing runs on another stream
    say("streams")
    R, E, K, N = 700, 8, 256, 512
    g = gen(31)
    a, b = draw(g, R, K, dtype=BF16), draw(g, E, K, N, dtype=BF16)
    off = offsets_of([R // E] * (E - 1) + [R - R // E * (E - 1)])
    want = moe.moe_grouped_matmul(*cuda(a, b, off))
    gm = torch.ones(K, device="cuda")
    wn = moe.moe_block_norm(a.cuda(), gamma=gm)["u"]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    ha, hb, ho = a.pin_memory(), b.pin_memory(), off.pin_memory()
    for s in streams:
        with torch.cuda.stream(s):
            da, db, do = (h.to("cuda", non_blocking=True) for h in (ha, hb, ho))
            for _ in range(20):
                y = moe.moe_grouped_matmul(da, db, do)
                u = moe.moe_block_norm(da, gamma=gm)["u"]
            got.append((y, u, da, db, do))
    torch.cuda.synchronize()
    for y, u, *_ in got:
        assert torch.equal(y, want) and torch.equal(u, wn)


def test_workspace_of_another_call_changes_nothing(moe):
    # a caller's workspace, larger than needed and full of other values
    say("workspace")
    s = route_inputs(130, 128, 8, 2, BF16, True, 4)
    x, W, p, idx, w, dw = cuda(*(s[n] for n in ("x", "W", "probs", "idx", "w", "dw")))
    want = moe.moe_route_backward(x, W, p, idx, w, dw, z_loss_grad=1.0)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    got = moe.moe_route_backward(x, W, p, idx, w, dw, z_loss_grad=1.0, workspace=ws)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    gm = torch.ones(128, device="cuda")
    f = moe.moe_block_norm(x, gamma=gm)
    a = moe.moe_block_norm_backward(x, d_u=x, rstd=f["rstd"], gamma=gm)
    b = moe.moe_block_norm_backward(x, d_u=x, rstd=f["rstd"], gamma=gm, workspace=ws)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dgamma"], b["dgamma"])
    rows, cols = draw(gen(5), 4000, 64, dtype=BF16).cuda(), draw(gen(6), 4000, 72, dtype=BF16).cuda()
    off = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
    a = moe.moe_grouped_matmul(rows, cols, off, form="tn")
    b = moe.moe_grouped_matmul(rows, cols, off, form="tn", workspace=ws)
    assert torch.equal(a, b)
