"""The bounds that the orthogonalisation documents, held as they stand, not by a model of its roundings:
matrices of every rank, of gradients and worse, by any number of steps, in each way that they are computed.

E is the definition in 64 bits. A result is held to the documented share of |E| plus what rounding E itself to its
type gives.
"""
from __future__ import annotations

import pytest
import torch

from .test_gpu_step import BF16, FP32, NS, moe, norm, plain, say, stack  # noqa: F401  (moe is a fixture)

pytestmark = pytest.mark.gpu


def low_rank(kind, E, m, n, r, seed=0):
    """E matrices of rank r: of random directions; of r tokens with sparse activations and gradients of
    different size; of signs; of channels of different size on both sides."""
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * r)

    def draw(*s):
        return torch.randn(*s, generator=g, device="cuda")
    a, b = draw(E, m, r), draw(E, r, n)
    if kind == "tokens":
        a = torch.relu(a) * (torch.rand(E, m, r, generator=g, device="cuda") < 0.3) * torch.exp(draw(E, 1, r))
    elif kind == "signs":
        a, b = torch.sign(a), torch.sign(b)
    elif kind == "channels":
        a, b = a * torch.exp(draw(E, m, 1)), b * torch.exp(draw(E, 1, n))
    return (a @ b).to(BF16)


KINDS = ("directions", "tokens", "signs", "channels")
RANKS = (1, 2, 4, 8, 16, 32, 64)


def in_fp32(g, steps, co, E):
    """What an iteration that keeps 22 bits may be off by, of two kinds. Against plain fp32: a rounding is 4 times
    its at most, a pair of steps takes twice as many, and plain fp32 (one draw of its roundings) counts twice.
    And by itself, where plain fp32 rounds less than usual (few different values, a power of two as the rank): half a
    step is 2^-22 of a value at most, 0.4 of that on the average (0.58, of values between 1 and 2); it is multiplied by
    up to a in every later step where the singular values are 0, and what a step brings there of X, A and P (norms 1, 1
    and at most a) is 1, |b + c| and a times it: 0.4 sqrt(1 + 2.74^2 + 3.44^2) 2^-22 = 3.6 2^-23 for the default
    coefficients, taken as 4 2^-23."""
    grown = sum(co[0] ** i for i in range(steps))
    return 16 * norm(plain(g, steps, co, 1e-7, FP32) - E) + (2.0 ** -20 + 4 * 2.0 ** -23 * grown) * norm(E)


def check(moe, g, steps, share, co=NS):  # noqa: F811
    """share: the documented bound, None: as in fp32."""
    E = plain(g, steps, co)
    got = moe.moe_orthogonalize(g, steps=steps, coefficients=co).double()
    own = norm(E.to(g.dtype).double() - E)
    most = own * 1.25 + (share * norm(E) if share else in_fp32(g, steps, co, E))
    off = norm(got - E)
    assert bool((off <= most).all()), ((off / norm(E)).tolist(), (most / norm(E)).tolist())


# few matrices with a short side of 129 to 256 (strips), many of them, and longer sides of either schedule
SIZES = [(2, 200, 1000), (1, 256, 512), (2, 1500, 200), (1, 129, 130), (40, 160, 800), (1, 300, 800), (2, 512, 512), (1, 2048, 1408)]


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_low_rank_in_bf16_is_within_2e_2(moe, size, steps):  # noqa: F811
    for kind in KINDS:
        for r in RANKS:
            say("low rank", size, steps, kind, r)
            check(moe, low_rank(kind, *size, r), steps, 2e-2)


@pytest.mark.parametrize("steps", [6, 8, 10])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_low_rank_by_many_steps_is_as_in_fp32(moe, size, steps):  # noqa: F811
    """Past five steps of the default coefficients bf16 matrices are kept in two terms."""
    for kind in KINDS:
        for r in RANKS:
            say("low rank", size, steps, kind, r)
            check(moe, low_rank(kind, *size, r), steps, None)


@pytest.mark.parametrize("size", [(2, 200, 1000), (1, 256, 512), (2, 1500, 200), (1, 129, 130), (4, 200, 500), (1, 200, 4096), (8, 440, 168)], ids=lambda s: "x".join(map(str, s)))
def test_low_rank_of_few_matrices_is_as_in_fp32(moe, size):  # noqa: F811
    """Few matrices of a short side of 129 to 256, of which the fewest take every step singly, are kept in two terms."""
    assert size[0] * -(-max(size[1:]) // 128) <= 32
    for kind in KINDS:
        for r in RANKS:
            say("low rank", size, kind, r)
            check(moe, low_rank(kind, *size, r), 5, None)


@pytest.mark.parametrize("co,steps", [((1.5, -0.5, 0.0), 11), ((1.5, -0.5, 0.0), 12), ((1.875, -1.25, 0.375), 8),
                                      ((1.875, -1.25, 0.375), 20), ((1.0, 0.0, 0.0), 64), ((2.0, -1.5, 0.5), 7), ((3.0, -3.2, 1.2), 5),
                                      ((4.0848, -6.8946, 2.9270), 4), ((1.0, 4.0, -4.0), 3)])
@pytest.mark.parametrize("size", [(1, 300, 800), (2, 512, 512)], ids=lambda s: "x".join(map(str, s)))
def test_other_coefficients_are_within_2e_2(moe, size, co, steps):  # noqa: F811
    """As many steps as one term takes of them, and more."""
    for kind in KINDS:
        for r in (1, 4, 16, 64):
            say("low rank", size, co, steps, kind, r)
            check(moe, low_rank(kind, *size, r), steps, 2e-2, co)


@pytest.mark.parametrize("size", [(8, 140, 300), (40, 160, 800), (4, 256, 1024), (4, 512, 512), (2, 512, 2048), (1, 1024, 4096), (1, 2048, 1408)],
                         ids=lambda s: "x".join(map(str, s)))
def test_full_rank_in_bf16_is_within_2e_3(moe, size):  # noqa: F811
    for steps in (3, 5):
        say("full rank", size, steps)
        check(moe, stack(*size, BF16), steps, 2e-3)
        check(moe, torch.randn(*size, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF16), steps, 2e-3)


@pytest.mark.parametrize("size", [(1, 512, 1024), (1, 1024, 4096), (1, 2048, 1408)], ids=lambda s: "x".join(map(str, s)))
def test_small_rows_among_others(moe, size):  # noqa: F811
    """Every other row (column of a tall matrix) 1e-2 to 1e-5 times the others. In one term values below 2^-14 are
    rounded to 2^-25, where X's, scaled, are k / sqrt(short side) or more: 0.58 2^-25 sqrt(short side) / k of such rows
    on the average; in the first step X, A X and P X carry it, 1 + |b| + 2 |c| = 9.8 times at most. In two terms to 2^-36."""
    s = min(size[1:])
    for k in (1e-2, 1e-3, 1e-4, 1e-5):
        g = torch.randn(*size, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
        part = (slice(None), slice(0, None, 2)) if size[1] < size[2] else (slice(None), slice(None), slice(0, None, 2))
        g[part] *= k
        g = g.to(BF16)
        say("small rows", size, k)
        E = plain(g, 5)
        for dt, share, bits in ((BF16, 2e-3, 25), (FP32, 1e-5, 36)):
            off = moe.moe_orthogonalize(g.to(dt)).double() - E
            own = E.to(dt).double() - E
            assert bool((norm(off) <= share * norm(E) + 1.25 * norm(own)).all())
            most = share + 9.8 * 0.58 * 2.0 ** -bits * s ** 0.5 / k
            assert bool((norm(off[part]) <= most * norm(E[part]) + 1.25 * norm(own[part])).all()), (k, dt)
