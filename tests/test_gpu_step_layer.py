"""The layer's update step as a whole: what a refused call leaves, and what a captured one relies on."""
from __future__ import annotations

import pytest
import torch

from .test_gpu_step import BF16, FP32, draw, gen, layer, moe  # noqa: F401  (moe is a fixture)

pytestmark = pytest.mark.gpu

NAMES = ("W_gate", "W_up", "W_down")


def trained(moe, dt, steps=1):  # noqa: F811
    """A layer after some steps, and the gradients of one more."""
    block, _, _, x = layer(moe, dt)
    for i in range(steps + 1):
        block(x.cuda())
        grads = block.backward(draw(gen(i), *x.shape).cuda())
        if i < steps:
            block.muon_update(grads, lr=0.02)
    return block, grads


REFUSED = {
    "absent": (KeyError, lambda b, g: g.pop("dW_down"), {}),
    "none": (ValueError, lambda b, g: g.update(dW_down=None), {}),
    "type": (TypeError, lambda b, g: g.update(dW_down=g["dW_down"].double()), {}),
    "shape": (ValueError, lambda b, g: g.update(dW_up=g["dW_up"][:-1]), {}),
    "strided": (ValueError, lambda b, g: g.update(dW_up=g["dW_up"].transpose(1, 2).contiguous().transpose(1, 2)), {}),
    "itself": (ValueError, lambda b, g: g.update(dW_down=b.W_down), {}),
    "momentum": (ValueError, lambda b, g: b.momentum.update(W_down=b.momentum["W_up"]), {}),
    "steps": (RuntimeError, lambda b, g: None, dict(steps=65)),
    "lr": (ValueError, lambda b, g: None, dict(lr=float("inf"))),
    "workspace": (ValueError, lambda b, g: setattr(b, "_update_ws", torch.empty(64 << 20, dtype=torch.uint8, device="cuda")[1:]), {}),
}


@pytest.mark.parametrize("name,steps", [(n, s) for n in sorted(REFUSED) for s in (0, 1) if s or n != "momentum"])
def test_refused_update_changes_nothing(moe, name, steps):  # noqa: F811
    error, spoil, kw = REFUSED[name]
    block, grads = trained(moe, FP32, steps)
    kept = dict(block.momentum)
    spoil(block, grads)
    weights = {n: getattr(block, n).clone() for n in NAMES}
    momentum = {n: t.clone() for n, t in kept.items()}
    with pytest.raises(error):
        block.muon_update(grads, **{"lr": 0.02, **kw})
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(block, n), weights[n]) for n in NAMES)
    assert all(torch.equal(kept[n], momentum[n]) for n in kept) and len(block.momentum) == len(kept)


def test_workspaces_of_a_captured_step_outlive_larger_ones(moe):  # noqa: F811
    """A graph holds the addresses of the workspaces that the eager step before it made. Calls of more rows and of
    updates by more steps put larger ones in their place; what is allocated then is not what the graph writes to."""
    eager, _, _, x = layer(moe, BF16)
    held, _, _, _ = layer(moe, BF16)
    rows = [draw(gen(40 + i), *x.shape).to(BF16).cuda() for i in range(4)]
    many = draw(gen(50), 4096, x.shape[1]).to(BF16).cuda()
    d_out = draw(gen(51), *x.shape).to(BF16).cuda()

    def one(block, r):
        y = block(r)
        block.muon_update(block.backward(d_out), lr=0.02, steps=2)
        return y

    def large(block):
        block(many)
        return block.backward(many)
    want = []
    for i, r in enumerate(rows):
        want.append(one(eager, r).clone())
        if i:
            eager.muon_update(large(eager), lr=0.02)
    buf = rows[0].clone()
    assert torch.equal(one(held, buf), want[0])
    torch.cuda.synchronize()
    before = held._ws, held._update_ws
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one(held, buf)
    assert held._ws is before[0] and held._update_ws is before[1]
    assert all(any(t is c for c in held._captured) for t in before)
    at = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in before]
    del before
    for r, w in zip(rows[1:], want[1:]):
        buf.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        held.muon_update(large(held), lr=0.02)
        other = [torch.full((b - a,), 1, dtype=torch.uint8, device="cuda") for a, b in at]
        for t in other + [held._ws, held._update_ws]:
            assert all(t.data_ptr() >= b or t.data_ptr() + t.numel() <= a for a, b in at)
    assert all(torch.equal(getattr(held, n), getattr(eager, n)) for n in NAMES)
    assert all(torch.equal(held.momentum[n], eager.momentum[n]) for n in NAMES)
    assert held._captured and len(held._captured) == 2


def test_layer_with_one_workspace_keeps_none_without_a_capture(moe):  # noqa: F811
    block, grads = trained(moe, FP32)
    block.muon_update(grads, lr=0.02)
    assert block._captured == []
