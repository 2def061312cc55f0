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
