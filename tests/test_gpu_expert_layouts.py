"""The expert layer on views: transposed and sliced arguments give what their
dense copies give, results and gradients, bit for bit."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from software_pipelined_loop_gb300.expert_layer import expert_layer

pytestmark = pytest.mark.gpu

T, K, E, C, H = 90, 2, 5, 72, 104


def dense(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(-1, E, (T, K), generator=g, device="cuda").int()
    return {"x": rand(T, C).to(dtype), "ids": ids, "weights": torch.softmax(rand(T, K), 1),
            "w1": (rand(E, C, H) * C ** -0.5).to(dtype), "w2": (rand(E, H, C) * H ** -0.5).to(dtype)}, rand(T, C).to(dtype)


def transposed(t):  # as a linear layer keeps its matrices
    return t.transpose(-1, -2).contiguous().transpose(-1, -2)


def sliced(t):  # the first columns of a wider tensor
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), 7, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def every_other(t):  # every second entry along the first dimension
    return torch.stack([t, torch.full_like(t, 3)], 1).flatten(0, 1)[::2]


def run(args, dy, keep8):
    leaves = {k: v.detach() if k == "ids" else v.detach().requires_grad_() for k, v in args.items()}
    assert all(leaves[k].stride() == args[k].stride() for k in args)
    y = expert_layer(leaves["x"], leaves["ids"], leaves["weights"], leaves["w1"], leaves["w2"], keep8)
    y.backward(dy)
    return [y.detach()] + [leaves[k].grad for k in ("x", "weights", "w1", "w2")]


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("view", [transposed, sliced, every_other], ids=lambda f: f.__name__)
@pytest.mark.parametrize("which", ["x", "ids", "weights", "w1", "w2", "all"])
def test_views_are_their_values(which, view, keep8):
    args, dy = dense(torch.bfloat16)
    want = run(args, dy, keep8)
    moved = {k: view(v) if which in (k, "all") else v for k, v in args.items()}
    assert any(not v.is_contiguous() for v in moved.values())
    got = run(moved, view(dy), keep8)
    for name, a, b in zip(("y", "x", "weights", "w1", "w2"), got, want):
        assert torch.equal(a, b), name
    assert gp.gemmpipe_get_device_status() == gp.OK


def test_expanded_weights():
    # One router weight for all choices, and one matrix for all experts, as stride-0 views.
    args, dy = dense(torch.float16)
    args["weights"], args["w1"] = torch.full((T, K), 0.5, device="cuda"), args["w1"][:1].repeat(E, 1, 1)
    want = run(args, dy, False)
    leaf_w, leaf_1 = torch.full((1, 1), 0.5, device="cuda").requires_grad_(), args["w1"][:1].clone().requires_grad_()
    y = expert_layer(args["x"], args["ids"], leaf_w.expand(T, K), leaf_1.expand(E, C, H), args["w2"])
    y.backward(dy)
    assert torch.equal(y.detach(), want[0])
    # The sums over the broadcast dimensions, of the same gradients.
    assert torch.equal(leaf_w.grad, want[2].sum((0, 1), keepdim=True))
    assert torch.equal(leaf_1.grad, want[3].sum(0, keepdim=True))
