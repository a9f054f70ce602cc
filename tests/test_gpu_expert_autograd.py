"""What autograd asks of the expert layer, and what the layer does for it."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from software_pipelined_loop_gb300.expert_layer import expert_layer

pytestmark = pytest.mark.gpu

T, K, E, C, H = 40, 2, 3, 64, 128


def leaves(grad=("x", "weights", "w1", "w2")):
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {"x": rand(T, C).bfloat16(), "weights": torch.softmax(rand(T, K), 1),
         "w1": (rand(E, C, H) * C ** -0.5).bfloat16(), "w2": (rand(E, H, C) * H ** -0.5).bfloat16()}
    for name in grad:
        t[name].requires_grad_()
    return t, torch.randint(-1, E, (T, K), generator=g, device="cuda").int(), rand(T, C).bfloat16()


@pytest.mark.parametrize("name", ["x", "weights", "w1", "w2"])
def test_second_derivatives_are_refused(name):
    # The gradients are made outside autograd: to differentiate them again is an error, not a zero.
    t, ids, dy = leaves()
    y = expert_layer(t["x"], ids, t["weights"], t["w1"], t["w2"])
    grad, = torch.autograd.grad(y, t[name], dy, create_graph=True)
    loss = grad.float().square().sum() + sum(v.float().square().sum() for v in t.values())
    with pytest.raises(RuntimeError, match="differentiated again"):
        loss.backward()
    assert gp.gemmpipe_get_device_status() == gp.OK
