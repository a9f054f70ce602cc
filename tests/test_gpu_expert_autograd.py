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


@pytest.fixture
def calls(monkeypatch):
    """Names of the library calls made, in order."""
    made = []
    for name in [n for n in dir(gp) if n.startswith(("gemm_grouped", "gemmpipe_keep8"))]:
        def counted(*args, _name=name, _call=getattr(gp, name)):
            made.append(_name)
            return _call(*args)
        monkeypatch.setattr(gp, name, counted)
    return made


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("grad, want", [
    (("x",), {"gemm_grouped_dx": 2}),                             # frozen experts
    (("weights",), {}),                                           # the router alone
    (("w1",), {"gemm_grouped_dx": 1, "gemm_grouped_dw": 1}),
    (("w2", "weights"), {"gemm_grouped_dw": 1}),
    (("w1", "w2"), {"gemm_grouped_dx": 1, "gemm_grouped_dw": 2}),  # rows that need no gradient
    (("x", "weights", "w1", "w2"), {"gemm_grouped_dx": 2, "gemm_grouped_dw": 2})], ids=lambda v: "+".join(v))
def test_only_the_gradients_asked_for(calls, grad, want, keep8):
    t, ids, dy = leaves()
    expert_layer(t["x"], ids, t["weights"], t["w1"], t["w2"], keep8).backward(dy)
    every = {k: v.grad for k, v in t.items()}
    t, ids, dy = leaves(grad)
    y = expert_layer(t["x"], ids, t["weights"], t["w1"], t["w2"], keep8)
    calls.clear()
    y.backward(dy)
    made = [c.replace("dw8", "dw") for c in calls]
    assert {c: made.count(c) for c in set(made)} == want
    for name, v in t.items():
        assert v.grad is None if name not in grad else torch.equal(v.grad, every[name]), name
    assert gp.gemmpipe_get_device_status() == gp.OK


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_without_a_backward_pass(calls, mode):
    t, ids, _ = leaves()
    with mode():
        y = expert_layer(t["x"], ids, t["weights"], t["w1"], t["w2"], True)
    assert calls == ["gemm_grouped"] * 2
    assert torch.equal(y, expert_layer(t["x"], ids, t["weights"], t["w1"], t["w2"]).detach())
