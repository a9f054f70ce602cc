"""The expert layer (forward, backward, 8-bit kept rows) against autograd of
the plain formula in 64 bits, and its gradients against differences."""
from __future__ import annotations

import subprocess
import sys

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from software_pipelined_loop_gb300.expert_layer import expert_layer

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(dtype, tokens=200, top_k=3, experts=5, c=136, h=264, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    best, ids = rand(tokens, experts).topk(top_k, dim=1)
    ids = torch.where(rand(tokens, top_k) > 1.5, -1, ids).int()
    w1 = (rand(experts, c, h) * c ** -0.5).to(dtype)
    w2 = (rand(experts, h, c) * h ** -0.5).to(dtype)
    return rand(tokens, c).to(dtype), ids, torch.softmax(best, 1), w1, w2, (rand(tokens, c) / 8).to(dtype)


def plain(x, ids, weights, w1, w2):
    y = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        for j in range(ids.shape[1]):
            has = ids[:, j] == e
            out = torch.nn.functional.silu(x[has] @ w1[e]) @ w2[e]
            y = y.index_add(0, has.nonzero()[:, 0], weights[has, j, None] * out)
    return y


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_against_the_formula(dtype, keep8):
    x, ids, weights, w1, w2, dy = make(dtype)
    args = [t.clone().requires_grad_() for t in (x, weights, w1, w2)]
    y = expert_layer(args[0], ids, args[1], args[2], args[3], keep8)
    y.backward(dy)
    ref = [t.double().requires_grad_() for t in (x, weights, w1, w2)]
    exact = plain(ref[0], ids, ref[1], ref[2], ref[3])
    exact.backward(dy.double())
    # Each result passes through at most eight roundings to 16 bits of values
    # of its own size (two products, the activation and its derivative, the
    # sum and its gradient), whose errors are independent from value to value;
    # the 8-bit rows add half a step of at most 1/64 of a group's largest
    # value, near 1/50 of a normal value's size (relative to the norm).
    u = UNIT[dtype]
    assert float((y.detach().double() - exact.detach()).norm() / exact.detach().norm()) <= 8 * u
    for name, a, r in zip(("x", "weights", "w1", "w2"), args, ref):
        rel = float((a.grad.double() - r.grad).norm() / r.grad.norm())
        loss = 1 / 50 if keep8 and name in ("w1", "w2") else 0.0
        assert rel <= 8 * u + loss, (name, rel)
    assert gp.gemmpipe_get_device_status() == gp.OK


@pytest.mark.parametrize("place", ["x", "weights", "w1", "w2"])
def test_gradients_against_differences(place):
    # L = <dy, layer>, along a direction d: (L(a + h d) - L(a - h d)) / 2h = <grad, d>.
    dtype, h = torch.float16, 2.0 ** -4
    x, ids, weights, w1, w2, dy = make(dtype, seed=3)
    values = {"x": x, "weights": weights, "w1": w1, "w2": w2}
    leaf = {k: v.clone().requires_grad_() for k, v in values.items()}
    y = expert_layer(leaf["x"], ids, leaf["weights"], leaf["w1"], leaf["w2"])
    y.backward(dy)
    g = torch.Generator(device="cuda").manual_seed(9)
    d = torch.randn(values[place].shape, generator=g, device="cuda").sign().double()
    d *= values[place].double().abs()  # a step of h times the value itself
    moved = {s: (values[place].double() + s * h * d).to(values[place].dtype) for s in (1, -1)}
    step = (moved[1].double() - moved[-1].double()) / (2 * h)  # the direction after rounding

    def loss(v, ref):
        args = {**values, place: v}
        if ref:
            args = {k: t.double() for k, t in args.items()}
            return float((plain(args["x"], ids, args["weights"], args["w1"], args["w2"]) * dy.double()).sum())
        out = expert_layer(args["x"], ids, args["weights"], args["w1"], args["w2"])
        return float((out.double() * dy.double()).sum())

    slope = (loss(moved[1], False) - loss(moved[-1], False)) / (2 * h)
    along = float((leaf[place].grad.double() * step).sum())
    # What the difference itself leaves out (its third order), from the formula in 64 bits.
    curve = abs((loss(moved[1], True) - loss(moved[-1], True)) / (2 * h) - along_exact(values, ids, dy, place, step))
    # Independent roundings of y (two evaluations, three roundings deep) and of the gradient: 6 sigma.
    u = UNIT[dtype]
    noise = 6 * u * float((dy.double() * y.double()).norm()) * 3 / h
    noise += 6 * 3 * u * float((leaf[place].grad.double() * step).norm())
    # The weighted sums inside y are larger than y where they cancel: at most by the norm of what is summed.
    assert abs(slope - along) <= noise + curve, (slope, along, noise, curve)


def along_exact(values, ids, dy, place, step):
    args = {k: v.double().requires_grad_() for k, v in values.items()}
    plain(args["x"], ids, args["weights"], args["w1"], args["w2"]).backward(dy.double())
    return float((args[place].grad * step).sum())


def test_one_token_and_dropped_tokens():
    x, ids, weights, w1, w2, _ = make(torch.bfloat16, tokens=1, seed=5)
    ids[:] = torch.tensor([[2, -1, 4]], dtype=torch.int32, device="cuda")
    y = expert_layer(x, ids, weights, w1, w2)
    exact = plain(x.double(), ids, weights.double(), w1.double(), w2.double())
    assert float((y.double() - exact).norm() / exact.norm()) <= 8 * UNIT[torch.bfloat16]
    ids[:] = -1
    assert int(expert_layer(x, ids, weights, w1, w2).count_nonzero()) == 0


def test_command():
    out = subprocess.run([sys.executable, "-m", "software_pipelined_loop_gb300.expert_layer", "--tokens", "300",
                          "--keep8"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert "training step" in out.stdout and "one token" in out.stdout
