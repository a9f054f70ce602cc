"""Refusals of the few-token operators for PyTorch, all before any device call (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import few_tokens as few

T, K, E, C, H = 6, 2, 3, 16, 24


def packed(e, k, n, group=32, dtype=torch.bfloat16):
    n4 = (n + 3) // 4 * 4
    return few.Packed4(torch.zeros(e, -(-k // 8), n4, dtype=torch.int32),
                       torch.zeros(e, -(-k // group), n4, dtype=dtype), k, n, group)


def arguments(four=False):
    make = (lambda *s: packed(*s)) if four else (lambda *s: torch.zeros(*s, dtype=torch.bfloat16))
    return {"x": torch.zeros(T, C, dtype=torch.bfloat16), "ids": torch.zeros(T, K, dtype=torch.int32),
            "weights": torch.zeros(T, K), "w1": make(E, C, H), "w2": make(E, H, C), "w3": make(E, C, H)}


@pytest.mark.parametrize("name, dtype", [
    ("x", torch.float32), ("x", torch.float16), ("ids", torch.int64), ("weights", torch.bfloat16),
    ("w1", torch.float16), ("w2", torch.float32), ("w3", torch.float16)])
def test_types(name, dtype):
    args = arguments()
    args[name] = args[name].to(dtype)
    with pytest.raises(TypeError):
        few.expert_step(**args)


@pytest.mark.parametrize("name, shape", [
    ("x", (T + 1, C)), ("x", (T, C + 1)), ("x", (T, C, 1)), ("ids", (T,)), ("ids", (T + 1, K)), ("weights", (T, K + 1)),
    ("weights", (1, K)), ("w1", (E, H, C)), ("w1", (C, H)), ("w2", (E + 1, H, C)), ("w2", (E, C, H)),
    ("w3", (E, H, C)), ("w3", (E - 1, C, H))])
def test_shapes(name, shape):
    args = arguments()
    args[name] = torch.zeros(shape, dtype=args[name].dtype)
    with pytest.raises(ValueError):
        few.expert_step(**args)


def test_too_many_tokens():
    args = arguments()
    args |= {"x": torch.zeros(65, C, dtype=torch.bfloat16), "ids": torch.zeros(65, K, dtype=torch.int32),
             "weights": torch.zeros(65, K)}
    with pytest.raises(ValueError, match="64"):
        few.expert_step(**args)
    with pytest.raises(ValueError, match="64"):
        few.rows4(args["x"], packed(1, C, H))


@pytest.mark.parametrize("change, error", [
    ({"w2": torch.zeros(E, H, C, dtype=torch.bfloat16)}, TypeError),  # 16 and 4 bits together
    ({"w3": packed(E, C, H, 64)}, ValueError),                        # another group
    ({"w1": packed(E, C, H, dtype=torch.float16)}, TypeError),
    ({"w2": packed(E, C, H)}, ValueError),
    ({"w1": packed(E, C, H)._replace(inner=C + 8)}, ValueError),
    ({"w1": packed(E, C, H)._replace(group=16)}, ValueError),
    ({"w1": packed(E, C, H)._replace(words=torch.zeros(E, 2, 24, dtype=torch.int64))}, TypeError)])
def test_packed_matrices(change, error):
    with pytest.raises(error):
        few.expert_step(**(arguments(True) | change))


def test_rows4_and_pack4():
    x = torch.zeros(T, C, dtype=torch.bfloat16)
    for bad, error in [((x.float(), packed(1, C, H)), TypeError), ((x, packed(2, C, H)), ValueError),
                       ((x, packed(1, C + 1, H)), ValueError), ((x[0], packed(1, C, H)), ValueError),
                       ((x, packed(1, C, H, dtype=torch.float16)), TypeError)]:
        with pytest.raises(error):
            few.rows4(*bad)
    with pytest.raises(TypeError):
        few.pack4(x.float())
    with pytest.raises(ValueError):
        few.pack4(x, 16)
    with pytest.raises(ValueError):
        few.pack4(x[0])
    with pytest.raises(ValueError):
        few.unpack4(packed(1, C, H)._replace(outer=H + 4))


def test_gradients_are_refused():
    for name in ("x", "weights", "w1", "w2", "w3"):
        args = arguments()
        args[name].requires_grad_()
        with pytest.raises(RuntimeError, match="gradients"):
            few.expert_step(**args)
    with pytest.raises(RuntimeError, match="gradients"):
        few.rows4(torch.zeros(T, C, dtype=torch.bfloat16, requires_grad=True), packed(1, C, H))
    with pytest.raises(RuntimeError, match="gradients"):
        few.pack4(torch.zeros(C, H, dtype=torch.bfloat16, requires_grad=True))


@pytest.mark.parametrize("four", [False, True])
def test_devices(four):
    with pytest.raises(ValueError, match="CUDA"):
        few.expert_step(**arguments(four))
    with pytest.raises(ValueError, match="CUDA"):
        few.rows4(torch.zeros(T, C, dtype=torch.bfloat16), packed(1, C, H))
    with pytest.raises(ValueError, match="CUDA"):
        few.pack4(torch.zeros(C, H, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        few.unpack4(packed(1, C, H))
