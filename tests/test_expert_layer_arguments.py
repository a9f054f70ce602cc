"""Refusals of the expert layer, all before any device call (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import expert_layer as layer

T, K, E, C, H = 6, 2, 3, 16, 24


def arguments():
    return {"x": torch.zeros(T, C, dtype=torch.bfloat16), "ids": torch.zeros(T, K, dtype=torch.int32),
            "weights": torch.zeros(T, K), "w1": torch.zeros(E, C, H, dtype=torch.bfloat16),
            "w2": torch.zeros(E, H, C, dtype=torch.bfloat16)}


@pytest.mark.parametrize("name, dtype", [
    ("x", torch.float32), ("x", torch.float16),                      # not a 16-bit type; not the matrices'
    ("ids", torch.int64), ("ids", torch.int16), ("ids", torch.bool),  # int64 is what topk returns
    ("weights", torch.bfloat16), ("weights", torch.float16), ("weights", torch.float64),
    ("w1", torch.float16), ("w1", torch.float32), ("w2", torch.float16), ("w2", torch.float64)])
def test_types(name, dtype):
    args = arguments()
    args[name] = args[name].to(dtype)
    with pytest.raises(TypeError, match=name):
        layer.expert_layer(**args)


@pytest.mark.parametrize("name, shape", [
    ("x", (T, C, 1)), ("x", (T + 1, C)), ("x", (T, C + 1)), ("x", (C,)),
    ("ids", (T,)), ("ids", (T + 1, K)), ("ids", (T, K, 1)),
    ("weights", (T, K + 1)), ("weights", (T - 1, K)), ("weights", (K, T)), ("weights", (T * K,)), ("weights", (1, K)),
    ("w1", (E, C + 8, H)), ("w1", (E, H, C)), ("w1", (C, H)), ("w1", (E, C, H + 1)),
    ("w2", (E, H + 8, C)), ("w2", (E, H, C + 1)), ("w2", (E + 1, H, C)), ("w2", (E - 1, H, C)), ("w2", (H, C))])
def test_shapes(name, shape):
    args = arguments()
    args[name] = torch.zeros(shape, dtype=args[name].dtype)
    with pytest.raises(ValueError):
        layer.expert_layer(**args)


@pytest.mark.parametrize("ids", [torch.zeros(T, K, dtype=torch.int64), torch.zeros(T, K, dtype=torch.float32)])
def test_route_types(ids):
    with pytest.raises(TypeError, match="ids"):
        layer.route(ids, E)


def test_route_shape():
    with pytest.raises(ValueError, match="ids"):
        layer.route(torch.zeros(T, dtype=torch.int32), E)


def test_devices():
    with pytest.raises(ValueError, match="CUDA"):
        layer.expert_layer(**arguments())
    with pytest.raises(ValueError, match="CUDA"):
        layer.route(arguments()["ids"], E)
    mixed = arguments()
    mixed["w2"] = mixed["w2"].to("meta")
    with pytest.raises(ValueError, match="CUDA"):
        layer.expert_layer(**mixed)
