"""The few-token operators have no gradients: whoever asks for them, in reverse or in forward mode and of any argument,
gets an error instead of a result without them (all before any device call, no GPU needed)."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from software_pipelined_loop_gb300 import few_tokens as few
from test_few_tokens_arguments import C, H, T, arguments, packed


def calls(mark):
    """(name, call) for every floating-point argument of every operator, that one marked."""
    for name in ("x", "weights", "w1", "w2", "w3"):
        args = arguments()
        yield name, lambda a=args | {name: mark(args[name])}: few.expert_step(**a)
    for name in ("w1", "w2", "w3"):
        args = arguments(True)
        m = args[name]._replace(scales=mark(args[name].scales))
        yield name + " in 4 bits", lambda a=args | {name: m}: few.expert_step(**a)
    x, m, w = torch.zeros(T, C, dtype=torch.bfloat16), packed(1, C, H), torch.zeros(C, H, dtype=torch.bfloat16)
    yield "rows4 x", lambda: few.rows4(mark(x), m)
    yield "rows4 scales", lambda: few.rows4(x, m._replace(scales=mark(m.scales)))
    yield "pack4", lambda: few.pack4(mark(w))
    yield "unpack4", lambda: few.unpack4(m._replace(scales=mark(m.scales)))


NAMES = [name for name, _ in calls(lambda t: t)]


@pytest.mark.parametrize("name", NAMES)
def test_reverse_mode(name):
    with pytest.raises(RuntimeError, match="gradients"):
        dict(calls(lambda t: t.clone().requires_grad_()))[name]()


@pytest.mark.parametrize("no_grad", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_forward_mode(name, no_grad):
    with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        with pytest.raises(RuntimeError, match="gradients"):
            dict(calls(lambda t: forward_ad.make_dual(t, torch.ones_like(t))))[name]()


@pytest.mark.parametrize("name", NAMES)
def test_without_gradients_the_call_goes_on(name):
    # (to the next check, which finds no GPU tensors)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        dict(calls(lambda t: t.clone().requires_grad_()))[name]()
    with forward_ad.dual_level(), pytest.raises(ValueError, match="CUDA"):
        dict(calls(lambda t: t))[name]()
    with forward_ad.dual_level():
        dual = dict(calls(lambda t: forward_ad.make_dual(t, torch.ones_like(t))))[name]
        with torch.inference_mode(), pytest.raises(ValueError, match="CUDA"):
            dual()
