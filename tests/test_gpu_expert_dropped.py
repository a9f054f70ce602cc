"""Dropped choices next to values that are not finite: what a token's dropped
choices get is an exact zero, whatever its gradient row holds."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("ty", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("C", [8, 264, 265, 2056, 3001])  # on and off 16-byte rows, one and several passes of a block
def test_gradient_of_dropped_choices_is_zero(C, ty, weighted):
    code = gp.F16 if ty == torch.float16 else gp.BF16
    T, k, E = 6, 3, 4
    g = torch.Generator(device="cuda").manual_seed(C)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    ids[1] = ids[4] = -1      # tokens without a choice
    ids[2, 1] = ids[5, 0] = -1
    off, slots, rows = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    gp.gemmpipe_route(T, k, E, ids, off, slots, rows)
    rows = rows.view(T, k)
    kept = rows >= 0
    dY = torch.randn(T, C, generator=g, device="cuda").to(ty)
    dY[1], dY[4, C // 2] = float("nan"), float("inf")
    dY[2, C - 1] = float("-inf")  # a token with kept and dropped choices
    Ys = torch.randn(T * k, C, generator=g, device="cuda").to(ty)
    weights = torch.rand(T, k, generator=g, device="cuda") if weighted else None
    dYs = torch.full((T * k, C), 9.0, dtype=ty, device="cuda")
    dweights = torch.full((T, k), 9.0, device="cuda")
    gp.gemmpipe_combine_grad(code, T, k, C, dY, C, Ys, C, rows, weights, dYs, C, dweights)
    assert int(dweights[~kept].count_nonzero()) == 0
    assert int(dYs[(~rows[~kept]).long()].count_nonzero()) == 0
    finite = torch.isfinite(dY).all(1)[:, None] & kept
    assert bool(torch.isfinite(dweights[finite]).all()) and bool(torch.isfinite(dYs[rows[finite].long()]).all())
    assert not bool(torch.isfinite(dweights[2][kept[2]]).any())  # a kept choice's does reach its weight
    assert gp.gemmpipe_get_device_status() == gp.OK
