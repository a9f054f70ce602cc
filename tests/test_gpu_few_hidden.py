"""Hidden values of any size in the few-token layer: the result is off by its last rounding only."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import few_tokens as few
from test_gpu_few import TYPES, generator, status_ok

pytestmark = pytest.mark.gpu


def exact_matrices(ws, four):
    if not four:
        return [w.double() for w in ws]
    exact = []
    for m in ws:
        q = torch.stack([(m.words >> (4 * [0, 2, 4, 6, 1, 3, 5, 7].index(r))) & 15 for r in range(8)], 2).flatten(1, 2)
        s = m.scales.double().repeat_interleave(four, 1)[:, :m.inner, :m.outer]
        exact.append((q[:, :m.inner, :m.outer].double() - 8) * s)
    return exact


def error_and_rounding(type_, four, t, k, e, c, h, small, key):
    """(Distance of expert_step from the exact result, of that result's rounding): hidden values near 2^-small."""
    g = generator(key, type_, four, t, small)
    dtype = TYPES[type_][1]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, weights = rand(t, c).to(dtype), torch.rand(t, k, generator=g, device="cuda")
    ids = torch.rand(t, e, generator=g, device="cuda").topk(k, 1).indices.int()
    w1, w2, w3 = rand(e, c, h) * c ** -0.5, rand(e, h, c) * h ** -0.5 * 2.0 ** small, rand(e, c, h) * c ** -0.5 * 2.0 ** -small
    ws = [w.to(dtype) for w in (w1, w2, w3)]
    if four:
        ws = [few.pack4(w, four) for w in ws]
    e1, e2, e3 = exact_matrices(ws, four)
    want = torch.zeros(t, c, dtype=torch.float64, device="cuda")
    for n in range(e):
        token, j = (ids == n).nonzero(as_tuple=True)
        hidden = torch.nn.functional.silu(x[token].double() @ e1[n]) * (x[token].double() @ e3[n])
        want.index_add_(0, token, weights[token, j].double()[:, None] * (hidden @ e2[n]))
    y = few.expert_step(x, ids, weights, *ws)
    status_ok()
    return float((y.double() - want).norm()), float((want.to(dtype).double() - want).norm())


@pytest.mark.parametrize("small", [0, 6, 12])
@pytest.mark.parametrize("t", [1, 3, 8])
@pytest.mark.parametrize("four", [0, 64])
@pytest.mark.parametrize("type_", TYPES)
def test_small_hidden_values(type_, four, t, small):
    error, once = error_and_rounding(type_, four, t, 3, 6, 520, 264, small, "small")
    # (besides: fp32 sums and the activation, some 2^-20 of the values, next to 2^-9 or 2^-12)
    assert error <= 1.05 * once


@pytest.mark.parametrize("t, k, e", [(9, 3, 6), (12, 2, 3), (13, 3, 6), (16, 8, 24), (17, 2, 3), (40, 2, 8), (64, 8, 24),
                                     (64, 4, 4)])
@pytest.mark.parametrize("four", [0, 32, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_many_tokens(type_, four, t, k, e):
    """More than 8 tokens, few and many rows of an expert: the same as for one."""
    error, once = error_and_rounding(type_, four, t, k, e, 520, 264, 4, "many")
    assert error <= 1.05 * once


@pytest.mark.parametrize("t", [11, 50])
def test_many_tokens_off_boundaries(t):
    error, once = error_and_rounding("f16", 0, t, 4, 12, 411, 101, 4, "odd")
    assert error <= 1.05 * once
