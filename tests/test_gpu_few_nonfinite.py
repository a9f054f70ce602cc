"""Infinities and NaN in the operands of the few-token operators: the results that the formulas give, and in a time
that is of the order of the finite ones'."""
from __future__ import annotations

import math

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import TYPES, generator, ints, run_step, scales_of, status_ok, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 3, 5, 8, 12, 20, 40])
@pytest.mark.parametrize("four", [0, 64])
@pytest.mark.parametrize("type_", TYPES)
def test_infinities_of_the_second_matrix(type_, four, t):
    """An infinite weight of w2 gives infinities in its column, of the sign of what it multiplies, and NaN only where
    the formula has infinity minus infinity; the other columns are as without it.  (In 4 bits an infinite scale makes
    its whole group's weights infinite: there hidden values are all positive.)"""
    e, k, c, h = 3, 2, 200, 136
    g = generator("infinite w2", type_, four, t)
    dtype = TYPES[type_][1]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w1, w3 = rand(t, c).to(dtype), rand(e, c, h) * c ** -0.5, rand(e, c, h) * c ** -0.5
    if four:
        x = x.abs()
    ids = torch.stack([torch.randperm(e, generator=g, device="cuda")[:k] for _ in range(t)]).int()
    weights = torch.rand(t, k, generator=g, device="cuda") + 0.5
    steps = ints(g, -7, 7, e, h, c)
    places = [(0, 5, 3, math.inf), (1, 70, 64, -math.inf), (2, 135, 199, math.inf)]  # expert, row, column
    args = {"x": x, "ids": ids, "weights": weights}
    if four:
        groups = -(-h // four)
        scale = torch.full((e, groups, c), 2.0 ** -7, dtype=torch.float64, device="cuda")
        for n, row, col, v in places:
            scale[n, row // four, col] = v
            steps[n, row // four * four:(row // four + 1) * four, col] = 7
        args["w2"] = words_of(steps), scales_of(scale, c, dtype)
        w2 = steps * scale.repeat_interleave(four, 1)[:, :h]
        for name, w in (("w1", w1), ("w3", w3)):
            q = (w * 4 * c ** 0.5).abs().round().clamp(0, 7).double()
            s = torch.full((e, -(-c // four), h), c ** -0.5 / 4, dtype=torch.float64, device="cuda").to(dtype).double()
            args[name] = words_of(q), scales_of(s, h, dtype)
            w.copy_(q * s.repeat_interleave(four, 1)[:, :c])
    else:
        w2 = (steps / 128).to(dtype).double()
        for n, row, col, v in places:
            w2[n, row, col] = v
        args |= {"w1": w1.to(dtype), "w2": w2.to(dtype), "w3": w3.to(dtype)}
        w1, w3 = args["w1"], args["w3"]
    hidden = torch.nn.functional.silu(torch.einsum("tc,ech->teh", x.double(), w1.double())) * \
        torch.einsum("tc,ech->teh", x.double(), w3.double())
    finite = torch.where(w2.isfinite(), w2, 0.0)
    sums = torch.einsum("teh,ehc->tec", hidden, finite)
    for n, row, col, v in places:
        rows = slice(row // four * four, (row // four + 1) * four) if four else slice(row, row + 1)
        by = hidden[:, n, rows].sum(1)
        assert float(by.abs().min()) > 1e-4  # (signs that rounding does not change)
        sums[:, n, col] = by * v
    factor = torch.zeros(t, e, dtype=torch.float64, device="cuda")
    factor.scatter_(1, ids.long(), weights.double())
    chosen = torch.zeros(t, e, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    want = torch.where(chosen[:, :, None], factor[:, :, None] * sums, 0.0).sum(1)
    y = run_step(type_, args, e, h, four)
    status_ok()
    infinite = want.isinf()
    assert bool(infinite.any()) and torch.equal(infinite, y.isinf()) and torch.equal(want.isnan(), y.isnan())
    assert torch.equal(y[infinite].double(), want[infinite])
    rest = want.isfinite()
    error = (y[rest].double() - want[rest]).norm() / want[rest].norm()
    assert float(error) <= 3 * torch.finfo(dtype).eps / 2  # (hidden rows and y: a rounding each, at most)


@pytest.mark.parametrize("what", ["rows", "scales", "large scales"])
@pytest.mark.parametrize("type_", TYPES)
def test_time_of_sums_that_are_not_finite(type_, what):
    """64 rows x 2^18 x 128 in groups of 32: every sum infinite, or its weights past the type's largest value."""
    m, k, n, group = 64, 1 << 18, 128, 32
    code, dtype = TYPES[type_]
    g = generator("slow", type_, what)
    x = ints(g, 0, 1, m, k).to(dtype)
    steps = ints(g, 1, 7, 1, k, n)
    scale = torch.full((1, k // group, n), 2.0 ** -6, dtype=torch.float64, device="cuda")
    if what == "rows":
        x[:, 1000] = math.inf
        want = torch.full((m, n), math.inf, dtype=dtype, device="cuda")
    elif what == "scales":
        scale[0, 77] = math.inf
        x[:, 77 * group] = 1
        want = torch.full((m, n), math.inf, dtype=dtype, device="cuda")
    else:
        # One group's weights are past the largest value; its rows of X bring them back to 7 * 2^-9.
        top = torch.finfo(dtype).max
        scale[0, 55] = 2.0 ** math.floor(math.log2(top))
        steps[0, 55 * group:56 * group] = 7
        x *= 0
        x[:, 55 * group] = 2.0 ** -24 if type_ == "f16" else 2.0 ** -130
        want = (x[:, 55 * group, None].double() * 7 * scale[:, 55]).to(dtype).expand(m, n)
    q, s = words_of(steps), scales_of(scale, n, dtype)
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    call = lambda: gp.gemm_rows4(code, m, n, k, group, x, k, q, s, y, n)  # noqa: E731
    call()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    call()
    stop.record()
    status_ok()
    assert torch.equal(y, want)
    # The finite sums take some 0.1 ms; one thread's whole sum after another, hundreds of ms.
    assert start.elapsed_time(stop) < 40
