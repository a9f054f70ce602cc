"""Every value of the types through gemmpipe_pack4: the kernel corrects products by their remainders instead of
dividing, which has to give the rounded quotients of the formula for all of them."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import status_ok
from test_gpu_pack4 import TYPES, formula, unpacked_words

pytestmark = pytest.mark.gpu


def pack(w, group):
    e, k, n = w.shape
    n4 = (n + 3) // 4 * 4
    q = torch.empty(e, -(-k // 8), n4, dtype=torch.int32, device="cuda")
    s = torch.empty(e, -(-k // group), n4, dtype=w.dtype, device="cuda")
    gp.gemmpipe_pack4({torch.float16: gp.F16, torch.bfloat16: gp.BF16}[w.dtype], e, k, n, group, w, q, s)
    status_ok()
    return unpacked_words(q, k, n)[:, :k, :n], s[:, :, :n]


def check(w, group):
    got_q, got_s = pack(w, group)
    want_q, want_s, _ = formula(w, group)
    assert torch.equal(got_s, want_s)
    assert torch.equal(got_q, want_q)


@pytest.mark.parametrize("dtype", TYPES)
def test_every_scale(dtype):
    # A group for each finite magnitude, of either sign, and it alone in its group.
    last = int(torch.tensor([torch.finfo(dtype).max], dtype=dtype).view(torch.int16))
    bits = torch.arange(last + 1, dtype=torch.int32, device="cuda").to(torch.int16)
    w = bits.view(dtype)
    check(torch.stack([w, -w])[:, None, :].contiguous(), 32)


@pytest.mark.parametrize("binade", [0, -3, 9])
@pytest.mark.parametrize("dtype", TYPES)
def test_every_quotient(dtype, binade):
    # Each significand as a group's largest magnitude, with every smaller value of six binades, of either sign.
    steps = round(1 / torch.finfo(dtype).eps)  # significands of a binade
    top = (1 + torch.arange(steps, device="cuda").double() / steps) * 2.0 ** binade
    values = torch.cat([top * 2.0 ** -i for i in range(7)])
    values = torch.cat([values, -values])
    group = 128
    rows = -(-len(values) // (group - 1))
    values = torch.nn.functional.pad(values, (0, rows * (group - 1) - len(values))).view(rows, group - 1)
    w = torch.zeros(rows, group, steps, dtype=torch.float64, device="cuda")
    w[:, 0] = top
    w[:, 1:] = torch.where(values[:, :, None].abs() <= top, values[:, :, None], 0.0)
    w = w.to(dtype)
    assert torch.equal(w[0, 0].double(), top)
    check(w.view(1, rows * group, steps), group)
