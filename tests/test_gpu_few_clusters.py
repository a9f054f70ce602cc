"""Blocks of a cluster that exchange their sums several times in a unit of work (more than 8 rows of an expert): the
sums of one exchange are read before those of the next are written over them."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import rows4_case, run_step, status_ok, step_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t, e", [(16, 1), (32, 1), (64, 1), (64, 2)])
@pytest.mark.parametrize("four", [0, 32])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_rows_of_one_expert(type_, four, t, e):
    # 64 columns, sums of 2048: eight blocks a unit, up to four exchanges each.
    c, h = 2048, 64
    args = step_case(type_, t, 1, e, c, h, True, four, dropped=0.0)
    ys = [run_step(type_, args, e, h, four) for _ in range(50)]
    status_ok()
    for y in ys:
        assert torch.equal(y, args["want"])


@pytest.mark.parametrize("m", [9, 16, 33, 64])
def test_rows_off_boundaries(m):
    # (X off 16-byte boundaries: these rows do not take tcgen05)
    k, n, group = 4104, 60, 64
    x, q, s, want = rows4_case("f16", m, k, n, group)
    room = torch.empty(m * k + 1, dtype=x.dtype, device="cuda")
    room[1:] = x.flatten()
    ys = [torch.empty(m, n, dtype=x.dtype, device="cuda") for _ in range(50)]
    for y in ys:
        gp.gemm_rows4(gp.F16, m, n, k, group, room[1:].view(m, k), k, q, s, y, n)
    status_ok()
    for y in ys:
        assert torch.equal(y, want)
