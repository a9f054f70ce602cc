"""Bounded waits of gemm_rows4 on tcgen05, in every size of group: a stage that never comes ends the call with a
status, and the next call is as ever.

A stage holds 128 of k (groups of 32: 64) and at most 8 blocks share a tile's stages, so that the first block has an
eighth of them at least."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import TYPES, rows4_case

pytestmark = pytest.mark.gpu

K = 8192


def stages(group):
    return K // (64 if group == 32 else 128)


def call_with_stall(type_, m, n, group, stage):
    x, q, s, want = rows4_case(type_, m, K, n, group)
    y = torch.empty(m, n, dtype=x.dtype, device="cuda")
    call = lambda: gp.gemm_rows4(TYPES[type_][0], m, n, K, group, x, K, q, s, y, n)  # noqa: E731
    gp.gemmpipe_test_inject_stall(stage, 20)
    call()
    status = gp.gemmpipe_get_device_status()
    if status == gp.OK:
        assert torch.equal(y, want)
    y.fill_(7)
    call()
    assert gp.gemmpipe_get_device_status() == gp.OK
    assert torch.equal(y, want)
    return status


@pytest.mark.parametrize("stage", [0, 1, 2, 7])
@pytest.mark.parametrize("m, n", [(64, 128), (20, 4096)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_a_stage_that_never_comes(type_, group, m, n, stage):
    assert stage < stages(group) // 8
    assert call_with_stall(type_, m, n, group, stage) == gp.ERR_TIMEOUT


@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_stage_that_there_is_not(group):
    assert call_with_stall("bf16", 64, 128, group, stages(group)) == gp.OK
