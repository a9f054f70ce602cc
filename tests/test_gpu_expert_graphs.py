"""The expert-layer operators recorded in CUDA graphs: replays on other inputs,
after a launch that gave up, and next to larger calls on the same stream."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

pytestmark = pytest.mark.gpu


def test_sums_in_parts_after_a_replay_that_gave_up():
    # A weight gradient of 20000 rows, 64 x 128: one tile a matrix, an expert of
    # more than 3072 rows in parts of at most 2048.  The first replay's unit 0
    # stalls at its k-block 30 (2048 rows have 32) while the others finish their
    # parts; in the second, on other bounds, unit 0 has 28 k-blocks and no stall.
    R, K, N, E = 20000, 64, 128, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randint(-2, 3, (R, K), generator=g, device="cuda").half()
    dY = torch.randint(-1, 2, (R, N), generator=g, device="cuda").half()
    off = torch.tensor([0, R, R], dtype=torch.int32, device="cuda")
    dW = torch.empty(E, K, N, dtype=torch.float16, device="cuda")

    def call():
        gp.gemm_grouped_dw(gp.F16, R, N, K, E, X, K, dY, N, off, dW)

    def check():
        bounds = off.tolist()
        for e in range(E):
            x, d = X[bounds[e]:bounds[e + 1]].double(), dY[bounds[e]:bounds[e + 1]].double()
            # Whole numbers: the sums are exact in fp32, their rounding the only one.
            assert torch.equal(dW[e], (x.t() @ d).half()), e

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gp.gemmpipe_test_inject_stall(30, 50)
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert gp.gemmpipe_get_device_status() == gp.ERR_TIMEOUT
    for first in (3500, 808, 3600):
        off[1] = first
        dW.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert gp.gemmpipe_get_device_status() == gp.OK
        check()
