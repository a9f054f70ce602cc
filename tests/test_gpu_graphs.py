"""GEMM calls recorded in CUDA graphs: every replay works on the operands'
values of its own time."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe

pytestmark = pytest.mark.gpu

# Plans that split tiles over several units (stream-K), one that does not, and misaligned operands.
SHAPES = [(256, 128, 8192), (512, 512, 4096), (300, 260, 5000), (1000, 40, 20000), (2048, 2048, 512), (333, 517, 4099)]


@pytest.mark.parametrize("dtype", ["f16", "s8"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_replays_follow_the_operands(shape, dtype):
    M, N, K = shape
    s8 = dtype == "s8"
    if shape in SHAPES[:4]:
        assert gemmpipe.gemmpipe_plan(0 if s8 else 1, M, N, K)["split_tiles"] > 0
    A = torch.empty(M, K, dtype=torch.int8 if s8 else torch.float16, device="cuda")
    B = torch.empty(K, N, dtype=A.dtype, device="cuda")
    C = torch.empty(M, N, dtype=torch.int32 if s8 else torch.float32, device="cuda")
    call = gemmpipe.gemm_s8s8s32 if s8 else gemmpipe.gemm_f16f32

    def fill(seed):
        # Whole numbers whose sums are exact in fp32.
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (A, B):
            t.copy_(torch.randint(-3, 4, t.shape, generator=g, device="cuda"))
        C.fill_(-1)
        torch.cuda.synchronize()
        return (A.double() @ B.double()).to(C.dtype)

    side = torch.cuda.Stream()
    want = fill(0)
    call(M, N, K, A, B, C, side)
    torch.cuda.synchronize()
    assert torch.equal(C, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(M, N, K, A, B, C, side)
    for seed in range(1, 13):
        want = fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want), seed
        if seed % 4 == 0:  # calls between the replays
            want = fill(100 + seed)
            call(M, N, K, A, B, C, side)
            torch.cuda.synchronize()
            assert torch.equal(C, want)
    # Replays one behind the other, with nothing between them.
    want = fill(50)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, want)
    assert gemmpipe.gemmpipe_get_device_status() == gemmpipe.OK
