"""gemm_rows4 with more than 16 rows (the tcgen05 kernel): sizes around its tiles,
stages and clusters against exact results, graphs, and its bounded waits."""
from __future__ import annotations

import math

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import TYPES, ints, generator, rows4_case, scales_of, words_of, off_by, pitched

pytestmark = pytest.mark.gpu


def run(type_, m, k, n, group):
    x, q, s, want = rows4_case(type_, m, k, n, group)
    room = torch.full((m * n + 16,), 7, dtype=x.dtype, device="cuda")
    y = room[8:8 + m * n].view(m, n)
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k, q, s, y, n)
    assert gp.gemmpipe_get_device_status() == gp.OK
    assert torch.equal(y, want)
    assert bool((room[:8] == 7).all()) and bool((room[8 + m * n:] == 7).all())


# Rows around 32; k around the 16, 64 and 128 of its steps, tiles and stages, and
# more stages than its rings have; columns around a tile; one tile and a cluster
# of eight, more tiles than run at once.
@pytest.mark.parametrize("m, k, n", [
    (17, 8, 128), (31, 16, 127), (32, 24, 129), (33, 64, 1), (48, 72, 130), (63, 128, 4), (64, 136, 260), (64, 192, 128),
    (40, 256, 300), (18, 1000, 126), (64, 1024, 131), (33, 2048, 128), (17, 4096, 257), (64, 5000, 96), (32, 16384, 64),
    (20, 40, 40000), (64, 256, 20500)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_exact(type_, group, m, k, n):
    run(type_, m, k, n, group)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("pad_x, pad_y, shift", [(8, 0, 0), (0, 3, 8), (64, 1, 16)])
def test_pitches(type_, pad_x, pad_y, shift):
    m, k, n, group = 37, 328, 150, 64
    x, q, s, want = rows4_case(type_, m, k, n, group)
    x = off_by(pitched(x, pad_x), shift)
    y = torch.full((m, n + pad_y), 7, dtype=x.dtype, device="cuda")
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k + pad_x, q, s, y, n + pad_y)
    assert gp.gemmpipe_get_device_status() == gp.OK
    assert torch.equal(y[:, :n], want) and bool((y[:, n:] == 7).all())


@pytest.mark.parametrize("type_", TYPES)
def test_the_other_kernel_gives_the_same(type_):
    # Rows off 16-byte boundaries take the warp-level kernel: equal on exact values.
    m, k, n, group = 50, 640, 200, 32
    x, q, s, want = rows4_case(type_, m, k, n, group)
    y = torch.empty(m, n, dtype=x.dtype, device="cuda")
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, off_by(x, 1), k, q, s, y, n)
    assert torch.equal(y, want)
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k, q, s, y, n)
    assert torch.equal(y, want)


def test_captured_with_new_rows():
    m, k, n, group = 64, 1024, 512, 128
    g = generator("captured wide")
    steps, scale = ints(g, -8, 7, 1, k, n), torch.ones(1, k // group, n, device="cuda").double()
    q, s = words_of(steps), scales_of(scale, n, torch.bfloat16)
    xs = [ints(g, -2, 2, m, k) for _ in range(3)]
    x, y = xs[0].bfloat16(), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    call = lambda: gp.gemm_rows4(gp.BF16, m, n, k, group, x, k, q, s, y, n)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for v in xs:
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, (v @ steps[0]).bfloat16())


def test_streams_at_once():
    # Two of these kernels and a grouped product, which all want tensor memory.
    cases = [rows4_case("f16", m, 2048, n, 64) for m, n in ((64, 4096), (24, 1024))]
    streams = [torch.cuda.Stream() for _ in range(3)]
    x, w = torch.ones(512, 256, device="cuda").half(), torch.ones(4, 256, 512, device="cuda").half()
    offsets = torch.tensor([0, 100, 100, 300, 512], dtype=torch.int32, device="cuda")
    ys = [torch.empty(c[3].shape, dtype=torch.float16, device="cuda") for c in cases]
    yg = torch.empty(512, 512, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        for (xc, q, s, want), y, st in zip(cases, ys, streams):
            gp.gemm_rows4(gp.F16, want.shape[0], want.shape[1], 2048, 64, xc, 2048, q, s, y, want.shape[1], stream=st)
        gp.gemm_grouped(gp.F16, 512, 512, 256, 4, x, 256, offsets, w, yg, 512, stream=streams[2])
    torch.cuda.synchronize()
    for c, y in zip(cases, ys):
        assert torch.equal(y, c[3])
    assert bool((yg == 256).all()) and gp.gemmpipe_get_device_status() == gp.OK


@pytest.mark.parametrize("k, n", [(4096, 4096), (1024, 128)])
@pytest.mark.parametrize("stage", [0, 1, 3])
def test_a_stage_that_never_comes(k, n, stage):
    x, q, s, want = rows4_case("bf16", 64, k, n, 32)
    y = torch.empty(64, n, dtype=torch.bfloat16, device="cuda")
    gp.gemmpipe_test_inject_stall(stage, 20)
    gp.gemm_rows4(gp.BF16, 64, n, k, 32, x, k, q, s, y, n)
    in_range = stage < (k // 128 if n > 128 else 1) or stage == 0
    status = gp.gemmpipe_get_device_status()
    if in_range:
        assert status == gp.ERR_TIMEOUT
    # The next call is as ever.
    gp.gemm_rows4(gp.BF16, 64, n, k, 32, x, k, q, s, y, n)
    assert gp.gemmpipe_get_device_status() == gp.OK
    assert torch.equal(y, want)


@pytest.mark.parametrize("m, k, n", [(9, 4096, 300), (16, 136, 130), (12, 2048, 1024), (10, 64, 40), (9, 8, 5)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_nine_rows_and_more(type_, group, m, k, n):
    run(type_, m, k, n, group)


@pytest.mark.parametrize("m", [20, 64])
@pytest.mark.parametrize("k", [160, 4096])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_infinities_and_large_scales(type_, group, k, m):
    """What is not finite, and scales whose weights are past the type's largest value, give what the formula
    gives."""
    n = 200
    g = generator("large", type_, group, k, m)
    dtype = TYPES[type_][1]
    x, steps = ints(g, -2, 2, m, k), ints(g, -8, 7, 1, k, n)
    scale = torch.exp2(ints(g, -2, 1, 1, -(-k // group), n))
    top = torch.finfo(dtype).max
    x[3, 5], x[4, 6], x[5, k - 1], x[5, 0] = math.inf, -math.inf, math.inf, math.inf
    x[6, 70], x[7] = math.nan, math.nan
    x[8, 2:] = 0
    scale[0, 1, 11], scale[0, 0, 12], scale[0, -1, 13] = math.inf, math.nan, -math.inf
    scale[0, :, 14] = top / 4              # times 7: past the largest value, times 2 ^ -13: not
    scale[0, :, 15] = -top
    x[9] *= 2.0 ** -13
    scale, x = scale.to(dtype).double(), x.to(dtype).double()
    parts = torch.stack([x[:, a:a + group] @ steps[0, a:a + group] for a in range(0, k, group)])
    want = (parts.float() * scale[0][:, None].float()).double().sum(0).float().to(dtype)
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x.to(dtype), k, words_of(steps), scales_of(scale, n, dtype), y, n)
    assert gp.gemmpipe_get_device_status() == gp.OK
    # (whole numbers, in row 9 times 2^-13, with sums below 2^24 of the scales' last bits: exact in fp32; sums of
    # infinities do not depend on the order)
    same = (y == want) | (y.isnan() & want.isnan())
    plain = torch.ones(n, dtype=torch.bool, device="cuda")
    plain[14:16] = False
    assert bool(same[:, plain].all())
    assert bool(same[9].all()) and bool(y[9, 14:16].isfinite().all())
