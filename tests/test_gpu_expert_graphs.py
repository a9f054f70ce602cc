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


class Step:
    """Every call that uses a workspace: a sort of more than 2048 choices,
    products off 16-byte rows, a weight gradient in parts, one from 8-bit rows.
    Whole numbers throughout, small enough that every sum is exact in fp32 and
    every result but the weight gradients' rounding is exact."""

    def __init__(self, T, K, N, E=3, k=2):
        self.T, self.K, self.N, self.E, self.k, R = T, K, N, E, k, T * k
        new = lambda *s, ty=torch.float16: torch.empty(*s, dtype=ty, device="cuda")  # noqa: E731
        i32 = torch.int32
        self.ids, self.off, self.slots, self.rows = new(T, k, ty=i32), new(E + 1, ty=i32), new(R, ty=i32), new(R, ty=i32)
        self.X, self.Xs, self.W, self.dY = new(T, K), new(R, K), new(E, K, N), new(R, N)
        self.Y, self.dX, self.dW, self.dW8 = new(R, N), new(R, K), new(E, K, N), new(E, K, N)
        self.Q, self.S = new(R, K, ty=torch.int8), new(R, -(-K // 32), ty=torch.uint8)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        small = lambda t: t.copy_(torch.randint(-1, 2, t.shape, generator=g, device="cuda"))  # noqa: E731
        # Most choices are the first expert's, so that its sum is long.
        self.ids.copy_((torch.rand(self.T, self.k, generator=g, device="cuda") ** 6 * (self.E + 0.2)).int())
        for t in (self.X, self.W, self.dY):
            small(t)
        for t in (self.Y, self.dX, self.dW, self.dW8, self.Xs):
            t.fill_(7)
        torch.cuda.synchronize()

    def run(self, stream=None):
        R, N, K, E = self.T * self.k, self.N, self.K, self.E
        gp.gemmpipe_route(self.T, self.k, E, self.ids, self.off, self.slots, self.rows, stream)
        gp.gemmpipe_dispatch(gp.F16, self.T, self.k, K, self.X, K, self.rows, None, self.Xs, K, stream)
        gp.gemm_grouped(gp.F16, R, N, K, E, self.Xs, K, self.off, self.W, self.Y, N, stream)
        gp.gemm_grouped_dx(gp.F16, R, N, K, E, self.dY, N, self.off, self.W, self.dX, K, stream)
        gp.gemm_grouped_dw(gp.F16, R, N, K, E, self.Xs, K, self.dY, N, self.off, self.dW, stream)
        gp.gemmpipe_keep8(gp.F16, R, K, self.Xs, K, self.Q, self.S, stream)
        gp.gemm_grouped_dw8(gp.F16, R, N, K, E, self.Q, self.S, self.dY, N, self.off, self.dW8, stream)

    def check(self):
        torch.cuda.synchronize()
        assert gp.gemmpipe_get_device_status() == gp.OK
        flat = self.ids.view(-1)
        order = torch.sort(torch.where(flat < self.E, flat, self.E), stable=True).indices
        counts = torch.bincount(flat.clamp(max=self.E), minlength=self.E + 1)[:self.E].tolist()
        assert self.off.tolist() == [sum(counts[:e]) for e in range(self.E + 1)]
        Xs = self.X[order // self.k].double()
        Xs[sum(counts):] = 0
        assert torch.equal(self.Xs.double(), Xs)
        at = 0
        for e, n in enumerate(counts):
            s, w, d = slice(at, at + n), self.W[e].double(), self.dY[at:at + n].double()
            assert torch.equal(self.Y[s].double(), Xs[s] @ w) and torch.equal(self.dX[s].double(), d @ w.t())
            dw = (Xs[s].t() @ d).half()
            assert torch.equal(self.dW[e], dw) and torch.equal(self.dW8[e], dw), e
            at += n
        assert int(self.Y[at:].count_nonzero()) == int(self.dX[at:].count_nonzero()) == 0


@pytest.fixture
def warm():
    # Every kernel has run in the process, none on the tests' streams.
    step = Step(3000, 69, 75)
    step.fill(0)
    step.run()
    step.check()


def recorded(step, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step.run(stream)
    return graph


def replayed(graph, step, seed):
    step.fill(seed)
    graph.replay()
    step.check()


def test_recording_on_a_stream_without_workspaces(warm):
    step = Step(4100, 69, 75)
    step.fill(1)
    graph = recorded(step, torch.cuda.Stream())
    for seed in range(2, 6):
        replayed(graph, step, seed)


def test_larger_calls_after_recording(warm):
    # The stream's workspaces grow; the recorded step keeps those it has.
    side = torch.cuda.Stream()
    small, large = Step(2500, 69, 75), Step(6000, 133, 141)
    small.fill(1)
    small.run(side)
    small.check()
    graph = recorded(small, side)
    replayed(graph, small, 2)
    for seed in range(3, 7):
        large.fill(seed)
        large.run(side)
        large.check()
        replayed(graph, small, seed)
    gp.gemmpipe_release_workspaces()  # what the recorded step uses too: it is not replayed again
    large.fill(8)
    large.run(side)
    large.check()


def test_recording_a_larger_step_than_the_stream_has_run(warm):
    side = torch.cuda.Stream()
    small, large = Step(2500, 69, 75), Step(6000, 133, 141)
    small.fill(1)
    small.run(side)
    small.check()
    large.fill(2)
    graph = recorded(large, side)
    for seed in range(3, 6):
        replayed(graph, large, seed)
        small.fill(seed)
        small.run(side)
        small.check()
