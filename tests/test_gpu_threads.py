"""Calls that several host threads make on one stream: each one's kernels are enqueued together, so that what they
keep in the stream's workspaces in between is their own, whoever else calls and however much larger a workspace
another call needs.  (A binding call runs without the interpreter's lock.)"""
from __future__ import annotations

import threading

import pytest
import torch

from software_pipelined_loop_gb300 import expert_layer as layer
from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import run_step, status_ok, step_case

pytestmark = pytest.mark.gpu

ROUNDS = 200


def at_once(*jobs):
    """Runs the jobs' steps, ROUNDS of each in a thread of its own on the default stream, from empty workspaces."""
    torch.cuda.synchronize()
    assert gp.gemmpipe_release_workspaces() is None
    start, failed = threading.Barrier(len(jobs)), []

    def run(job):
        try:
            start.wait(30)
            for i in range(ROUNDS):
                job(i)
        except Exception as error:  # noqa: BLE001 (reported below)
            failed.append(error)

    threads = [threading.Thread(target=run, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
        assert not t.is_alive()
    assert not failed, failed
    status_ok()


class Steps:
    """expert_step calls of one thread, with buffers of their own; every result is kept and looked at afterwards."""

    def __init__(self, t, sizes, four, key):
        self.cases = [(step_case("f16", t, 2, 6, c, h, True, four, key=key + i), h) for i, (c, h) in enumerate(sizes)]
        self.four, self.ys = four, []
        for args, h in self.cases:
            args["hidden"] = torch.empty(t * 2, (h + 7) // 8 * 8, dtype=torch.float16, device="cuda")
        self.ys = [torch.full_like(self.cases[i * len(self.cases) // ROUNDS][0]["x"], 7) for i in range(ROUNDS)]

    def __call__(self, i):
        args, h = self.cases[i * len(self.cases) // ROUNDS]  # (sizes grow with the rounds)
        run_step("f16", args, 6, h, self.four, y=self.ys[i], hidden=args["hidden"])

    def check(self):
        for i, y in enumerate(self.ys):
            assert torch.equal(y, self.cases[i * len(self.cases) // ROUNDS][0]["want"]), i


GROWING = [(64, 24), (136, 40), (264, 136), (520, 264), (776, 520)]


@pytest.mark.parametrize("four", [0, 32])
@pytest.mark.parametrize("first, second", [((3, GROWING[2:3]), (8, GROWING[2:3])), ((5, GROWING[1:2]), (8, GROWING)),
                                           ((40, GROWING[2:3]), (64, GROWING)), ((7, GROWING), (20, GROWING))])
def test_steps(first, second, four):
    a, b = Steps(*first, four, 1), Steps(*second, four, 50)
    at_once(a, b)
    a.check(), b.check()


def test_other_calls_that_use_the_workspace():
    """int8 products widened there, fp16 operands padded there, choices sorted there, odd experts' matrices copied
    there: two threads each, all exact."""
    g = torch.Generator(device="cuda").manual_seed(8)
    ints = lambda low, high, *s: torch.randint(low, high + 1, s, generator=g, device="cuda")  # noqa: E731
    jobs, checks = [], []

    def add(call, outputs, want):
        jobs.append(lambda i: call(outputs[i]))
        checks.append((outputs, want))

    for m, n, k in ((160, 136, 200), (300, 200, 400)):
        a, b = ints(-128, 127, m, k).to(torch.int8), ints(-128, 127, k, n).to(torch.int8)
        ys = [torch.zeros(m, n, dtype=torch.int32, device="cuda") for _ in range(ROUNDS)]
        add(lambda y, a=a, b=b, m=m, n=n, k=k: gp.gemm_s8s8s32(m, n, k, a, b, y), ys, (a.double() @ b.double()).int())
        a, b = ints(-4, 4, m, k + 1).half(), ints(-4, 4, k + 1, n + 1).half()
        ys = [torch.zeros(m, n + 1, device="cuda") for _ in range(ROUNDS)]
        add(lambda y, a=a, b=b, m=m, n=n, k=k: gp.gemm_f16f32(m, n + 1, k + 1, a, b, y), ys, a.float() @ b.float())
        x, w = ints(-3, 3, m, 41).half(), ints(-3, 3, 2, 41, 57).half()
        offsets = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
        want = torch.cat([x[:m // 3].double() @ w[0].double(), x[m // 3:].double() @ w[1].double()]).half()
        ys = [torch.zeros(m, 57, dtype=torch.float16, device="cuda") for _ in range(ROUNDS)]
        add(lambda y, x=x, w=w, m=m, o=offsets: gp.gemm_grouped(gp.F16, m, 57, 41, 2, x, 41, o, w, y, 57), ys, want)
    for tokens in (3000, 9000):
        ids = ints(-1, 15, tokens, 4).int()
        sorted_ = torch.sort(torch.where(ids < 0, 99, ids).flatten(), stable=True).indices.int()
        kept = int((ids >= 0).sum())
        outs = [tuple(torch.zeros(s, dtype=torch.int32, device="cuda") for s in (17, tokens * 4, tokens * 4))
                for _ in range(ROUNDS)]
        jobs.append(lambda i, outs=outs, ids=ids, tokens=tokens: gp.gemmpipe_route(tokens, 4, 16, ids, *outs[i]))
        checks.append(([o[1][:kept] for o in outs], sorted_[:kept]))
        want_offsets, want_slots, _ = layer.route(ids, 16)
        assert torch.equal(want_slots[:kept], sorted_[:kept]) and int(want_offsets[-1]) == kept
    at_once(*jobs)
    for outputs, want in checks:
        for y in outputs:
            assert torch.equal(y, want)
