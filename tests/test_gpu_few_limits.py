"""The few-token operators at the ends of their ranges, and next to other calls:
addresses past 2^31 elements, the largest tables, the longest and shortest
sums, the workspace that calls of one stream share."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import few_tokens as few
from software_pipelined_loop_gb300 import gemmpipe as gp
from test_gpu_few import generator, ints, rows4_case, run_step, scales_of, status_ok, step_case, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 12])
def test_experts_behind_2_31_elements(t):
    """The last of 600 experts of 2048 x 2048 (2.5e9 elements) as the only one of a call with that one."""
    e, c = 600, 2048
    g = generator("far", t)
    one = [(torch.randn(1, c, c, generator=g, device="cuda") * c ** -0.5).bfloat16() for _ in range(2)]
    x = torch.randn(t, c, generator=g, device="cuda").bfloat16()
    ids = torch.zeros(t, 1, dtype=torch.int32, device="cuda")
    weights = torch.ones(t, 1, device="cuda")
    want = few.expert_step(x, ids, weights, *one)
    far = []
    for w in one:
        far.append(torch.zeros(e, c, c, dtype=torch.bfloat16, device="cuda"))
        far[-1][-1] = w[0]
    # (more experts may be split otherwise among blocks: sums in another order, each rounded as far as here)
    near = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm()) <= 2 * 2.0 ** -8  # noqa: E731
    assert near(few.expert_step(x, ids + (e - 1), weights, *far), want)
    packed, packed_one = [few.pack4(w) for w in far], [few.pack4(w) for w in one]
    for a, b in zip(packed, packed_one):
        assert torch.equal(a.words[-1:], b.words) and torch.equal(a.scales[-1:], b.scales)
    del far
    assert torch.equal(few.unpack4(packed[0])[-1:], few.unpack4(packed_one[0]))
    assert near(few.expert_step(x, ids + (e - 1), weights, *packed), few.expert_step(x, ids, weights, *packed_one))
    status_ok()


def test_words_behind_2_31():
    """Words of a matrix of 2^24 + 8 rows of 1024: 2^31 + 1024 of them."""
    k, n, group = (1 << 24) + 8, 1024, 128
    words = torch.full((1, k // 8, n), -2004318072, dtype=torch.int32, device="cuda")  # 0x88888888: zeros
    scales = torch.ones(1, -(-k // group), n, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(20, k, dtype=torch.bfloat16, device="cuda")
    x[:, -2:] = torch.arange(1, 21, device="cuda")[:, None]
    words[0, -1] += (1 << 12) + (3 << 28)  # rows 6 and 7 of the last words
    m = few.Packed4(words, scales, k, n, group)
    want = (x[:, -2:].double() @ torch.tensor([[1.0], [3.0]], device="cuda").double()).bfloat16().expand(20, n)
    for rows in (1, 20):
        assert torch.equal(few.rows4(x[:rows], m), want[:rows])
    status_ok()


@pytest.mark.parametrize("four", [0, 32])
def test_largest_tables(four):
    t, k, e, c, h = 64, 64, 1024, 24, 16
    args = step_case("f16", t, k, e, c, h, True, four)
    y = run_step("f16", args, e, h, four)
    status_ok()
    assert torch.equal(y, args["want"])


@pytest.mark.parametrize("m", [1, 8, 40])
@pytest.mark.parametrize("k, n", [(1 << 20, 3), (262147, 17), (9, 300001), (1, 1 << 20)])
def test_long_and_short_sums(m, k, n):
    g = generator("long", m, k, n)
    x = (torch.rand(m, k, generator=g, device="cuda") < 0.05).double()  # sums of whole numbers below 2^24
    steps = ints(g, -8, 7, 1, k, n)
    scale = torch.ones(1, -(-k // 64), n, dtype=torch.float64, device="cuda")
    y = torch.empty(m, n, dtype=torch.float16, device="cuda")
    gp.gemm_rows4(gp.F16, m, n, k, 64, x.half(), k, words_of(steps), scales_of(scale, n, torch.float16), y, n)
    status_ok()
    assert torch.equal(y, (x @ steps[0]).half())


@pytest.mark.parametrize("four", [0, 64])
@pytest.mark.parametrize("t", [3, 20])
@pytest.mark.parametrize("c, h", [(8, 4100), (20000, 8), (1, 4099)])
def test_narrow_layers(four, t, c, h):
    args = step_case("bf16", t, 2, 3, c, h, False, four)
    y = run_step("bf16", args, 3, h, four)
    status_ok()
    assert torch.equal(y, args["want"])


def test_too_many_units_are_refused():
    """1024 experts' 64-column blocks of 2^31 - 1024 columns cannot be counted: refused before any launch."""
    t, k, e, c, h = 64, 64, 1024, 1, 2 ** 31 - 1024
    any_ = torch.zeros(4096, device="cuda")
    with pytest.raises(gp.GemmpipeError) as error:
        gp.gemmpipe_expert_step(gp.BF16, t, k, e, c, h, any_, c, any_, any_, any_, any_, None, any_, any_, c)
    assert error.value.status == gp.ERR_INVALID_VALUE


def test_calls_of_a_stream_share_its_workspace():
    """Rows by choice, widened operands and stream-K sums one after the other, eagerly and in a graph."""
    args = step_case("f16", 40, 4, 8, 264, 136, True)
    x4, q4, s4, want4 = rows4_case("f16", 40, 640, 200, 32)
    a = torch.randint(-128, 128, (300, 400), device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (400, 200), device="cuda", dtype=torch.int8)
    want8 = (a.double() @ b.double()).int()
    y = torch.empty(40, 264, dtype=torch.float16, device="cuda")
    y4 = torch.empty(40, 200, dtype=torch.float16, device="cuda")
    y8 = torch.empty(300, 200, dtype=torch.int32, device="cuda")
    hidden = torch.empty(160, 136, dtype=torch.float16, device="cuda")

    def all_of_them():
        for _ in range(3):
            gp.gemm_s8s8s32(300, 200, 400, a, b, y8)
            run_step("f16", args, 8, 136, 0, y=y, hidden=hidden)
            gp.gemm_rows4(gp.F16, 40, 200, 640, 32, x4, 640, q4, s4, y4, 200)

    def check():
        torch.cuda.synchronize()
        assert torch.equal(y, args["want"]) and torch.equal(y4, want4) and torch.equal(y8, want8)
        status_ok()
        y.fill_(3), y4.fill_(3), y8.fill_(3)

    all_of_them()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_of_them()
    for _ in range(5):
        graph.replay()
    check()


def test_choices_written_just_before():
    """The choices, weights and rows come from kernels of the same stream right before each call."""
    e, c, h = 8, 200, 96
    for t in (3, 20):
        cases = [step_case("f16", t, 2, e, c, h, True, key=10 + i) for i in range(6)]
        held = {n: v.clone() for n, v in cases[0].items()}
        got = []
        for case in cases * 5:
            for n in ("x", "ids", "weights", "w1", "w2", "w3"):
                held[n].copy_(case[n])
            got.append(run_step("f16", held, e, h, 0))
        for y, case in zip(got, cases * 5):
            assert torch.equal(y, case["want"])
    status_ok()


@pytest.mark.parametrize("t", [12, 13, 16, 17])
@pytest.mark.parametrize("k, e, c, h", [(8, 5, 320, 200), (3, 40, 65, 264), (64, 3, 40, 24)])
@pytest.mark.parametrize("four", [0, 32, 128])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_tokens_around_the_ways_of_summing(type_, four, k, e, c, h, t):
    args = step_case(type_, t, k, e, c, h, True, four)
    y = run_step(type_, args, e, h, four)
    status_ok()
    assert torch.equal(y, args["want"])


@pytest.mark.parametrize("m", [1, 9, 12, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_subnormal_scales(type_, group, m):
    """Scales below the type's normal numbers are taken as they are, and weights made of them."""
    k, n = 520, 136
    g = generator("subnormal", type_, group, m)
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[type_]
    code = {"f16": gp.F16, "bf16": gp.BF16}[type_]
    least, lift = (2.0 ** -24, 1.0) if type_ == "f16" else (2.0 ** -133, 2.0 ** 100)
    x, steps = ints(g, -2, 2, m, k) * lift, ints(g, -8, 7, 1, k, n)
    scale = ints(g, 0, 100, 1, -(-k // group), n) * least
    want = (x @ (steps * scale.repeat_interleave(group, 1)[:, :k])[0]).to(dtype)  # exact sums, one rounding
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    gp.gemm_rows4(code, m, n, k, group, x.to(dtype), k, words_of(steps), scales_of(scale, n, dtype), y, n)
    status_ok()
    assert torch.equal(y, want)


def test_subnormal_scales_of_the_step():
    """The same through the whole layer: fp16 scales of 2^-24 to 2^-18 in the second product."""
    t, k, e, c, h = 9, 2, 4, 96, 64
    args = step_case("f16", t, k, e, c, h, True, 32)
    q2, s2 = args["w2"]
    args["w2"] = q2, s2 * 2.0 ** -20
    y = run_step("f16", args, e, h, 32)
    status_ok()
    want = args["want"].double() * 2.0 ** -20
    # (want is rounded once to 11 bits, the result again, to multiples of 2^-24)
    assert bool(((y.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25).all())


@pytest.mark.parametrize("t", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("four", [0, 64])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_few_tokens_are_rounded_once(type_, four, t):
    """Up to 8 tokens: the distance from the exact result is that of its rounding."""
    e, c, h, k = 6, 520, 264, 3
    g = generator("once", type_, four, t)
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[type_]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, weights = rand(t, c).to(dtype), torch.rand(t, k, generator=g, device="cuda")
    ids = torch.randint(0, e, (t, k), generator=g, device="cuda").int()
    ws = [(rand(e, a, b) * a ** -0.5).to(dtype) for a, b in ((c, h), (h, c), (c, h))]
    if four:
        ws = [few.pack4(w, four) for w in ws]
        exact = []
        for m in ws:
            q = torch.stack([(m.words >> (4 * [0, 2, 4, 6, 1, 3, 5, 7].index(r))) & 15 for r in range(8)], 2).flatten(1, 2)
            s = m.scales.double().repeat_interleave(four, 1)[:, :m.inner, :m.outer]
            exact.append((q[:, :m.inner, :m.outer].double() - 8) * s)
    else:
        exact = [w.double() for w in ws]
    want = torch.zeros(t, c, dtype=torch.float64, device="cuda")
    for i in range(t):
        for j in range(k):
            e1, e2, e3 = (w[int(ids[i, j])] for w in exact)
            hidden = torch.nn.functional.silu(x[i].double() @ e1) * (x[i].double() @ e3)
            want[i] += weights[i, j].double() * (hidden @ e2)
    y = few.expert_step(x, ids, weights, *ws)
    status_ok()
    once = float((want.to(dtype).double() - want).norm())
    # (besides: fp32 sums and the activation, some 2^-20 of the values, next to 2^-9 or 2^-12)
    assert float((y.double() - want).norm()) <= 1.05 * once
