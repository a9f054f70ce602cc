"""The few-token operators against plain forms in 64 bits.

Most cases are made of small whole numbers: every product and sum is exact in
fp32, the activation's argument is at least 20 (where silu(a) = a in fp32) and
hidden values are exact in 16 bits, so the result is the exact one rounded once
and has to be equal, bit for bit.  Random values are held to a bound."""
from __future__ import annotations

import math
import zlib

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

pytestmark = pytest.mark.gpu

TYPES = {"f16": (gp.F16, torch.float16), "bf16": (gp.BF16, torch.bfloat16)}
ROW_OF_NIBBLE = [0, 2, 4, 6, 1, 3, 5, 7]


def generator(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def ints(g, low, high, *shape):
    return torch.randint(low, high + 1, shape, generator=g, device="cuda").double()


def words_of(steps):
    """Words of whole numbers from -8 to 7 (experts x K x N); past K and N: anything (here 5)."""
    e, k, n = steps.shape
    full = torch.full((e, -(-k // 8) * 8, -(-n // 4) * 4), 5, dtype=torch.int64, device="cuda")
    full[:, :k, :n] = steps.long() + 8
    blocks = full.view(e, -1, 8, full.shape[2])
    word = sum(blocks[:, :, row] << (4 * i) for i, row in enumerate(ROW_OF_NIBBLE))
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32).contiguous()


def scales_of(values, n, dtype):
    """Scales (experts x groups x N) in their layout; past N: NaN."""
    e, groups, _ = values.shape
    out = torch.full((e, groups, -(-n // 4) * 4), math.nan, dtype=dtype, device="cuda")
    out[:, :, :n] = values.to(dtype)
    return out


def off_by(t, elements):
    """A copy of t that starts `elements` elements behind a 256-byte boundary."""
    room = torch.empty(t.numel() + elements, dtype=t.dtype, device="cuda")
    room[elements:] = t.reshape(-1)
    return room[elements:].view(t.shape)


def pitched(t, pad, fill=math.nan):
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide


def status_ok():
    assert gp.gemmpipe_get_device_status() == gp.OK


# ------------------------------------------------------------------- rows4


def rows4_case(type_, m, k, n, group):
    g = generator("rows4", type_, m, k, n, group)
    dtype = TYPES[type_][1]
    x, steps = ints(g, -2, 2, m, k), ints(g, -8, 7, 1, k, n)
    scale = torch.exp2(ints(g, -2, 1, 1, -(-k // group), n))
    values = steps * scale.repeat_interleave(group, 1)[:, :k]
    # |x w| <= 2 * 16, in quarters: below 2^24 quarters up to 2^17 products.
    return x.to(dtype), words_of(steps), scales_of(scale, n, dtype), (x @ values[0]).to(dtype)


ROWS4 = [(1, 2048, 256, 128), (1, 8, 4, 32), (1, 1, 1, 32), (1, 4096, 64, 64), (2, 33, 65, 32), (3, 4107, 301, 64),
         (7, 31, 30, 32), (8, 512, 192, 128), (9, 130, 67, 128), (16, 1000, 129, 64), (17, 264, 200, 32),
         (32, 640, 96, 64), (33, 257, 130, 32), (40, 96, 72, 128), (63, 127, 66, 32), (64, 1024, 128, 32),
         (64, 16, 1000, 32), (5, 20000, 40, 128), (1, 64, 20000, 64), (1, 32, 8, 32), (8, 288, 60, 32)]


@pytest.mark.parametrize("m, k, n, group", ROWS4)
@pytest.mark.parametrize("type_", TYPES)
def test_rows4_exact(type_, m, k, n, group):
    x, q, s, want = rows4_case(type_, m, k, n, group)
    y = torch.full((m, n), 7, dtype=x.dtype, device="cuda")
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k, q, s, y, n)
    status_ok()
    assert torch.equal(y, want)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("m", [1, 6, 21])
@pytest.mark.parametrize("shift, pad_x, pad_y", [(1, 0, 0), (0, 1, 3), (3, 5, 0), (8, 8, 8), (0, 16, 1)])
def test_rows4_places(type_, m, shift, pad_x, pad_y):
    # Rows at any place and pitch; what lies between the rows of X is not used, of Y not written.
    k, n, group = 200, 75, 64
    x, q, s, want = rows4_case(type_, m, k, n, group)
    x = off_by(pitched(x, pad_x), shift)
    room = torch.full((m * (n + pad_y) + 16,), 7, dtype=x.dtype, device="cuda")
    y = room[shift:shift + m * (n + pad_y)].view(m, n + pad_y)
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k + pad_x, q, s, y, n + pad_y)
    status_ok()
    assert torch.equal(y[:, :n], want)
    assert bool((y[:, n:] == 7).all()) and bool((room[:shift] == 7).all())
    assert bool((room[shift + m * (n + pad_y):] == 7).all())


def test_rows4_no_products():
    y = torch.full((3, 10), 7, dtype=torch.float16, device="cuda")
    gp.gemm_rows4(gp.F16, 3, 8, 0, 32, None, 0, None, None, y, 10)
    status_ok()
    assert bool((y[:, :8] == 0).all()) and bool((y[:, 8:] == 7).all())


@pytest.mark.parametrize("type_", TYPES)
def test_rows4_infinities_stay_in_their_row_and_column(type_):
    m, k, n, group = 11, 96, 40, 32
    x, q, s, want = rows4_case(type_, m, k, n, group)
    x[4, 7] = math.inf
    s[0, 1, 9] = math.nan
    y = torch.empty(m, n, dtype=x.dtype, device="cuda")
    gp.gemm_rows4(TYPES[type_][0], m, n, k, group, x, k, q, s, y, n)
    status_ok()
    assert bool(y[:, 9].isnan().all())
    assert not bool(torch.isfinite(y[4]).any())
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[4], keep[:, 9] = False, False
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("m, k, n, group", [(1, 4096, 333, 128), (13, 1111, 150, 32), (64, 768, 80, 64)])
def test_rows4_random(type_, m, k, n, group):
    g = generator("random", type_, m, k, n)
    code, dtype = TYPES[type_]
    x = torch.randn(m, k, generator=g, device="cuda").to(dtype)
    steps = ints(g, -8, 7, 1, k, n)
    scale = (torch.rand(1, -(-k // group), n, generator=g, device="cuda") + 0.1).to(dtype)
    values = (steps * scale.double().repeat_interleave(group, 1)[:, :k])[0]
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    gp.gemm_rows4(code, m, n, k, group, x, k, words_of(steps), scales_of(scale, n, dtype), y, n)
    status_ok()
    want, size = x.double() @ values, x.double().abs() @ values.abs()
    # One rounding to 16 bits, and fp32 sums: a product goes through at most
    # k / 16 + 80 additions (16 a matrix instruction, then scales, warps, blocks),
    # each off by at most 2^-22 of what has been summed, and sums are at most `size`.
    bound = torch.finfo(dtype).eps / 2 * want.abs() + (k / 16 + 80) * 2.0 ** -22 * size
    assert bool(((y.double() - want).abs() <= bound * (1 + 1e-3)).all())


# ------------------------------------------------------------ expert layer


def step_case(type_, t, k, e, c, h, gated, four=0, dropped=0.2, key=0):
    """Inputs whose results are exact (see above), and the result in 64 bits."""
    g = generator("step", type_, t, k, e, c, h, gated, four, key)
    dtype = TYPES[type_][1]
    x = ints(g, -1, 1, t, c)
    x[:, 0] = 1
    group = four or 32
    first = 56 if four else 64  # a = first +- 32, or more sure of it: 16 ones at most on either side

    def sparse(e, k_, n, ones, lead):
        # Up to `ones` entries of -1 or 1 a column behind the first group, `lead` in row 0.
        w = torch.zeros(e, k_, n, dtype=torch.float64, device="cuda")
        if k_ > group:
            at = torch.randint(group, k_, (e, ones, n), generator=g, device="cuda")
            w.scatter_(1, at, ints(g, 0, 1, e, ones, n) * 2 - 1)
        w[:, 0] = lead
        return w

    w1 = sparse(e, c, h, 32, first)
    w2 = ints(g, -2, 2, e, h, c)
    w3 = sparse(e, c, h, 1, 1) if gated else None
    ids = torch.randint(0, e, (t, k), generator=g, device="cuda")
    ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < dropped, torch.where(ids % 2 == 0, -1, e), ids)
    weights = (ints(g, -8, 8, t, k) / 8).float()
    a = torch.einsum("tc,ech->teh", x, w1)
    assert float(a.min()) >= 20
    if gated:
        a = a * torch.einsum("tc,ech->teh", x, w3)
    assert float(a.abs().max()) <= 256
    factor = torch.zeros(t, e, dtype=torch.float64, device="cuda")
    for j in range(k):
        ok = (ids[:, j] >= 0) & (ids[:, j] < e)
        factor[ok.nonzero()[:, 0], ids[ok, j]] += weights[ok, j].double()
    # (whole numbers below 256 x 2 x h and weights of eighths: exact in fp32 up to 2^24)
    assert 256 * 2 * h * k * 8 < 2 ** 24 or float((factor.abs()[:, :, None] * a.abs()).sum((1, 2)).max()) * 2 * 8 < 2 ** 24
    want = torch.einsum("te,teh,ehc->tc", factor, a, w2)
    weights = torch.where((ids < 0) | (ids >= e), math.nan, weights)  # not to be used
    args = {"x": x.to(dtype), "ids": ids.int(), "weights": weights, "want": want.to(dtype)}
    for name, w in (("1", w1), ("2", w2), ("3", w3)):
        if w is None or not four:
            args["w" + name] = None if w is None else w.to(dtype)
            continue
        scale = torch.ones(e, -(-w.shape[1] // group), w.shape[2], dtype=torch.float64, device="cuda")
        if name == "1":
            scale[:, 0] = 8
        steps = w / scale.repeat_interleave(group, 1)[:, :w.shape[1]]
        args["w" + name] = (words_of(steps), scales_of(scale, w.shape[2], dtype))
    if four and not gated:
        args["w3"] = (None, None)
    return args


def run_step(type_, args, e, h, four, y=None, hidden=None, **changes):
    a = args | changes
    code, (t, c), k = TYPES[type_][0], a["x"].shape, a["ids"].shape[1]
    ldx = changes.get("ldx", c)
    c = changes.get("c", c)
    y = torch.full((t, c), 7, dtype=a["x"].dtype, device="cuda") if y is None else y
    if hidden is None:
        hidden = torch.full((t * k, (h + 7) // 8 * 8), math.nan, dtype=a["x"].dtype, device="cuda")
    if four:
        gp.gemmpipe_expert_step4(code, t, k, e, c, h, four, a["x"], ldx, a["ids"], a["weights"], *a["w1"], *a["w2"],
                                 *a["w3"], hidden, y, y.stride(0))
    else:
        gp.gemmpipe_expert_step(code, t, k, e, c, h, a["x"], ldx, a["ids"], a["weights"], a["w1"], a["w2"], a["w3"],
                                hidden, y, y.stride(0))
    return y


STEPS = [  # t, k, e, c, h
    (1, 1, 1, 8, 8), (1, 8, 64, 256, 128), (1, 2, 8, 520, 72), (1, 1, 1, 1, 1), (1, 4, 1000, 64, 40), (2, 3, 4, 33, 31),
    (4, 2, 8, 1030, 300), (5, 4, 24, 411, 101), (7, 64, 5, 48, 56), (8, 2, 3, 129, 65), (9, 4, 6, 200, 64), (16, 2, 16, 96, 104),
    (31, 1, 2, 72, 33), (33, 2, 2, 64, 130), (40, 1, 1, 40, 24), (64, 8, 64, 128, 96), (64, 2, 3, 70, 70),
    (64, 64, 70, 32, 16), (64, 1, 1024, 16, 8), (3, 2, 5, 7, 2), (1, 8, 8, 64, 640)]


@pytest.mark.parametrize("t, k, e, c, h", STEPS)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("four", [0, 32, 128])
@pytest.mark.parametrize("type_", TYPES)
def test_step_exact(type_, four, gated, t, k, e, c, h):
    args = step_case(type_, t, k, e, c, h, gated, four)
    y = run_step(type_, args, e, h, four)
    status_ok()
    assert torch.equal(y, args["want"])


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("four", [0, 64])
def test_step_without_choices(type_, four):
    args = step_case(type_, 6, 2, 4, 96, 64, True, four)
    args["ids"].fill_(-1)
    y = run_step(type_, args, 4, 64, four)
    assert bool((y == 0).all())
    # Some tokens without any, among others.
    args = step_case(type_, 11, 2, 4, 96, 64, False, four, key=1)
    keep = args["want"].clone()
    args["ids"][3], args["ids"][10] = 4, -2 ** 31
    keep[3] = keep[10] = 0
    y = run_step(type_, args, 4, 64, four)
    status_ok()
    assert torch.equal(y, keep)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("t, four", [(3, 0), (12, 0), (3, 32), (40, 64)])
def test_step_same_expert_twice(type_, t, four):
    args = step_case(type_, t, 5, 3, 104, 48, True, four, dropped=0.0)
    assert any(len(set(r)) < 5 for r in args["ids"].tolist())
    y = run_step(type_, args, 3, 48, four)
    status_ok()
    assert torch.equal(y, args["want"])


@pytest.mark.parametrize("four", [0, 32])
@pytest.mark.parametrize("t", [2, 10])
def test_step_unused_experts_do_not_show(t, four):
    e, c, h = 6, 72, 40
    args = step_case("bf16", t, 2, e, c, h, True, four)
    args["ids"] = torch.where(args["ids"] == 2, 3, args["ids"])
    args["weights"] = torch.where(args["weights"].isnan(), math.nan, 1.0)
    want = run_step("bf16", args, e, h, four)
    for name in ("w1", "w2", "w3"):
        (args[name][1] if four else args[name])[2] = math.nan
    y = run_step("bf16", args, e, h, four)
    status_ok()
    assert torch.equal(y, want) and bool(y.isfinite().all())


@pytest.mark.parametrize("four", [0, 32])
@pytest.mark.parametrize("t", [5, 20])
def test_step_infinite_token_stays_alone(t, four):
    e, c, h = 3, 64, 48
    args = step_case("f16", t, 2, e, c, h, False, four, dropped=0.0)
    args["x"][1, 5] = math.nan
    y = run_step("f16", args, e, h, four)
    status_ok()
    others = [i for i in range(t) if i != 1]
    assert bool(y[1].isnan().all()) and torch.equal(y[others], args["want"][others])


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("t", [1, 5, 19])
@pytest.mark.parametrize("what", ["x", "w1", "w2", "w3", "y", "pitch", "all"])
def test_step_places(type_, t, what):
    # Operands at any place, rows at any pitch; nothing is written outside the rows of Y.
    e, c, h = 4, 136, 88
    args = step_case(type_, t, 2, e, c, h, True)
    changes = {}
    for i, name in enumerate(("x", "w1", "w2", "w3")):
        if what in (name, "all"):
            changes[name] = off_by(args[name], 1 + 2 * i)
    if what in ("pitch", "all"):
        changes["x"] = off_by(pitched(args["x"], 3), 1)
        changes |= {"ldx": c + 3, "c": c}
    pad = 5 if what in ("y", "all") else 0
    room = torch.full((t * (c + pad) + 8,), 7, dtype=args["x"].dtype, device="cuda")
    shift = 3 if what in ("y", "all") else 0
    y = room[shift:shift + t * (c + pad)].view(t, c + pad)
    run_step(type_, args, e, h, 0, y=y, **changes)
    status_ok()
    assert torch.equal(y[:, :c], args["want"])
    assert bool((y[:, c:] == 7).all()) and bool((room[:shift] == 7).all())
    assert bool((room[shift + t * (c + pad):] == 7).all())


def test_step_without_hidden():
    y = torch.full((3, 10), 7, dtype=torch.float16, device="cuda")
    gp.gemmpipe_expert_step(gp.F16, 3, 2, 4, 8, 0, None, 8, None, None, None, None, None, None, y, 10)
    status_ok()
    assert bool((y[:, :8] == 0).all()) and bool((y[:, 8:] == 7).all())


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("t, k, e, c, h, gated", [(1, 4, 8, 512, 200, True), (6, 2, 3, 130, 515, False),
                                                  (37, 4, 6, 256, 128, True)])
def test_step_random(type_, t, k, e, c, h, gated):
    g = generator("random step", type_, t, c)
    code, dtype = TYPES[type_]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w1, w2 = rand(t, c).to(dtype), (rand(e, c, h) * c ** -0.5).to(dtype), (rand(e, h, c) * h ** -0.5).to(dtype)
    w3 = (rand(e, c, h) * c ** -0.5).to(dtype) if gated else None
    ids = torch.stack([torch.randperm(e, generator=g, device="cuda")[:k] for _ in range(t)]).int()
    weights = torch.softmax(rand(t, k), 1)
    y, hidden = torch.empty_like(x), torch.empty(t * k, (h + 7) // 8 * 8, dtype=dtype, device="cuda")
    gp.gemmpipe_expert_step(code, t, k, e, c, h, x, c, ids, weights, w1, w2, w3, hidden, y, c)
    status_ok()
    u, f = torch.finfo(dtype).eps / 2, 2.0 ** -22
    want, bound = torch.zeros(t, c, dtype=torch.float64, device="cuda"), torch.zeros(t, c, dtype=torch.float64, device="cuda")
    for j in range(k):
        for i in range(t):
            n = int(ids[i, j])
            xi, w = x[i].double(), float(weights[i, j])
            a, size = xi @ w1[n].double(), xi.abs() @ w1[n].double().abs()
            # silu has slopes up to 1.1; fp32 exp, sum and quotient add up to 8 steps of 2^-22.
            s = a * torch.sigmoid(a)
            ds = 1.1 * (c / 16 + 80) * f * size + 8 * f * s.abs()
            if gated:
                b, size3 = xi @ w3[n].double(), xi.abs() @ w3[n].double().abs()
                ds = ds * b.abs() + (s.abs() + ds) * (c / 16 + 80) * f * size3
                s = s * b
            # The hidden value is rounded to 16 bits (fp16: absolutely below 2^-14).
            ds = ds + u * s.abs() + (2.0 ** -25 if dtype == torch.float16 else 0)
            m = w2[n].double()
            want[i] += w * (s @ m)
            bound[i] += w * (ds @ m.abs() + (k * h / 16 + 80) * f * (s.abs() @ m.abs()))
    bound = bound + u * want.abs()
    assert bool(((y.double() - want).abs() <= bound * (1 + 1e-2)).all())


def test_step_repeats_bit_for_bit():
    g = generator("repeat")
    for t, e, c, h in ((1, 16, 1024, 256), (48, 8, 256, 192)):
        x, w1, w2, w3 = (torch.randn(*s, generator=g, device="cuda").half() for s in
                         ((t, c), (e, c, h), (e, h, c), (e, c, h)))
        ids = torch.randint(0, e, (t, 4), generator=g, device="cuda").int()
        args = {"x": x * 0.05, "ids": ids, "weights": torch.rand(t, 4, generator=g, device="cuda"), "w1": w1 * 0.1,
                "w2": w2 * 0.1, "w3": w3 * 0.1}
        first = run_step("f16", args, e, h, 0)
        for _ in range(20):
            assert torch.equal(run_step("f16", args, e, h, 0), first)
        assert bool(first.isfinite().all())


# -------------------------------------------------- streams, graphs, the run


@pytest.mark.parametrize("four", [0, 64])
def test_two_streams_at_once(four):
    cases = [step_case("bf16", t, 4, 8, 264, 136, True, four, key=t) for t in (1, 24)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        ys = []
        for args, s in zip(cases, streams):
            with torch.cuda.stream(s):
                ys.append(run_step("bf16", args, 8, 136, four))
        torch.cuda.synchronize()
        for y, args in zip(ys, cases):
            assert torch.equal(y, args["want"])


@pytest.mark.parametrize("four", [0, 32])
def test_captured_and_replayed(four):
    # New inputs between replays, among them other experts; rows4 in the same graph.
    e, c, h = 8, 200, 96
    cases = [step_case("f16", 3, 2, e, c, h, True, four, key=i) for i in range(4)]
    held = {n: (tuple(None if p is None else p.clone() for p in v) if isinstance(v, tuple) else v.clone())
            for n, v in cases[0].items()}
    x4, q4, s4, want4 = rows4_case("f16", 3, c, 50, 32)
    y, y4 = torch.empty(3, c, dtype=torch.float16, device="cuda"), torch.empty(3, 50, dtype=torch.float16, device="cuda")
    hidden = torch.empty(6, 96, dtype=torch.float16, device="cuda")

    def both():
        run_step("f16", held, e, h, four, y=y, hidden=hidden)
        gp.gemm_rows4(gp.F16, 3, 50, c, 32, x4, c, q4, s4, y4, 50)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for case in cases[1:] + cases[:1]:
        for n, v in case.items():
            for to, fr in zip(held[n], v) if isinstance(v, tuple) else [(held[n], v)]:
                to.copy_(fr)
        y.fill_(7), y4.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, case["want"]) and torch.equal(y4, want4)
    status_ok()


def test_launches_are_counted_and_timed():
    args = step_case("bf16", 2, 2, 4, 64, 64, True)
    x, q, s, _ = rows4_case("bf16", 1, 64, 64, 32)
    y = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    n = gp.gemmpipe_launch_count()
    gp.gemmpipe_timing_enable(True)
    try:
        gp.gemmpipe_timing_read()
        run_step("bf16", args, 4, 64, 0)
        gp.gemm_rows4(gp.BF16, 1, 64, 64, 32, x, 64, q, s, y, 64)
        ms, count, _, _ = gp.gemmpipe_timing_read()
    finally:
        gp.gemmpipe_timing_enable(False)
    assert gp.gemmpipe_launch_count() == n + 3 and count >= 2 and ms > 0
