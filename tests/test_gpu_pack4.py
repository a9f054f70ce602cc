"""Weights into 4 bits and back, against the formula, and the few-token
operators for PyTorch as they are used together."""
from __future__ import annotations

import math

import pytest
import torch

from software_pipelined_loop_gb300 import few_tokens as few
from software_pipelined_loop_gb300 import gemmpipe as gp
from software_pipelined_loop_gb300.expert_layer import expert_layer

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
ROW_OF_NIBBLE = [0, 2, 4, 6, 1, 3, 5, 7]


def formula(w, group):
    """(q, scales, values) of experts x K x N in 64 bits: scales rounded to the type."""
    e, k, n = w.shape
    pad = torch.nn.functional.pad(w.double(), (0, 0, 0, -k % group)).view(e, -1, group, n)
    finite = pad.isfinite().all(2, keepdim=True)
    # (the quotient of two 16-bit values and 7: rounding to fp32 in between changes nothing)
    scale = (pad.abs().amax(2, keepdim=True) / 7).to(w.dtype).double()
    steps = torch.where(finite & (scale > 0), pad / scale, 0.0).round().clamp(-8, 7)
    scale = torch.where(finite, scale, math.nan)
    q = (steps + 8).long().view(e, -1, n)[:, :k]
    return q, scale[:, :, 0].to(w.dtype), (steps * scale).view(e, -1, n)[:, :k]


def unpacked_words(words, k, n):
    q = torch.stack([(words >> (4 * ROW_OF_NIBBLE.index(r))) & 15 for r in range(8)], 2)
    return q.flatten(1, 2)


def special(w):
    w.view(-1)[::37] = 0
    if w.shape[1] > 40 and w.shape[2] > 9:
        w[0, :32, 0] = 0                       # a group of zeros (for groups of 32)
        w[0, 5, 1], w[-1, 40, 2] = math.inf, math.nan
        w[0, :, 3] = torch.finfo(w.dtype).max
        w[0, :, 4] = torch.finfo(w.dtype).tiny / 4
        w[0, 1::2, 5] = -w[0, 1::2, 5].abs() * 2
        w[0, :, 6] = w[0, 0, 6]                # one magnitude
        w[0, ::2, 6] *= -1
        w[0, :, 7] = torch.arange(w.shape[1], device="cuda").remainder(29).sub(14).to(w.dtype) / 2  # scale 1: ties
    return w


SHAPES = [(1, 128, 64), (1, 1, 1), (2, 33, 5), (3, 130, 67), (1, 4096, 12), (2, 64, 1001), (24, 41, 10), (1, 7, 4000),
          (5, 257, 129), (1, 1000, 256)]


@pytest.mark.parametrize("e, k, n", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_pack_and_unpack(dtype, group, e, k, n, shift):
    g = torch.Generator(device="cuda").manual_seed(k * n)
    room = torch.empty(e * k * n + shift, dtype=dtype, device="cuda")
    w = room[shift:].view(e, k, n)
    w.copy_(special(torch.randn(e, k, n, generator=g, device="cuda").to(dtype)))
    n4, code = (n + 3) // 4 * 4, {torch.float16: gp.F16, torch.bfloat16: gp.BF16}[dtype]
    q = torch.full((e, -(-k // 8), n4), -1, dtype=torch.int32, device="cuda")
    s = torch.full((e, -(-k // group), n4), 7, dtype=dtype, device="cuda")
    gp.gemmpipe_pack4(code, e, k, n, group, w, q, s)
    back = torch.full((e * k * n + shift + 1,), 7, dtype=dtype, device="cuda")
    gp.gemmpipe_unpack4(code, e, k, n, group, q, s, back[shift:])
    assert gp.gemmpipe_get_device_status() == gp.OK
    want_q, want_s, want = formula(w, group)
    got_q = unpacked_words(q, k, n)
    assert torch.equal(got_q[:, :k, :n], want_q)
    assert bool((got_q[:, k:] == 8).all()) and bool((got_q[:, :, n:] == 8).all()) and bool((s[:, :, n:] == 0).all())
    assert torch.equal(s[:, :, :n].nan_to_num(nan=-1.0), want_s.nan_to_num(nan=-1.0))
    got = back[shift:-1].view(e, k, n)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0), want.to(dtype).nan_to_num(nan=0.0))
    assert bool((back[:shift] == 7).all()) and float(back[-1]) == 7


# ------------------------------------------------------------ used together


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("t", [1, 12, 64])
def test_packed_layer_is_the_layer_of_the_unpacked_values(dtype, gated, t):
    """pack4, then a step in 4 bits, one in 16 bits on the unpacked values, and expert_layer on them."""
    e, k, c, h = 6, 2, 192, 160
    g = torch.Generator(device="cuda").manual_seed(t)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, weights = rand(t, c).to(dtype), torch.softmax(rand(t, k), 1)
    ids = rand(t, e).topk(k, 1).indices.int()
    packed = [few.pack4((rand(e, *s) * s[0] ** -0.5).to(dtype), 64) for s in ((c, h), (h, c), (c, h))[:3 if gated else 2]]
    plain = [few.unpack4(m) for m in packed]
    with torch.no_grad():
        four, sixteen = few.expert_step(x, ids, weights, *packed), few.expert_step(x, ids, weights, *plain)
        layer = None if gated else expert_layer(x, ids, weights, *plain)
    u = torch.finfo(dtype).eps / 2

    def exact(mats):
        y = torch.zeros(t, c, dtype=torch.float64, device="cuda")
        for j in range(k):
            rows = [m[ids[:, j].long()].double() for m in mats]
            a = torch.einsum("tc,tch->th", x.double(), rows[0])
            a = a * torch.sigmoid(a)
            if gated:
                a = a * torch.einsum("tc,tch->th", x.double(), rows[2])
            y += weights[:, j, None].double() * torch.einsum("th,thc->tc", a, rows[1])
        return y

    want16 = exact(plain)
    values = [(few.unpack4(m._replace(scales=torch.ones_like(m.scales))).double() *
               m.scales.double().repeat_interleave(m.group, 1)[:, :m.inner, :m.outer]) for m in packed]
    want4 = exact(values)
    # In the 2-norm: roundings to 16 bits are independent; hidden rows and Y once each (expert_layer: the product,
    # its silu, each expert's row and the sum), each at most u of its value and sqrt(3) less in the mean square.
    for got, want, roundings in ((four, want4, 2), (sixteen, want16, 2), (layer, want16, 4)):
        if got is not None:
            assert float((got.double() - want).norm() / want.norm()) <= roundings * u
    assert gp.gemmpipe_get_device_status() == gp.OK


@pytest.mark.parametrize("dtype", TYPES)
def test_rows4_and_the_unpacked_product(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(300, 90, generator=g, device="cuda") * 300 ** -0.5).to(dtype)
    x = torch.randn(64, 300, generator=g, device="cuda").to(dtype)
    m = few.pack4(w, 32)
    y = few.rows4(x, m)
    values = few.unpack4(m)
    many = torch.empty(64, 90, dtype=dtype, device="cuda")
    offsets = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    gp.gemm_grouped({torch.float16: 0, torch.bfloat16: 1}[dtype], 64, 90, 300, 1, x, 300, offsets, values, many, 90)
    u = torch.finfo(dtype).eps / 2
    # Each side rounds its result once, and one side its weights: in the 2-norm at most 3 u.
    assert float((y.double() - many.double()).norm() / many.double().norm()) <= 3 * u
    # One expert's matrix out of several, and strided rows.
    ms = few.pack4(torch.stack([w, w * 2]), 32)
    wide = torch.full((64, 307), math.nan, dtype=dtype, device="cuda")
    wide[:, 4:304] = x
    assert torch.equal(few.rows4(wide[:, 4:304], ms.expert(1)), few.rows4(x, ms.expert(0)) * 2)
    assert torch.equal(few.rows4(x[::3], m), y[::3].contiguous())
    assert torch.equal(few.rows4(x.t().contiguous().t(), m), y)
    assert few.rows4(x[:0], m).shape == (0, 90)


def test_strided_arguments_of_the_step():
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    e, c, h = 4, 64, 40
    x, w1, w2 = rand(6, c).bfloat16(), (rand(e, c, h) * 0.1).bfloat16(), (rand(e, h, c) * 0.1).bfloat16()
    ids, weights = torch.randint(0, e, (6, 2), generator=g, device="cuda").int(), rand(6, 2)
    want = few.expert_step(x, ids, weights, w1, w2)
    turn = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)  # noqa: E731
    got = few.expert_step(turn(x), turn(ids), turn(weights), turn(w1), turn(w2))
    assert torch.equal(got, want)
    assert torch.equal(few.expert_step(x[2:3].expand(6, c), ids, weights, w1, w2)[2], want[2])
    leaf = w1.clone().requires_grad_()
    with torch.no_grad():
        assert torch.equal(few.expert_step(x, ids, weights, leaf, w2), want)


def test_memory_of_another_stream():
    """Tensors made on another stream, used after its event, as torch asks for."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, w = torch.ones(2, 64, device="cuda").half(), torch.ones(64, 32, device="cuda").half()
        m = few.pack4(w, 32)
    torch.cuda.current_stream().wait_stream(s)
    assert bool((few.rows4(x, m) == (64 * 7 * torch.tensor(1 / 7).half().double()).half()).all())
