"""The expert-layer operators on the GPU against plain formulas in 64 bits.

Tolerances.  A result of the products is an fp32 sum of exact 16-bit products
rounded once to 16 bits.  With u half a unit in the last place of the type
(2^-11 fp16, 2^-8 bf16, relative; 2^-25 absolute for fp16's finest step), and
the tensor core adding 16 products to the fp32 sum at a time with at most one
unit lost per addition (2^-22 of the largest partial sum, itself at most the
sum of magnitudes):
    |error| <= u |exact| + 2^-25 + (depth / 16 + 16) 2^-22 sum |a| |b|.
The rows' operators have no tensor core: u |exact| + 2^-25 and, for a sum of n
terms in fp32, n 2^-23 sum |terms|.
"""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

pytestmark = pytest.mark.gpu

TYPES = {"f16": (gp.F16, torch.float16, 2.0 ** -11), "bf16": (gp.BF16, torch.bfloat16, 2.0 ** -8)}
NAN = float("nan")


@pytest.fixture(autouse=True)
def _device_status():
    yield
    assert gp.gemmpipe_get_device_status() == gp.OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, ty=torch.float16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(ty)


def pitched(x, ld, offset=0):
    """A copy of x with rows `ld` elements apart, starting `offset` elements into its storage; NaN around it."""
    buf = torch.full((x.shape[0] * ld + offset + 64,), NAN, dtype=x.dtype, device=x.device)
    view = buf[offset:offset + x.shape[0] * ld].view(x.shape[0], ld)[:, :x.shape[1]]
    view.copy_(x)
    return view


def offsets_of(counts, head=0):
    o = [head]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check_close(got, exact, bound, what=""):
    err = (got.double() - exact).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float(err[bad].max()):.3g} at {bad.nonzero()[0].tolist()}"


def product_bound(u, depth, exact, magnitude):
    return u * exact.abs() + 2.0 ** -25 + (depth / 16 + 16) * 2.0 ** -22 * magnitude


# Rows per expert.  The mean decides the tile (32, 64, 128 or 256 rows): each
# list stays on one side, with experts of no row, one row and more than a tile.
COUNTS = {
    "one_row": [0, 0, 1, 0],
    "few": [0, 1, 7, 33, 0, 16, 2, 1],
    "mean_32": [64, 0, 65, 1, 31, 3],
    "mean_96": [0, 200, 96, 129, 1, 50],
    "large": [700, 0, 256, 257, 1, 511],
    "one_expert": [777],
}
# (inner, outer): whole tiles, below one tile, odd, just past a tile.
SIZES = [(64, 128), (8, 8), (200, 136), (129, 257), (1000, 300), (333, 65), (1, 1), (512, 640)]


def setup(counts, K, N, ty, seed, head=0, unused=0):
    g = gen(seed)
    off = offsets_of(counts, head)
    R = int(off[-1]) + unused
    X = randn(g, R, K, ty=ty)
    dY = randn(g, R, N, ty=ty, scale=0.25)
    W = randn(g, len(counts), K, N, ty=ty, scale=K ** -0.5)
    for t in (X, dY):
        t[:head] = NAN
        t[R - unused:] = NAN
    return off, R, X, dY, W


def rows_reference(off, A, B):
    """(exact, magnitude) of A[r] @ B[e] for each expert's rows."""
    o = off.tolist()
    y = torch.zeros(A.shape[0], B.shape[2], dtype=torch.float64, device="cuda")
    m = torch.zeros_like(y)
    for e in range(len(o) - 1):
        a, b = A[o[e]:o[e + 1]].double(), B[e].double()
        y[o[e]:o[e + 1]] = a @ b
        m[o[e]:o[e + 1]] = a.abs() @ b.abs()
    return y, m


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("counts", COUNTS)
def test_products_of_rows(counts, size, ty):
    code, dtype, u = TYPES[ty]
    K, N = size
    c = COUNTS[counts]
    off, R, X, dY, W = setup(c, K, N, dtype, seed=7, unused=5)
    Y = torch.full((R, N), 3.0, dtype=dtype, device="cuda")
    gp.gemm_grouped(code, R, N, K, len(c), X, K, off, W, Y, N)
    exact, mag = rows_reference(off, X, W)
    check_close(Y, exact, product_bound(u, K, exact, mag), "forward")
    dX = torch.full((R, K), 3.0, dtype=dtype, device="cuda")
    gp.gemm_grouped_dx(code, R, N, K, len(c), dY, N, off, W, dX, K)
    exact, mag = rows_reference(off, dY, W.transpose(1, 2))
    check_close(dX, exact, product_bound(u, N, exact, mag), "gradient to the rows")


def weights_reference(off, X, dY):
    o = off.tolist()
    E = len(o) - 1
    w = torch.zeros(E, X.shape[1], dY.shape[1], dtype=torch.float64, device="cuda")
    m = torch.zeros_like(w)
    for e in range(E):
        a, b = X[o[e]:o[e + 1]].double(), dY[o[e]:o[e + 1]].double()
        w[e] = a.t() @ b
        m[e] = a.t().abs() @ b.abs()
    return w, m


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("counts", COUNTS)
def test_gradient_to_weights(counts, size, ty):
    code, dtype, u = TYPES[ty]
    K, N = size
    c = COUNTS[counts]
    # Rows before the first and after the last expert are NaN: read into no sum.
    off, R, X, dY, W = setup(c, K, N, dtype, seed=11, head=3, unused=70)
    dW = torch.full((len(c), K, N), 3.0, dtype=dtype, device="cuda")
    gp.gemm_grouped_dw(code, R, N, K, len(c), X, K, dY, N, off, dW)
    exact, mag = weights_reference(off, X, dY)
    check_close(dW, exact, product_bound(u, max(c), exact, mag), "gradient to the weights")


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("size", [(64, 128), (300, 257), (1, 8), (512, 640)], ids=str)
@pytest.mark.parametrize("counts", [[5000], [1025, 0, 7, 3333, 1024, 1], [40] * 300 + [2500, 0, 1500]], ids=len)
def test_gradient_to_weights_in_parts(counts, size, ty):
    # Matrices of few tiles and experts of many rows: their sums are split (300 experts: too many to sort).
    code, dtype, u = TYPES[ty]
    K, N = size
    off, R, X, dY, W = setup(counts, K, N, dtype, seed=17, head=1, unused=33)
    dW = torch.full((len(counts), K, N), 3.0, dtype=dtype, device="cuda")
    gp.gemm_grouped_dw(code, R, N, K, len(counts), X, K, dY, N, off, dW)
    exact, mag = weights_reference(off, X, dY)
    check_close(dW, exact, product_bound(u, max(counts), exact, mag))
    again = torch.empty_like(dW)
    gp.gemm_grouped_dw(code, R, N, K, len(counts), X, K, dY, N, off, again)
    assert torch.equal(dW, again)


@pytest.mark.parametrize("size", [(64, 128), (200, 136), (129, 257)], ids=str)
def test_rows_of_other_experts_are_not_mixed(size):
    # Every other expert's rows are infinite or NaN: the rest stay finite and right.
    K, N = size
    c = [17, 40, 5, 90, 64, 3]
    off, R, X, dY, W = setup(c, K, N, torch.float16, seed=3)
    o = off.tolist()
    for e in (1, 3, 5):
        X[o[e]:o[e + 1]] = float("inf") if e == 1 else NAN
        dY[o[e]:o[e + 1]] = NAN
    Y = torch.empty(R, N, dtype=torch.float16, device="cuda")
    gp.gemm_grouped(gp.F16, R, N, K, len(c), X, K, off, W, Y, N)
    dW = torch.empty(len(c), K, N, dtype=torch.float16, device="cuda")
    gp.gemm_grouped_dw(gp.F16, R, N, K, len(c), X, K, dY, N, off, dW)
    exact, mag = rows_reference(off, X, W)
    exact_w, mag_w = weights_reference(off, X, dY)
    for e in (0, 2, 4):
        s = slice(o[e], o[e + 1])
        check_close(Y[s], exact[s], product_bound(2.0 ** -11, K, exact[s], mag[s]))
        check_close(dW[e], exact_w[e], product_bound(2.0 ** -11, c[e], exact_w[e], mag_w[e]))
    assert bool(torch.isnan(dW[3]).all())


@pytest.mark.parametrize("mean", [4, 40, 400])
def test_pitches_and_alignments(mean):
    K, N, E = 136, 72, 3
    off, R, X, dY, W = setup([mean, 2 * mean, 0], K, N, torch.float16, seed=5)
    exact, mag = rows_reference(off, X, W)
    exact_w, mag_w = weights_reference(off, X, dY)
    for ld, shift in ((K + 8, 8), (K + 3, 0), (K, 1), (K + 1, 3)):
        Xp = pitched(X, ld, shift)
        dYp = pitched(dY, N + ld - K, shift)
        Y = pitched(torch.zeros(R, N, dtype=torch.float16, device="cuda"), N + ld - K, shift)
        keep = Y._base.clone()
        gp.gemm_grouped(gp.F16, R, N, K, E, Xp, ld, off, W, Y, N + ld - K)
        check_close(Y, exact, product_bound(2.0 ** -11, K, exact, mag), f"pitch {ld} + {shift}")
        Y.zero_()
        assert torch.equal(torch.isnan(Y._base), torch.isnan(keep))  # nothing written between the rows
        dW = torch.empty(E, K, N, dtype=torch.float16, device="cuda")
        gp.gemm_grouped_dw(gp.F16, R, N, K, E, Xp, ld, dYp, N + ld - K, off, dW)
        check_close(dW, exact_w, product_bound(2.0 ** -11, 2 * mean, exact_w, mag_w))
    Wp = torch.empty(W.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(W)
    Wp.copy_(W)
    Y = torch.empty(R, N, dtype=torch.float16, device="cuda")
    gp.gemm_grouped(gp.F16, R, N, K, E, X, K, off, Wp, Y, N)
    check_close(Y, exact, product_bound(2.0 ** -11, K, exact, mag))


@pytest.mark.parametrize("N", [64, 65])  # 65: only the weights of experts with rows are copied
def test_bounds_out_of_order_are_clamped(N):
    K, R = 64, 50
    g = gen(1)
    X, W, dY = randn(g, R, K), randn(g, 4, K, N, scale=0.1), randn(g, R, N)
    wild = torch.tensor([-7, 30, 10, 60, 2 ** 30], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 30, 30, 50, 50], dtype=torch.int32, device="cuda")
    out = [torch.empty(R, N, dtype=torch.float16, device="cuda") for _ in range(2)]
    grad = [torch.empty(4, K, N, dtype=torch.float16, device="cuda") for _ in range(2)]
    for off, y, w in zip((wild, tame), out, grad):
        gp.gemm_grouped(gp.F16, R, N, K, 4, X, K, off, W, y, N)
        gp.gemm_grouped_dw(gp.F16, R, N, K, 4, X, K, dY, N, off, w)
    assert torch.equal(out[0], out[1]) and torch.equal(grad[0], grad[1])


def test_many_experts_and_long_sums():
    # 1024 experts with a row or none each; then one sum of 20000 products.
    g = gen(2)
    counts = (torch.rand(1024, generator=g, device="cuda") < 0.4).int().tolist()
    off, R, X, dY, W = setup(counts, 72, 64, torch.bfloat16, seed=9)
    Y = torch.empty(R, 64, dtype=torch.bfloat16, device="cuda")
    gp.gemm_grouped(gp.BF16, R, 64, 72, 1024, X, 72, off, W, Y, 64)
    exact, mag = rows_reference(off, X, W)
    check_close(Y, exact, product_bound(2.0 ** -8, 72, exact, mag))
    off, R, X, dY, W = setup([0, 20000, 9], 64, 128, torch.bfloat16, seed=10)
    dW = torch.empty(3, 64, 128, dtype=torch.bfloat16, device="cuda")
    gp.gemm_grouped_dw(gp.BF16, R, 128, 64, 3, X, 64, dY, 128, off, dW)
    exact, mag = weights_reference(off, X, dY)
    check_close(dW, exact, product_bound(2.0 ** -8, 20000, exact, mag))


def test_row_offsets_past_32_bits():
    # Rows whose elements lie beyond 2^31 elements of the buffers.
    K, ld, R = 64, 1 << 20, 2600
    buf = torch.zeros(R * ld, dtype=torch.float16, device="cuda")
    X = buf.view(R, ld)[:, :K]
    out = torch.zeros(R * ld, dtype=torch.float16, device="cuda").view(R, ld)[:, :K]
    g = gen(4)
    X.copy_(randn(g, R, K))
    W = randn(g, 1, K, K, scale=0.1)
    off = offsets_of([R])
    gp.gemm_grouped(gp.F16, R, K, K, 1, X, ld, off, W, out, ld)
    exact, mag = rows_reference(off, X.contiguous(), W)
    check_close(out, exact, product_bound(2.0 ** -11, K, exact, mag))


def test_empty_products():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y = torch.full((4, 8), 1.0, dtype=torch.float16, device="cuda")
    gp.gemm_grouped(gp.F16, 4, 8, 0, 2, None, 0, off, None, Y, 8)  # nothing to sum
    assert int(Y.count_nonzero()) == 0
    dW = torch.full((2, 8, 8), 1.0, dtype=torch.float16, device="cuda")
    gp.gemm_grouped_dw(gp.F16, 0, 8, 8, 2, None, 8, None, 8, off, dW)  # no rows
    assert int(dW.count_nonzero()) == 0
    n = gp.gemmpipe_launch_count()
    gp.gemm_grouped(gp.F16, 0, 8, 8, 2, None, 8, None, None, None, 8)
    gp.gemm_grouped_dx(gp.F16, 4, 8, 0, 2, None, 8, None, None, None, 0)
    gp.gemmpipe_dispatch(gp.F16, 0, 2, 8, None, 8, None, None, None, 8)
    assert gp.gemmpipe_launch_count() == n


# ------------------------------------------------------------------ routing


def route(ids, E, top_k):
    T = ids.numel() // top_k
    new = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")  # noqa: E731
    off, slots, rows = new(E + 1), new(T * top_k), new(T * top_k)
    gp.gemmpipe_route(T, top_k, E, ids, off, slots, rows)
    return off, slots, rows


def route_reference(ids, E):
    lists = [[] for _ in range(E + 1)]
    for s, e in enumerate(ids.tolist()):
        lists[e if 0 <= e < E else E].append(s)
    slots = [s if e < E else ~s for e in range(E + 1) for s in lists[e]]
    rows = [0] * len(slots)
    for r, s in enumerate(slots):
        rows[s if s >= 0 else ~s] = r if s >= 0 else ~r
    off = [0]
    for e in range(E):
        off.append(off[-1] + len(lists[e]))
    return off, slots, rows


@pytest.mark.parametrize("E", [1, 3, 64, 257, 1024])
@pytest.mark.parametrize("R", [1, 31, 512, 2048, 2049, 40001])
def test_route(R, E):
    g = gen(R + E)
    ids = torch.randint(-1, E + 1, (R,), generator=g, device="cuda").int()
    ids[torch.rand(R, generator=g, device="cuda") < 0.02] = -2 ** 31
    off, slots, rows = route(ids, E, 1)
    want = route_reference(ids, E)
    assert (off.tolist(), slots.tolist(), rows.tolist()) == want


def test_route_skewed_and_large():
    E, R = 16, 700_000
    g = gen(0)
    ids = torch.where(torch.rand(R, generator=g, device="cuda") < 0.9, 5,
                      torch.randint(0, E, (R,), generator=g, device="cuda")).int()
    off, slots, rows = route(ids, E, 1)
    order = torch.sort(ids, stable=True).indices.int()
    assert torch.equal(slots, order)
    assert torch.equal(rows[order.long()], torch.arange(R, dtype=torch.int32, device="cuda"))
    assert torch.equal(off[1:].long(), torch.cumsum(torch.bincount(ids, minlength=E), 0))


def test_route_none():
    off = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    gp.gemmpipe_route(0, 2, 8, None, off, None, None)
    assert off.tolist() == [0] * 9
    ids = torch.full((6,), -1, dtype=torch.int32, device="cuda")  # every choice dropped
    off, slots, rows = route(ids, 4, 2)
    assert off.tolist() == [0] * 5 and slots.tolist() == rows.tolist() == [~i for i in range(6)]


# ------------------------------------------------- rows out, back, gradient

SHAPES = [(1, 8, 2048), (1, 1, 1), (5, 3, 7), (33, 8, 264), (130, 2, 3001), (64, 13, 130), (257, 4, 1000), (9, 64, 36)]


def routing(T, k, E, seed, drop=0.1):
    g = gen(seed)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    ids[torch.rand(T, k, generator=g, device="cuda") < drop] = -1
    if T > 2:
        ids[1] = -1  # a token whose choices are all dropped
    off, slots, rows = route(ids.view(-1), E, k)
    return g, rows.view(T, k), int(off[-1])


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_out_and_back(shape, weighted, ty):
    code, dtype, u = TYPES[ty]
    T, k, C = shape
    R = T * k
    g, rows, kept = routing(T, k, 7, seed=T + C)
    w = torch.rand(T, k, generator=g, device="cuda") if weighted else None
    if weighted:
        w[rows < 0] = NAN  # a dropped choice's weight is not used
    wd = torch.where(rows >= 0, w.double() if weighted else torch.ones(T, k, dtype=torch.float64, device="cuda"), 0.0)
    place = torch.where(rows >= 0, rows, ~rows).long()

    X = randn(g, T, C, ty=dtype)
    Xs = torch.full((R, C), 9.0, dtype=dtype, device="cuda")
    gp.gemmpipe_dispatch(code, T, k, C, X, C, rows, w, Xs, C)
    exact = torch.zeros(R, C, dtype=torch.float64, device="cuda")
    exact[place.view(-1)] = (wd[:, :, None] * X.double()[:, None, :]).view(R, C)
    if weighted:
        # One rounding of the fp32 product of an fp32 weight and a 16-bit value.
        check_close(Xs, exact, u * exact.abs() + 2.0 ** -23 * exact.abs() + 2.0 ** -25, "dispatch")
    else:
        assert torch.equal(Xs.double(), exact)

    Ys = randn(g, R, C, ty=dtype)
    Ys[kept:] = NAN
    Y = torch.full((T, C), 9.0, dtype=dtype, device="cuda")
    gp.gemmpipe_combine(code, T, k, C, Ys, C, rows, w, Y, C)
    terms = wd[:, :, None] * torch.where((rows >= 0)[:, :, None], Ys[place].double(), 0.0)
    exact = terms.sum(1)
    check_close(Y, exact, u * exact.abs() + 2.0 ** -25 + k * 2.0 ** -23 * terms.abs().sum(1), "combine")

    dY = randn(g, T, C, ty=dtype)
    dYs = torch.full((R, C), 9.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), 9.0, device="cuda")
    gp.gemmpipe_combine_grad(code, T, k, C, dY, C, Ys, C, rows, w, dYs, C, dw)
    exact = torch.zeros(R, C, dtype=torch.float64, device="cuda")
    exact[place.view(-1)] = (wd[:, :, None] * dY.double()[:, None, :]).view(R, C)
    check_close(dYs, exact, u * exact.abs() + 2.0 ** -23 * exact.abs() + 2.0 ** -25, "gradient to the rows")
    terms = torch.where((rows >= 0)[:, :, None], Ys[place].double(), 0.0) * dY.double()[:, None, :]
    check_close(dw, terms.sum(2), (C + 2) * 2.0 ** -23 * terms.abs().sum(2), "gradient to the weights")


def test_rows_with_pitches():
    T, k, C = 40, 3, 72
    g, rows, kept = routing(T, k, 5, seed=1)
    X = randn(g, T, C)
    plain = torch.empty(T * k, C, dtype=torch.float16, device="cuda")
    gp.gemmpipe_dispatch(gp.F16, T, k, C, X, C, rows, None, plain, C)
    w = torch.rand(T, k, generator=g, device="cuda")
    Y = torch.empty(T, C, dtype=torch.float16, device="cuda")
    gp.gemmpipe_combine(gp.F16, T, k, C, plain, C, rows, w, Y, C)
    dY = randn(g, T, C)
    grads = [torch.empty(T * k, C, dtype=torch.float16, device="cuda"), torch.empty(T, k, device="cuda")]
    gp.gemmpipe_combine_grad(gp.F16, T, k, C, dY, C, plain, C, rows, w, grads[0], C, grads[1])
    for ld, shift in ((C + 8, 8), (C + 4, 4), (C + 2, 2), (C + 1, 0), (C, 3)):
        Xs = pitched(torch.zeros_like(plain), ld, shift)
        gp.gemmpipe_dispatch(gp.F16, T, k, C, pitched(X, ld, shift), ld, rows, None, Xs, ld)
        assert torch.equal(Xs, plain)
        Z = pitched(torch.zeros_like(Y), ld, shift)
        gp.gemmpipe_combine(gp.F16, T, k, C, Xs, ld, rows, w, Z, ld)
        assert torch.equal(Z, Y)
        dYs, dw = pitched(torch.zeros_like(plain), ld, shift), torch.empty(T, k, device="cuda")
        gp.gemmpipe_combine_grad(gp.F16, T, k, C, pitched(dY, ld, shift), ld, Xs, ld, rows, w, dYs, ld, dw)
        assert torch.equal(dYs, grads[0])
        # The sum over c is split by the access width: same terms, another order.
        terms = Xs[torch.where(rows >= 0, rows, ~rows).long()].double() * dY.double()[:, None, :]
        check_close(dw, grads[1].double(), 2 * (C + 2) * 2.0 ** -23 * terms.abs().sum(2) + 1e-30)


@pytest.mark.parametrize("T", [3, 1025])  # few and many tokens
@pytest.mark.parametrize("C", [1, 7, 8, 9, 247, 248, 249, 255, 743, 744, 745, 1489])
def test_rows_at_every_alignment(C, T):
    # Whole numbers: every product and sum is exact.  What lies between the
    # rows is NaN before and after.
    k = 2
    g, rows, _ = routing(T, k, 5, seed=C)
    place = torch.where(rows >= 0, rows, ~rows).long()
    X = torch.randint(-8, 9, (T, C), generator=g, device="cuda").half()
    w = torch.randint(1, 4, (T, k), generator=g, device="cuda").float()
    kept = (rows >= 0)[:, :, None]
    out = torch.zeros(T * k, C, device="cuda")
    out[place.view(-1)] = torch.where(kept, X.float()[:, None, :], 0.0).expand(T, k, C).reshape(-1, C)
    weighted = torch.zeros_like(out)
    weighted[place.view(-1)] = (w[:, :, None] * torch.where(kept, X.float()[:, None, :], 0.0)).reshape(-1, C)
    back = (w[:, :, None] * torch.where(kept, out[place], 0.0)).sum(1)
    dot = (out[place] * X.float()[:, None, :]).sum(2)

    def buffer(n, ld, shift):
        buf = torch.full((n * ld + shift + 64,), NAN, dtype=torch.float16, device="cuda")
        return buf, buf[shift:shift + n * ld].view(n, ld)[:, :C]

    def check(buf, view, want):
        assert torch.equal(view.float(), want)
        view.fill_(NAN)
        assert bool(torch.isnan(buf).all())

    for shift in range(8):
        ld = C + (shift + 1) % 3
        x = pitched(X, ld, shift)
        buf, Xs = buffer(T * k, ld, 7 - shift)
        gp.gemmpipe_dispatch(gp.F16, T, k, C, x, ld, rows, None, Xs, ld)
        check(buf, Xs, out)
        gp.gemmpipe_dispatch(gp.F16, T, k, C, x, ld, rows, w, Xs, ld)
        check(buf, Xs, weighted)
        Ys = pitched(out.half(), ld, (3 * shift) % 8)
        buf, Y = buffer(T, ld, (5 * shift + 1) % 8)
        gp.gemmpipe_combine(gp.F16, T, k, C, Ys, ld, rows, w, Y, ld)
        check(buf, Y, back)
        buf, dYs = buffer(T * k, ld, 7 - shift)
        dw = torch.empty(T, k, device="cuda")
        gp.gemmpipe_combine_grad(gp.F16, T, k, C, x, ld, Ys, ld, rows, w, dYs, ld, dw)
        check(buf, dYs, weighted)
        assert torch.equal(dw, dot)


def test_entries_outside_the_rows_are_passed_over():
    T, k, C = 4, 2, 32
    rows = torch.arange(8, dtype=torch.int32, device="cuda").view(T, k)
    wild = rows.clone()
    wild[1, 0], wild[2, 1] = 1000, ~1000
    X = randn(gen(0), T, C)
    out = torch.full((8, C), 5.0, dtype=torch.float16, device="cuda")
    gp.gemmpipe_dispatch(gp.F16, T, k, C, X, C, wild, None, out, C)
    want = X.repeat_interleave(2, 0)
    want[2] = want[5] = 5.0
    assert torch.equal(out, want)
    Y = torch.empty(T, C, dtype=torch.float16, device="cuda")
    gp.gemmpipe_combine(gp.F16, T, k, C, want, C, wild, None, Y, C)
    assert torch.equal(Y[1], X[1]) and torch.equal(Y[2], X[2])
    dYs, dw = torch.full_like(out, 5.0), torch.empty(T, k, device="cuda")
    gp.gemmpipe_combine_grad(gp.F16, T, k, C, X, C, want, C, wild, None, dYs, C, dw)
    assert torch.equal(dYs, want) and float(dw[1, 0]) == float(dw[2, 1]) == 0.0


# ------------------------------------------------------------- 8-bit copies


def keep8_reference(x, least):
    """(q, step byte, value) in 64 bits, element by element of the definition."""
    R, C = x.shape
    G = -(-C // 32)
    xd = torch.zeros(R, G * 32, dtype=torch.float64, device="cuda")
    xd[:, :C] = x.double()
    xd = xd.view(R, G, 32)
    bad = ~torch.isfinite(xd).all(2)
    xd = torch.where(bad[:, :, None], 0.0, xd)
    top = xd.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 7, least).clamp_min(least).double()
    q = (xd / torch.exp2(e)[:, :, None]).round().clamp(-127, 127)
    value = torch.where(bad[:, :, None], NAN, q * torch.exp2(e)[:, :, None])
    byte = torch.where(bad, 255, e + 127)
    return q.view(R, -1)[:, :C], byte, value.view(R, -1)[:, :C]


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (5, 32), (7, 33), (64, 512), (33, 1000), (2, 4096), (1000, 96)],
                         ids=str)
def test_keep8(shape, ty):
    code, dtype, _ = TYPES[ty]
    R, C = shape
    g = gen(R * C)
    x = torch.randn(R, C, generator=g, device="cuda") * torch.exp2(
        torch.randint(-30, 12, (R, C), generator=g, device="cuda").float())
    x = x.to(dtype)
    flat = x.view(-1)
    flat[:: 97] = 0
    flat[: min(32, C)] = 0           # an empty group
    if R > 2:
        x[1, C // 2], x[2, 0] = NAN, float("-inf")
    q = torch.empty(R, C, dtype=torch.int8, device="cuda")
    s = torch.empty(R, -(-C // 32), dtype=torch.uint8, device="cuda")
    back = torch.empty(R, C, dtype=dtype, device="cuda")
    gp.gemmpipe_keep8(code, R, C, x, C, q, s)
    gp.gemmpipe_restore8(code, R, C, q, s, back, C)
    wq, ws, wv = keep8_reference(x, -24 if ty == "f16" else -127)
    assert torch.equal(q.double(), wq) and torch.equal(s.double(), ws)
    assert torch.equal(torch.nan_to_num(back.double(), nan=7e9), torch.nan_to_num(wv, nan=7e9))
    # Pitched and misaligned rows give the same.
    for ld, shift in ((C + 8, 8), (C + 5, 1)):
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        gp.gemmpipe_keep8(code, R, C, pitched(x, ld, shift), ld, q2, s2)
        assert torch.equal(q2, q) and torch.equal(s2, s)
        b2 = pitched(torch.zeros_like(back), ld, shift)
        gp.gemmpipe_restore8(code, R, C, q, s, b2, ld)
        assert torch.equal(torch.nan_to_num(b2, nan=77.0), torch.nan_to_num(back, nan=77.0))


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", [(1025, 1), (1030, 100), (1027, 257), (1026, 520), (1031, 777), (1500, 2001),
                                   (1025, 8300), (5, 257), (6, 513), (3, 2049), (2, 8500)], ids=str)
def test_keep8_rows_in_blocks(shape, ty):
    # Few and many rows of one span of 256 values up to more than a block takes.
    test_keep8(shape, ty)


@pytest.mark.parametrize("ty", TYPES)
def test_keep8_extremes(ty):
    # The type's largest, its smallest, and every power of two between.
    code, dtype, _ = TYPES[ty]
    info = torch.finfo(dtype)
    tiny = 2.0 ** -24 if ty == "f16" else 2.0 ** -133
    lo, hi = (-24, 15) if ty == "f16" else (-133, 127)
    rows = [[info.max] * 32, [-info.max] + [1.0] * 31, [tiny] * 32, [0.0] * 31 + [-tiny]]
    rows += [[2.0 ** p, 2.0 ** p * (2 - info.eps), -(2.0 ** p)] + [2.0 ** (p - 7)] * 29 for p in range(lo + 11, hi)]
    x = torch.tensor(rows, dtype=torch.float64, device="cuda").to(dtype)
    R, C = x.shape
    q = torch.empty(R, C, dtype=torch.int8, device="cuda")
    s = torch.empty(R, 1, dtype=torch.uint8, device="cuda")
    back = torch.empty_like(x)
    gp.gemmpipe_keep8(code, R, C, x, C, q, s)
    gp.gemmpipe_restore8(code, R, C, q, s, back, C)
    wq, ws, wv = keep8_reference(x, lo if ty == "f16" else -127)
    assert torch.equal(q.double(), wq) and torch.equal(s.double(), ws) and torch.equal(back.double(), wv)
    assert bool(torch.isfinite(back).all())


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("counts", ["few", "mean_96", "large"])
def test_gradient_to_weights_from_8_bits(counts, size, ty):
    code, dtype, u = TYPES[ty]
    K, N = size
    c = COUNTS[counts]
    off, R, X, dY, W = setup(c, K, N, dtype, seed=13, head=2, unused=9)
    q = torch.empty(R, K, dtype=torch.int8, device="cuda")
    s = torch.empty(R, -(-K // 32), dtype=torch.uint8, device="cuda")
    gp.gemmpipe_keep8(code, R, K, X, K, q, s)  # the NaN rows among them
    dW = torch.full((len(c), K, N), 3.0, dtype=dtype, device="cuda")
    gp.gemm_grouped_dw8(code, R, N, K, len(c), q, s, dY, N, off, dW)
    _, _, value = keep8_reference(X, -24 if ty == "f16" else -127)
    exact, mag = weights_reference(off, value, dY)
    check_close(dW, exact, product_bound(u, max(c), exact, mag))
    rounded = torch.empty(R, K, dtype=dtype, device="cuda")
    gp.gemmpipe_restore8(code, R, K, q, s, rounded, K)
    other = torch.empty_like(dW)
    gp.gemm_grouped_dw(code, R, N, K, len(c), rounded, K, dY, N, off, other)
    assert torch.equal(dW, other)


# ------------------------------------------------- streams, repeats, errors


def test_results_repeat_and_follow_the_stream():
    K, N, E, T, k = 520, 392, 6, 300, 2
    g, rows, kept = routing(T, k, E, seed=2)
    R = T * k
    X, W, w = randn(g, T, K), randn(g, E, K, N, scale=0.05), torch.rand(T, k, generator=g, device="cuda")
    ids = torch.randint(0, E, (R,), generator=g, device="cuda").int()
    torch.cuda.synchronize()

    def once(stream):
        new = lambda *s, ty=torch.float16: torch.empty(*s, dtype=ty, device="cuda")  # noqa: E731
        off, slots, at = new(E + 1, ty=torch.int32), new(R, ty=torch.int32), new(R, ty=torch.int32)
        Xs, Ys, Y, dYs, dw = new(R, K), new(R, N), new(T, N), new(R, N), new(T, k, ty=torch.float32)
        dX, dW, dT = new(R, K), new(E, K, N), new(T, K)
        torch.cuda.synchronize()
        gp.gemmpipe_route(T, k, E, ids, off, slots, at, stream)
        gp.gemmpipe_dispatch(gp.F16, T, k, K, X, K, at, None, Xs, K, stream)
        gp.gemm_grouped(gp.F16, R, N, K, E, Xs, K, off, W, Ys, N, stream)
        gp.gemmpipe_combine(gp.F16, T, k, N, Ys, N, at, w, Y, N, stream)
        gp.gemmpipe_combine_grad(gp.F16, T, k, N, Y, N, Ys, N, at, w, dYs, N, dw, stream)
        gp.gemm_grouped_dx(gp.F16, R, N, K, E, dYs, N, off, W, dX, K, stream)
        gp.gemm_grouped_dw(gp.F16, R, N, K, E, Xs, K, dYs, N, off, dW, stream)
        gp.gemmpipe_combine(gp.F16, T, k, K, dX, K, at, None, dT, K, stream)
        torch.cuda.synchronize()
        return off, slots, at, Xs, Ys, Y, dYs, dw, dX, dW, dT

    first = once(None)
    side = torch.cuda.Stream()
    for again in (once(None), once(side), once(side)):
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_captured_in_a_graph():
    K, N, E, T, k = 256, 128, 8, 16, 2
    g = gen(6)
    R = T * k
    ids = torch.randint(0, E, (R,), generator=g, device="cuda").int()
    X, W, w = randn(g, T, K), randn(g, E, K, N, scale=0.05), torch.rand(T, k, generator=g, device="cuda")
    off, slots, at = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, R, R))
    Xs, Ys, Y = (torch.empty(*s, dtype=torch.float16, device="cuda") for s in ((R, K), (R, N), (T, N)))

    def step():
        gp.gemmpipe_route(T, k, E, ids, off, slots, at)
        gp.gemmpipe_dispatch(gp.F16, T, k, K, X, K, at, None, Xs, K)
        gp.gemm_grouped(gp.F16, R, N, K, E, Xs, K, off, W, Ys, N)
        gp.gemmpipe_combine(gp.F16, T, k, N, Ys, N, at, w, Y, N)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(torch.randint(0, E, (R,), generator=g, device="cuda").int())
    X.copy_(randn(g, T, K))
    graph.replay()
    torch.cuda.synchronize()
    seen = Y.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(seen, Y) and bool(torch.isfinite(Y).all())


def test_host_memory_is_refused():
    host = torch.zeros(64, 64, dtype=torch.float16)
    dev = torch.zeros(64, 64, dtype=torch.float16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    for args in ((host, 64, off, dev, dev, 64), (dev, 64, off, host, dev, 64), (dev, 64, off, dev, host, 64),
                 (dev, 64, off.cpu(), dev, dev, 64)):
        with pytest.raises(gp.GemmpipeError) as e:
            gp.gemm_grouped(gp.F16, 64, 64, 64, 1, *args)
        assert e.value.status == gp.ERR_INVALID_VALUE


@pytest.mark.parametrize("mean", [4, 300])
def test_a_stalled_pipeline_times_out(mean):
    # The wait for a k-block that never arrives ends the kernel, which reports it; the next call is unharmed.
    K, N, E = 512, 256, 2
    off, R, X, dY, W = setup([mean, mean], K, N, torch.float16, seed=21)
    Y = torch.empty(R, N, dtype=torch.float16, device="cuda")
    dW = torch.empty(E, K, N, dtype=torch.float16, device="cuda")
    calls = [lambda: gp.gemm_grouped(gp.F16, R, N, K, E, X, K, off, W, Y, N),
             lambda: gp.gemm_grouped_dw(gp.F16, R, N, K, E, X, K, dY, N, off, dW)]
    for call in calls:
        gp.gemmpipe_test_inject_stall(0, 50)
        call()
        assert gp.gemmpipe_get_device_status() == gp.ERR_TIMEOUT
        call()
        assert gp.gemmpipe_get_device_status() == gp.OK
    exact, mag = rows_reference(off, X, W)
    check_close(Y, exact, product_bound(2.0 ** -11, K, exact, mag))
    exact, mag = weights_reference(off, X, dY)
    check_close(dW, exact, product_bound(2.0 ** -11, mean, exact, mag))
