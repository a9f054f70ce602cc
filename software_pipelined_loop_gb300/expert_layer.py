"""An expert layer for PyTorch on libgemmpipe's operators, forward and backward.

    y[t] = sum over the chosen experts e of token t:
               weight[t, e] * (silu(x[t] @ W1[e]) @ W2[e])

`expert_layer` is differentiable in x, the router's weights, W1 and W2; with
``keep8=True`` the rows that the weight gradients need (the inputs of both
products) are kept in 8 bits between the passes.  The routing's sort, the rows'
way to the experts and back, the products and their gradients run in the CUDA
library.  torch supplies memory, autograd's bookkeeping, the activation between
the products and its derivative; the choice of the experts and its weights are
the caller's.  Gradients of the gradients are refused.

    python -m software_pipelined_loop_gb300.expert_layer [--tokens N] [--keep8]

runs a training step and a one-token step on the GPU and prints their times.
"""
from __future__ import annotations

import argparse
import functools

import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

_CODE = {torch.float16: gp.F16, torch.bfloat16: gp.BF16}


def _check_ids(ids: torch.Tensor) -> None:
    if ids.dtype != torch.int32:
        raise TypeError(f"ids: int32 is needed, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError(f"ids: tokens x top_k is needed, got {tuple(ids.shape)}")


def _check_devices(first: torch.Tensor, *others: torch.Tensor) -> None:
    # The library launches on the current device's stream.
    here = torch.cuda.current_device() if first.is_cuda else -2
    for t in (first, *others):
        if t.get_device() != here:
            raise ValueError("tensors on the current CUDA device are needed, got " +
                             ", ".join(str(t.device) for t in (first, *others)))


def _check_arguments(x, ids, weights, w1, w2) -> None:
    ty = x.dtype
    if ty not in _CODE:
        raise TypeError(f"x: float16 or bfloat16 is needed, got {ty}")
    _check_ids(ids)
    if weights.dtype != torch.float32:
        raise TypeError(f"weights: float32 is needed, got {weights.dtype}")
    if w1.dtype != ty or w2.dtype != ty:
        raise TypeError(f"w1, w2: the type of x, {ty}, is needed, got {w1.dtype}, {w2.dtype}")
    if w1.dim() != 3:
        raise ValueError(f"w1: one matrix per expert is needed, got {tuple(w1.shape)}")
    choices, (experts, c, h) = ids.shape, w1.shape
    if x.shape != (choices[0], c) or weights.shape != choices or w2.shape != (experts, h, c):
        raise ValueError(f"x {(choices[0], c)}, weights {tuple(choices)} and w2 {(experts, h, c)} are needed, "
                         f"got {tuple(x.shape)}, {tuple(weights.shape)} and {tuple(w2.shape)}")
    _check_devices(x, ids, weights, w1, w2)


# The functions below hand their arguments to the library by address: they take
# dense tensors (expert_layer makes them so) and make their gradients dense.


def _empty(like, *shape, dtype=None):
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


class _Last(torch.autograd.Function):
    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the expert layer's gradients cannot be differentiated again")


def _once(backward):
    """For gradients made outside autograd: where a graph of them is asked for
    (create_graph), they get a node whose differentiation is an error, whatever
    else requires a gradient -- without one their derivatives would be dropped."""
    @functools.wraps(backward)
    def run(ctx, dy):
        if not torch.is_grad_enabled():
            return backward(ctx, dy)
        with torch.no_grad():
            grads = backward(ctx, dy)
        made = [g for g in grads if g is not None]
        if not made:
            return grads
        marked = iter(_Last.apply(torch.empty(0, requires_grad=True), *made))
        return tuple(g if g is None else next(marked) for g in grads)
    return run


def route(ids: torch.Tensor, experts: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(offsets, slots, rows) of the choices `ids` (tokens x top_k, int32), sorted by expert."""
    _check_ids(ids)
    _check_devices(ids)
    return _route(ids, experts)


def _route(ids, experts):
    t, k = ids.shape
    new = lambda n: torch.empty(n, dtype=torch.int32, device=ids.device)  # noqa: E731
    offsets, slots, rows = new(experts + 1), new(t * k), new(t * k)
    gp.gemmpipe_route(t, k, experts, ids.contiguous(), offsets, slots, rows)
    return offsets, slots, rows


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, k):
        t, c = x.shape
        xs = _empty(x, t * k, c)
        gp.gemmpipe_dispatch(_CODE[x.dtype], t, k, c, x, c, rows, None, xs, c)
        ctx.save_for_backward(rows)
        ctx.k = k
        return xs

    @staticmethod
    @_once
    def backward(ctx, dxs):
        rows, = ctx.saved_tensors
        dxs = dxs.contiguous()
        t, c = dxs.shape[0] // ctx.k, dxs.shape[1]
        dx = _empty(dxs, t, c)
        gp.gemmpipe_combine(_CODE[dxs.dtype], t, ctx.k, c, dxs, c, rows, None, dx, c)
        return dx, None, None


class _Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, keep8):
        r, k = x.shape
        e, _, n = w.shape
        y = _empty(x, r, n)
        gp.gemm_grouped(_CODE[x.dtype], r, n, k, e, x, k, offsets, w, y, n)
        # What the gradients that may be asked for need, and no more.
        x_grad, w_grad = ctx.needs_input_grad[:2]
        kept = ()
        if w_grad and keep8:
            kept = _empty(x, r, k, dtype=torch.int8), _empty(x, r, (k + 31) // 32, dtype=torch.uint8)
            gp.gemmpipe_keep8(_CODE[x.dtype], r, k, x, k, *kept)
        elif w_grad:
            kept = (x,)
        ctx.save_for_backward(offsets, w if x_grad else None, *kept)
        ctx.shape = e, k, n
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        offsets, w, *kept = ctx.saved_tensors
        dy = dy.contiguous()
        e, k, n = ctx.shape
        r, ty = dy.shape[0], _CODE[dy.dtype]
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = _empty(dy, r, k)
            gp.gemm_grouped_dx(ty, r, n, k, e, dy, n, offsets, w, dx, k)
        if ctx.needs_input_grad[1]:
            dw = _empty(dy, e, k, n)
            if len(kept) == 2:
                gp.gemm_grouped_dw8(ty, r, n, k, e, *kept, dy, n, offsets, dw)
            else:
                gp.gemm_grouped_dw(ty, r, n, k, e, *kept, k, dy, n, offsets, dw)
        return dx, dw, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, rows):
        t, k = weights.shape
        c = ys.shape[1]
        y = _empty(ys, t, c)
        gp.gemmpipe_combine(_CODE[ys.dtype], t, k, c, ys, c, rows, weights, y, c)
        ctx.save_for_backward(ys, weights, rows)
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        ys, weights, rows = ctx.saved_tensors
        dy = dy.contiguous()
        t, k = weights.shape
        c = ys.shape[1]
        dys, dweights = torch.empty_like(ys), torch.empty_like(weights)
        gp.gemmpipe_combine_grad(_CODE[ys.dtype], t, k, c, dy, c, ys, c, rows, weights, dys, c, dweights)
        return dys, dweights, None


def expert_layer(x, ids, weights, w1, w2, keep8: bool = False):
    """x: tokens x c; ids: tokens x top_k int32 (outside [0, experts): dropped);
    weights: tokens x top_k fp32; w1: experts x c x h; w2: experts x h x c.
    x, w1 and w2 have one 16-bit floating-point type.  Strided tensors are
    copied to dense ones first; another type, shape or device is refused."""
    _check_arguments(x, ids, weights, w1, w2)
    keep8 = keep8 and torch.is_grad_enabled()  # (needs_input_grad goes by the tensors alone)
    offsets, _, rows = _route(ids, w1.shape[0])
    xs = _Dispatch.apply(x.contiguous(), rows, ids.shape[1])
    hidden = torch.nn.functional.silu(_Product.apply(xs, w1.contiguous(), offsets, keep8))
    ys = _Product.apply(hidden, w2.contiguous(), offsets, keep8)
    return _Combine.apply(ys, weights.contiguous(), rows)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--keep8", action="store_true", help="keep the saved rows in 8 bits")
    args = ap.parse_args()
    top_k, experts, c, h = 4, 32, 2048, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w1 = (rand(experts, c, h) * c ** -0.5).bfloat16().requires_grad_()
    w2 = (rand(experts, h, c) * h ** -0.5).bfloat16().requires_grad_()

    def inputs(tokens):
        best, ids = rand(tokens, experts).topk(top_k, dim=1)
        return rand(tokens, c).bfloat16().requires_grad_(), ids.int(), torch.softmax(best, 1).requires_grad_()

    def timed(step, reps=10):
        step()
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(reps):
            step()
        stop.record()
        torch.cuda.synchronize()
        return start.elapsed_time(stop) / reps

    x, ids, weights = inputs(args.tokens)
    target = rand(args.tokens, c).bfloat16()

    def train():
        for leaf in (x, weights, w1, w2):
            leaf.grad = None
        expert_layer(x, ids, weights, w1, w2, args.keep8).backward(target)

    ms = timed(train)
    flops = 3 * 2 * 2 * args.tokens * top_k * c * h
    print(f"training step, {args.tokens} tokens x {top_k} of {experts} experts, {c} x {h}: {ms:.3f} ms "
          f"({flops / ms / 1e9:.0f} TFLOP/s)")
    one = inputs(1)
    with torch.no_grad():
        print(f"one token: {timed(lambda: expert_layer(*one, w1, w2), 100) * 1e3:.1f} us")
    status = gp.gemmpipe_get_device_status()
    if status != gp.OK:
        raise SystemExit(f"device status {gp.STATUS.get(status, status)}")


if __name__ == "__main__":
    main()
