"""Workloads of the expert-layer operators: token routing, the grouped products
and the 8-bit activation copies, with their plain forms in elementary torch
operations.

With `own` false, run() computes a pass in 32 bits with elementary torch
operations; with `own` true it makes the calls of the library's binding.
exact() computes the same results in 64 bits, expert by expert.

A case is a dict: "op" says which operator, "type" the element type of the
activations and weights ("f16" or "bf16"), the rest are sizes:
  tokens, top_k, experts   tokens, experts chosen per token, experts in all
  inner, outer             a weight matrix has inner x outer elements
  width                    elements of one activation row
  drop                     share of the tokens that go to no expert (padding)
  skew                     spread of the router's preference among experts
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_CODE = {"f16": 0, "bf16": 1}
_GROUP = 32  # elements that share one scale of the 8-bit copy


def listed():
    return [
        # One generated token of one request: latency of the routing step.
        {"name": "route_one", "op": "route", "type": "f16", "tokens": 1, "top_k": 8, "experts": 64, "width": 2048,
         "drop": 0.0, "skew": 0.5},
        # A large prefill batch with padding tokens, many experts.
        {"name": "route_prompt", "op": "route", "type": "bf16", "tokens": 16384, "top_k": 8, "experts": 128,
         "width": 2048, "drop": 0.03, "skew": 0.5},
        # One decoding step of a small batch, rows back to token order.
        {"name": "combine_step", "op": "combine", "type": "f16", "tokens": 33, "top_k": 8, "experts": 64,
         "width": 2048, "drop": 0.0, "skew": 0.5},
        # A prefill of ragged length, odd width.
        {"name": "combine_odd", "op": "combine", "type": "f16", "tokens": 4093, "top_k": 4, "experts": 32,
         "width": 3001, "drop": 0.02, "skew": 0.5},
        # The weighted sum's gradient in a training step.
        {"name": "combine_grad", "op": "combine_grad", "type": "bf16", "tokens": 8192, "top_k": 8, "experts": 64,
         "width": 4096, "drop": 0.0, "skew": 0.5},
        # One token's experts: every weight byte is used once.
        {"name": "product_one", "op": "product", "type": "bf16", "tokens": 1, "top_k": 8, "experts": 64,
         "inner": 2048, "outer": 1024, "drop": 0.0, "skew": 0.5},
        # A decoding step of a batch: a handful of rows for each expert.
        {"name": "product_step", "op": "product", "type": "f16", "tokens": 64, "top_k": 8, "experts": 64,
         "inner": 4096, "outer": 1536, "drop": 0.0, "skew": 0.5},
        # A training batch or a long prefill.
        {"name": "product_train", "op": "product", "type": "f16", "tokens": 16384, "top_k": 4, "experts": 64,
         "inner": 4096, "outer": 1536, "drop": 0.0, "skew": 0.5},
        # Gradient to the rows, with sizes off every tile and pitch.
        {"name": "product_dx_odd", "op": "product_dx", "type": "f16", "tokens": 4093, "top_k": 4, "experts": 24,
         "inner": 4107, "outer": 1001, "drop": 0.02, "skew": 0.5},
        # Gradient to the weights in a training step.
        {"name": "product_dw", "op": "product_dw", "type": "bf16", "tokens": 8192, "top_k": 4, "experts": 32,
         "inner": 4096, "outer": 1536, "drop": 0.0, "skew": 0.5},
        # The rows of a training step put away in 8 bits and brought back.
        {"name": "keep8_train", "op": "keep8", "type": "bf16", "tokens": 32768, "top_k": 1, "experts": 1,
         "width": 4096, "drop": 0.0, "skew": 0.0},
        # Gradient to the weights from the rows kept in 8 bits.
        {"name": "keep8_dw", "op": "keep8_dw", "type": "bf16", "tokens": 8192, "top_k": 4, "experts": 32,
         "inner": 4096, "outer": 1536, "drop": 0.0, "skew": 0.5},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row's length: whole 64s more often than not, anything the rest."""
    if rng.random() < 0.4:
        return _spread(rng, low, high)
    blocks = _spread(rng, low // 64, high // 64)
    return 64 * (47 if blocks == 48 else blocks)


def draw(rng):
    op = rng.choice(["route", "combine", "combine_grad", "product", "product", "product_dx", "product_dw", "keep8",
                     "keep8_dw"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"]), "drop": rng.choice([0.0, 0.0, 0.05]),
            "skew": rng.choice([0.0, 0.5, 1.5])}
    size = lambda low, high: _width(rng, low, high)  # noqa: E731
    if op == "keep8":
        return {**case, "tokens": _spread(rng, 1, 32768), "top_k": 1, "experts": 1, "width": size(64, 4096),
                "drop": 0.0, "skew": 0.0}
    case["experts"] = _spread(rng, 8, 128)
    case["top_k"] = rng.choice([1, 2, 4, 8])
    if op in ("route", "combine", "combine_grad"):
        return {**case, "tokens": _spread(rng, 1, 65536 // case["top_k"]), "width": size(64, 4096)}
    case["experts"] = min(case["experts"], 64)
    least = 1 if op == "product" else 256
    return {**case, "tokens": _spread(rng, least, 65536 // case["top_k"]), "inner": size(256, 4096),
            "outer": size(256, 1536)}


def work(case):
    """Bytes and operations of one pass: every input once, every output once
    (8-bit copies: a byte per value and one per group of 32)."""
    rows, op = case["tokens"] * case["top_k"], case["op"]
    if op == "route":
        return {"bytes": 2 * case["width"] * (case["tokens"] + rows) + 12 * rows + 4 * case["experts"], "flops": 0}
    if op == "combine":
        return {"bytes": 2 * case["width"] * (case["tokens"] + rows) + 8 * rows, "flops": 2 * rows * case["width"]}
    if op == "combine_grad":
        return {"bytes": 2 * case["width"] * (case["tokens"] + 2 * rows) + 12 * rows,
                "flops": 3 * rows * case["width"]}
    if op == "keep8":
        return {"bytes": rows * case["width"] * 2 * 3 + rows * -(-case["width"] // _GROUP) * 2, "flops": 0}
    k, n = case["inner"], case["outer"]
    matrices = min(case["experts"], rows) if op in ("product", "product_dx") else case["experts"]
    kept = rows * (k + -(-k // _GROUP)) if op == "keep8_dw" else 2 * rows * k
    return {"bytes": kept + 2 * rows * n + 2 * matrices * k * n, "flops": 2 * rows * k * n}


def _routing(case, g):
    """Expert ids of every token's choices (distinct per token, -1 for padding
    tokens) and their weights, as a router gives them."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    liking = torch.randn(e, generator=g, device="cuda") * case["skew"]
    scores = torch.randn(t, e, generator=g, device="cuda") + liking
    best, ids = scores.topk(k, dim=1)
    weights = torch.softmax(best, dim=1)
    dropped = torch.rand(t, generator=g, device="cuda") < case["drop"]
    ids = torch.where(dropped[:, None], -1, ids).to(torch.int32)
    return ids.contiguous(), weights.contiguous()


def _sorted_rows(ids, experts):
    """offsets, slots and rows of a stable sort of the choices by expert; the
    dropped ones come last, in order, marked by the complement."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, experts)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    ends = (key[None, :] <= torch.arange(experts, device=key.device)[:, None]).sum(1) if key.numel() <= 1024 else \
        torch.cumsum(torch.bincount(key, minlength=experts + 1)[:experts], 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    rows = torch.where(kept, place, ~place)
    slots = torch.where(kept[order], order, ~order)
    return offsets.to(torch.int32), slots.to(torch.int32), rows.to(torch.int32)


def _randn(g, *shape, type_, scale=1.0):
    """Normal values made in parts, so that no 32-bit copy of a large tensor is held."""
    out = torch.empty(shape, dtype=type_, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * scale)
    return out


def _power(exponent):
    """2 to the power of whole numbers from -127 to 127, exactly (by its bits)."""
    return torch.where(exponent > -127, (exponent + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _group_exponents(x32, type_):
    """Exponent of the shared scale of every group of 32 along the rows: that of
    the group's largest magnitude less 6, so that it becomes 64 to 127 steps."""
    pad = -x32.shape[1] % _GROUP
    grouped = torch.nn.functional.pad(x32, (0, pad)).view(x32.shape[0], -1, _GROUP)
    least = -24 if type_ == "f16" else -127
    top = grouped.abs().amax(2)
    return grouped, torch.where(top > 0, (torch.frexp(top).exponent - 7).clamp(least, 127), least)


def _pack(x, type_):
    """(whole numbers, scale bytes) of the rows in 8 bits."""
    grouped, exponent = _group_exponents(x.float(), type_)
    q = torch.round(grouped * _power(-exponent)[:, :, None]).clamp(-127, 127)
    return q.view(x.shape[0], -1)[:, :x.shape[1]].to(torch.int8).contiguous(), (exponent + 127).to(torch.uint8)


def _unpack(q, s):
    """The values that the 8-bit rows stand for, in 32 bits."""
    pad = -q.shape[1] % _GROUP
    grouped = torch.nn.functional.pad(q.float(), (0, pad)).view(q.shape[0], -1, _GROUP)
    return (grouped * _power(s.to(torch.int32) - 127)[:, :, None]).view(q.shape[0], -1)[:, :q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, ty = case["op"], _TYPES[case["type"]]
    t, e, r = case["tokens"], case["experts"], case["tokens"] * case["top_k"]
    new = lambda *shape, type_=ty: torch.empty(shape, dtype=type_, device="cuda")  # noqa: E731
    s = {"case": case}
    if op == "keep8":
        w = case["width"]
        # Activations: a few channels far larger than the rest.
        loud = torch.exp2(4 * (torch.rand(w, generator=g, device="cuda") < 0.01).float())
        s["x"] = new(r, w)
        for part in s["x"].split(max(1, (1 << 27) // w)):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * loud)
        s["q"], s["s"] = new(r, w, type_=torch.int8), new(r, -(-w // _GROUP), type_=torch.uint8)
        s["out"] = new(r, w)
        return s
    ids, weights = _routing(case, g)
    offsets, slots, rows = _sorted_rows(ids, e)
    unused = slots < 0  # rows past the last kept one: a user's buffer holds anything there
    if op == "route":
        s |= {"ids": ids, "x": _randn(g, t, case["width"], type_=ty), "xs": new(r, case["width"])}
        s |= {"offsets": new(e + 1, type_=torch.int32), "slots": new(r, type_=torch.int32),
              "rows": new(t, case["top_k"], type_=torch.int32)}
    elif op in ("combine", "combine_grad"):
        s |= {"rows": rows.view(t, -1), "weights": weights, "ys": _randn(g, r, case["width"], type_=ty)}
        s["ys"][unused] = math.nan
        if op == "combine":
            s["y"] = new(t, case["width"])
        else:
            s |= {"dy": _randn(g, t, case["width"], type_=ty, scale=0.1), "dys": new(r, case["width"]),
                  "dweights": new(t, case["top_k"], type_=torch.float32)}
    else:
        k, n = case["inner"], case["outer"]
        s["offsets"] = offsets
        if op in ("product", "product_dx"):
            s["w"] = _randn(g, e, k, n, type_=ty, scale=k ** -0.5)
        if op in ("product", "product_dw", "keep8_dw"):
            s["x"] = _randn(g, r, k, type_=ty)
            s["x"][unused] = math.nan
        if op == "product":
            s["y"] = new(r, n)
        else:
            s["dy"] = _randn(g, r, n, type_=ty, scale=0.1)
            s["dy"][unused] = math.nan
        if op == "product_dx":
            s["dx"] = new(r, k)
        if op in ("product_dw", "keep8_dw"):
            s["dw"] = new(e, k, n)
        if op == "keep8_dw":
            x = s.pop("x")
            x[unused] = 0
            s["q"], s["s"] = _pack(x, case["type"])
            s["s"][unused] = 255
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from software_pipelined_loop_gb300 import gemmpipe as gp
    c, ty = s["case"], _CODE[s["case"]["type"]]
    op, t, k, e = c["op"], c["tokens"], c["top_k"], c["experts"]
    r = t * k
    if op == "route":
        gp.gemmpipe_route(t, k, e, s["ids"], s["offsets"], s["slots"], s["rows"])
        gp.gemmpipe_dispatch(ty, t, k, c["width"], s["x"], c["width"], s["rows"], None, s["xs"], c["width"])
        return {n: s[n] for n in ("offsets", "slots", "rows", "xs")}
    if op == "combine":
        gp.gemmpipe_combine(ty, t, k, c["width"], s["ys"], c["width"], s["rows"], s["weights"], s["y"], c["width"])
        return s["y"]
    if op == "combine_grad":
        gp.gemmpipe_combine_grad(ty, t, k, c["width"], s["dy"], c["width"], s["ys"], c["width"], s["rows"],
                                 s["weights"], s["dys"], c["width"], s["dweights"])
        return {"dys": s["dys"], "dweights": s["dweights"]}
    if op == "keep8":
        gp.gemmpipe_keep8(ty, r, c["width"], s["x"], c["width"], s["q"], s["s"])
        gp.gemmpipe_restore8(ty, r, c["width"], s["q"], s["s"], s["out"], c["width"])
        return s["out"]
    i, o = c["inner"], c["outer"]
    if op == "product":
        gp.gemm_grouped(ty, r, o, i, e, s["x"], i, s["offsets"], s["w"], s["y"], o)
        return s["y"]
    if op == "product_dx":
        gp.gemm_grouped_dx(ty, r, o, i, e, s["dy"], o, s["offsets"], s["w"], s["dx"], i)
        return s["dx"]
    if op == "product_dw":
        gp.gemm_grouped_dw(ty, r, o, i, e, s["x"], i, s["dy"], o, s["offsets"], s["dw"])
        return s["dw"]
    gp.gemm_grouped_dw8(ty, r, o, i, e, s["q"], s["s"], s["dy"], o, s["offsets"], s["dw"])
    return s["dw"]


def _by_expert(offsets, r):
    """For every row its expert, its place among that expert's rows and whether
    it has one, and the most rows of an expert."""
    at = torch.arange(r, device=offsets.device)
    offsets = offsets.long()
    expert = torch.searchsorted(offsets[1:], at, right=True)
    kept = expert < offsets.numel() - 1
    expert = torch.where(kept, expert, 0)
    return expert, at - offsets[expert], kept, max(1, int(offsets.diff().max()))


def _stacked(x32, expert, place, kept, experts, most):
    """Rows as a batch of one matrix per expert, zeros below its last row."""
    out = x32.new_zeros(experts, most, x32.shape[1])
    out[expert[kept], place[kept]] = x32[kept]
    return out


def _run_plain(s):
    c = s["case"]
    op, ty, t, k, e = c["op"], _TYPES[c["type"]], c["tokens"], c["top_k"], c["experts"]
    r = t * k
    if op == "route":
        offsets, slots, rows = _sorted_rows(s["ids"], e)
        kept = slots >= 0
        xs = torch.where(kept[:, None], s["x"][torch.where(kept, slots, ~slots).long() // k], 0)
        return {"offsets": offsets, "slots": slots, "rows": rows.view(t, k), "xs": xs}
    if op in ("combine", "combine_grad"):
        kept = s["rows"] >= 0
        place = torch.where(kept, s["rows"], ~s["rows"]).long()
        chosen = torch.where(kept[:, :, None], s["ys"][place].float(), 0.0)
        weights = torch.where(kept, s["weights"], 0.0)
        if op == "combine":
            return (chosen * weights[:, :, None]).sum(1).to(ty)
        dy = s["dy"].float()
        dys = torch.empty_like(s["ys"])
        dys[place] = (weights[:, :, None] * dy[:, None, :]).to(ty)
        return {"dys": dys, "dweights": (chosen * dy[:, None, :]).sum(2)}
    if op == "keep8":
        return _unpack(*_pack(s["x"], c["type"])).to(ty)
    expert, place, kept, most = _by_expert(s["offsets"], r)
    stack = lambda x: _stacked(x.float(), expert, place, kept, e, most)  # noqa: E731
    back = lambda y: torch.where(kept[:, None], y[expert, torch.where(kept, place, 0)], 0.0).to(ty)  # noqa: E731
    if op == "product":
        return back(torch.bmm(stack(s["x"]), s["w"].float()))
    if op == "product_dx":
        return back(torch.bmm(stack(s["dy"]), s["w"].float().transpose(1, 2)))
    x = _unpack(s["q"], s["s"]) if op == "keep8_dw" else s["x"]
    return torch.bmm(stack(x).transpose(1, 2), stack(s["dy"])).to(ty)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits; None in the place of
    the routing's whole numbers."""
    s = prepare(case, seed)
    op, t, k, e = case["op"], case["tokens"], case["top_k"], case["experts"]
    r = t * k
    if op == "route":
        ids = s["ids"].cpu().reshape(-1).tolist()
        xs = torch.zeros(r, case["width"], dtype=torch.float64, device="cuda")
        # One list of choices per expert, in order: row by row what each expert gets.
        lists = [[] for _ in range(e)]
        for slot, expert in enumerate(ids):
            if 0 <= expert < e:
                lists[expert].append(slot // k)
        tokens = torch.tensor([token for chosen in lists for token in chosen], dtype=torch.long, device="cuda")
        xs[:tokens.numel()] = s["x"].double()[tokens]
        return {"offsets": None, "slots": None, "rows": None, "xs": xs}
    if op == "combine":
        y = torch.zeros(t, case["width"], dtype=torch.float64, device="cuda")
        for j in range(k):
            has = s["rows"][:, j] >= 0
            y[has] += s["weights"][has, j].double()[:, None] * s["ys"][s["rows"][has, j].long()].double()
        return y
    if op == "combine_grad":
        dys = torch.zeros(r, case["width"], dtype=torch.float64, device="cuda")
        dweights = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            has = s["rows"][:, j] >= 0
            to, dy = s["rows"][has, j].long(), s["dy"][has].double()
            dys[to] = s["weights"][has, j].double()[:, None] * dy
            dweights[has, j] = torch.einsum("tc,tc->t", s["ys"][to].double(), dy)
        return {"dys": dys, "dweights": dweights}
    if op == "keep8":
        out = torch.empty(r, case["width"], dtype=torch.float64, device="cuda")
        least = -24 if case["type"] == "f16" else -127
        for c0 in range(0, case["width"], _GROUP):
            x = s["x"][:, c0:c0 + _GROUP].double()
            top = x.abs().amax(1).clamp_min(2.0 ** -200)
            step = torch.exp2((torch.floor(torch.log2(top) + 1e-9) - 6).clamp_min(least))
            out[:, c0:c0 + _GROUP] = (x / step[:, None]).round().clamp(-127, 127) * step[:, None]
        return out
    bounds = s["offsets"].cpu().tolist()
    i, o = case["inner"], case["outer"]
    if op in ("product", "product_dx"):
        out = torch.zeros(r, o if op == "product" else i, dtype=torch.float64, device="cuda")
        for n in range(e):
            at = slice(bounds[n], bounds[n + 1])
            w = s["w"][n].double()
            out[at] = s["x"][at].double() @ w if op == "product" else s["dy"][at].double() @ w.t()
        return out
    out = torch.zeros(e, i, o, dtype=torch.float64, device="cuda")
    for n in range(e):
        at = slice(bounds[n], bounds[n + 1])
        if op == "keep8_dw":
            steps = torch.exp2(s["s"][at].double() - 127).repeat_interleave(_GROUP, 1)[:, :i]
            x = s["q"][at].double() * steps
        else:
            x = s["x"][at].double()
        out[n] = x.t() @ s["dy"][at].double()
    return out
