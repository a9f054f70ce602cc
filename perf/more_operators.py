"""Workloads of the few-token operators: rows times weights in 4 bits, the whole
expert layer for a few tokens (weights in 16 or in 4 bits), and the way of
weights into 4 bits and back, with their plain forms in elementary torch
operations.

With `own` false, run() computes a pass in 32 bits with elementary torch
operations; with `own` true it makes the calls of the library's binding.
exact() computes the same results in 64 bits, expert by expert.

A case is a dict: "op" says which operator, "type" the element type of the
activations, scales and 16-bit weights ("f16" or "bf16"), the rest are sizes:
  rows, inner, outer       rows4: rows times an inner x outer matrix
  tokens, top_k, experts   tokens, experts chosen per token, experts in all
  width, hidden            an expert's matrices: width x hidden and back
  gated                    whether a third matrix gates the hidden values
  group                    rows of a weight matrix that share a scale
  drop                     share of the choices that go to no expert
  skew                     spread of the router's preference among experts

Weights in 4 bits: a 32-bit word holds eight rows k = 8b .. 8b+7 of one column,
row 8b + [0, 2, 4, 6, 1, 3, 5, 7][i] in its bits 4i .. 4i+3, as value + 8; the
words of a row block b lie side by side, columns rounded up to a multiple of 4,
and so do the scales of a group of rows.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_CODE = {"f16": 0, "bf16": 1}
_ROW_OF_NIBBLE = [0, 2, 4, 6, 1, 3, 5, 7]


def listed():
    return [
        # One generated token through a small projection: latency.
        {"name": "rows4_small", "op": "rows4", "type": "f16", "rows": 1, "inner": 2048, "outer": 2048, "group": 128},
        # One generated token through a wide projection: every weight byte is used once.
        {"name": "rows4_one", "op": "rows4", "type": "bf16", "rows": 1, "inner": 4096, "outer": 16384, "group": 128},
        # A few sequences, sizes off every tile, pitch and group.
        {"name": "rows4_odd", "op": "rows4", "type": "f16", "rows": 3, "inner": 4107, "outer": 3001, "group": 64},
        # A decoding step of a large batch: fewest weights a scale, most products.
        {"name": "rows4_batch", "op": "rows4", "type": "bf16", "rows": 64, "inner": 16384, "outer": 4096,
         "group": 32},
        # One generated token through its experts.
        {"name": "step_one", "op": "step", "type": "bf16", "tokens": 1, "top_k": 8, "experts": 64, "width": 2048,
         "hidden": 1024, "gated": True, "drop": 0.0, "skew": 0.5},
        # A few sequences, some of them finished, sizes off every tile and pitch.
        {"name": "step_odd", "op": "step", "type": "f16", "tokens": 5, "top_k": 4, "experts": 24, "width": 4107,
         "hidden": 1001, "gated": False, "drop": 0.05, "skew": 0.5},
        # A decoding step of a batch: a handful of rows for each expert.
        {"name": "step_batch", "op": "step", "type": "f16", "tokens": 64, "top_k": 8, "experts": 64, "width": 4096,
         "hidden": 1536, "gated": True, "drop": 0.0, "skew": 0.5},
        # One generated token, many experts in 4 bits.
        {"name": "step4_one", "op": "step4", "type": "bf16", "tokens": 1, "top_k": 8, "experts": 128, "width": 4096,
         "hidden": 1536, "gated": True, "group": 128, "drop": 0.0, "skew": 0.5},
        # A few sequences, odd sizes, 4 bits.
        {"name": "step4_odd", "op": "step4", "type": "f16", "tokens": 9, "top_k": 4, "experts": 24, "width": 4107,
         "hidden": 1001, "gated": False, "group": 64, "drop": 0.05, "skew": 0.5},
        # A decoding step of a batch, 4 bits, fewest weights a scale.
        {"name": "step4_batch", "op": "step4", "type": "bf16", "tokens": 48, "top_k": 8, "experts": 64, "width": 4096,
         "hidden": 1536, "gated": True, "group": 32, "drop": 0.0, "skew": 0.5},
        # A large matrix into 4 bits, and back for a long prompt's products.
        {"name": "pack4_matrix", "op": "pack4", "type": "bf16", "experts": 1, "inner": 4096, "outer": 16384,
         "group": 128},
        # The odd experts' matrices into 4 bits and back.
        {"name": "pack4_odd", "op": "pack4", "type": "f16", "experts": 24, "inner": 4107, "outer": 1001, "group": 32},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row's length: whole 64s more often than not, anything the rest."""
    if rng.random() < 0.4:
        return _spread(rng, low, high)
    return 64 * _spread(rng, max(1, low // 64), high // 64)


def draw(rng):
    op = rng.choice(["rows4", "rows4", "step", "step", "step4", "step4", "pack4"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op != "step":
        case["group"] = rng.choice([32, 64, 128])
    if op == "rows4":
        return {**case, "rows": _spread(rng, 1, 64), "inner": _width(rng, 64, 16384), "outer": _width(rng, 64, 16384)}
    if op == "pack4":
        return {**case, "experts": _spread(rng, 1, 32), "inner": _width(rng, 64, 4096),
                "outer": _width(rng, 64, 4096)}
    return {**case, "tokens": _spread(rng, 1, 64), "top_k": rng.choice([1, 2, 4, 8]),
            "experts": _spread(rng, 8, 64), "width": _width(rng, 64, 4096), "hidden": _width(rng, 64, 1536),
            "gated": rng.random() < 0.6, "drop": rng.choice([0.0, 0.0, 0.1]), "skew": rng.choice([0.0, 0.5, 1.5])}


def work(case):
    """Bytes and operations of one pass: every input once (of the experts those
    that the choices can reach), every output once."""
    op = case["op"]
    if op in ("rows4", "pack4"):
        k, n = case["inner"], case["outer"]
        kept = k * n // 2 + 2 * -(-k // case["group"]) * n
        if op == "pack4":
            return {"bytes": case["experts"] * 2 * (2 * k * n + kept), "flops": 0}
        return {"bytes": kept + 2 * case["rows"] * (k + n), "flops": 2 * case["rows"] * k * n}
    t, c, h, slots = case["tokens"], case["width"], case["hidden"], case["tokens"] * case["top_k"]
    matrices = 3 if case["gated"] else 2
    per = 2 * c * h
    if op == "step4":
        per = c * h // 2 + 2 * -(-c // case["group"]) * h
    return {"bytes": min(case["experts"], slots) * matrices * per + 4 * t * c + 8 * slots,
            "flops": 2 * slots * matrices * c * h}


def _randn(g, *shape, type_, scale=1.0):
    """Normal values made in parts, so that no 32-bit copy of a large tensor is held."""
    out = torch.empty(shape, dtype=type_, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * scale)
    return out


def _round4(n):
    return (n + 3) // 4 * 4


def _random4(g, experts, k, n, group, type_):
    """Random weights in 4 bits: whole words (columns past n: anything) and scales
    that bring the values to about k ** -0.5."""
    words = torch.randint(-2 ** 31, 2 ** 31, (experts, -(-k // 8), _round4(n)), generator=g, device="cuda",
                          dtype=torch.int32)
    scales = torch.empty(experts, -(-k // group), _round4(n), device="cuda")
    scales.uniform_(0.12, 0.32, generator=g)
    return words, (scales * k ** -0.5).to(type_)


def _choices(case, g):
    """Expert ids of every token's choices (distinct per token, -1 where dropped)
    and their weights, as a router gives them."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    liking = torch.randn(e, generator=g, device="cuda") * case["skew"]
    best, ids = (torch.randn(t, e, generator=g, device="cuda") + liking).topk(k, dim=1)
    dropped = torch.rand(t, k, generator=g, device="cuda") < case["drop"]
    return torch.where(dropped, -1, ids).to(torch.int32).contiguous(), torch.softmax(best, dim=1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, ty = case["op"], _TYPES[case["type"]]
    new = lambda *shape, type_=ty: torch.empty(shape, dtype=type_, device="cuda")  # noqa: E731
    s = {"case": case}
    if op == "rows4":
        m, k, n = case["rows"], case["inner"], case["outer"]
        s["x"], s["y"] = _randn(g, m, k, type_=ty), new(m, n)
        s["q"], s["s"] = _random4(g, 1, k, n, case["group"], ty)
        return s
    if op == "pack4":
        e, k, n = case["experts"], case["inner"], case["outer"]
        s["w"], s["out"] = _randn(g, e, k, n, type_=ty, scale=k ** -0.5), new(e, k, n)
        s["q"] = new(e, -(-k // 8), _round4(n), type_=torch.int32)
        s["s"] = new(e, -(-k // case["group"]), _round4(n))
        return s
    t, e, c, h = case["tokens"], case["experts"], case["width"], case["hidden"]
    s["ids"], s["weights"] = _choices(case, g)
    s["x"], s["y"] = _randn(g, t, c, type_=ty), new(t, c)
    s["hidden"] = new(t * case["top_k"], (h + 7) // 8 * 8)
    sides = [("1", c, h), ("2", h, c)] + [("3", c, h)] * case["gated"]
    for name, k, n in sides:
        if op == "step":
            s["w" + name] = _randn(g, e, k, n, type_=ty, scale=k ** -0.5)
        else:
            s["q" + name], s["s" + name] = _random4(g, e, k, n, case["group"], ty)
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from software_pipelined_loop_gb300 import gemmpipe as gp
    c, ty = s["case"], _CODE[s["case"]["type"]]
    op = c["op"]
    if op == "rows4":
        gp.gemm_rows4(ty, c["rows"], c["outer"], c["inner"], c["group"], s["x"], c["inner"], s["q"], s["s"], s["y"],
                      c["outer"])
        return s["y"]
    if op == "pack4":
        sizes = (c["experts"], c["inner"], c["outer"], c["group"])
        gp.gemmpipe_pack4(ty, *sizes, s["w"], s["q"], s["s"])
        gp.gemmpipe_unpack4(ty, *sizes, s["q"], s["s"], s["out"])
        return s["out"]
    t, k, e, w, h = c["tokens"], c["top_k"], c["experts"], c["width"], c["hidden"]
    if op == "step":
        gp.gemmpipe_expert_step(ty, t, k, e, w, h, s["x"], w, s["ids"], s["weights"], s["w1"], s["w2"], s.get("w3"),
                                s["hidden"], s["y"], w)
    else:
        gp.gemmpipe_expert_step4(ty, t, k, e, w, h, c["group"], s["x"], w, s["ids"], s["weights"], s["q1"], s["s1"],
                                 s["q2"], s["s2"], s.get("q3"), s.get("s3"), s["hidden"], s["y"], w)
    return s["y"]


def _unpack(q, s, k, n, group):
    """The values of weights in 4 bits, in 32 bits."""
    shifts = torch.empty(8, dtype=torch.int32, device=q.device)
    for i, row in enumerate(_ROW_OF_NIBBLE):
        shifts[row] = 4 * i
    steps = (q.unsqueeze(2) >> shifts[:, None]) & 15
    steps = steps.flatten(1, 2)[:, :k, :n] - 8
    return steps.float() * s.float().repeat_interleave(group, 1)[:, :k, :n]


def _run_plain(s):
    c, ty = s["case"], _TYPES[s["case"]["type"]]
    op = c["op"]
    if op == "rows4":
        return (s["x"].float() @ _unpack(s["q"], s["s"], c["inner"], c["outer"], c["group"])[0]).to(ty)
    if op == "pack4":
        e, k, n, group = c["experts"], c["inner"], c["outer"], c["group"]
        w = torch.nn.functional.pad(s["w"].float(), (0, 0, 0, -k % group)).view(e, -1, group, n)
        scale = (w.abs().amax(2, keepdim=True) / 7).to(ty).float()
        steps = torch.where(scale > 0, (w / scale).round().clamp(-8, 7), 0.0)
        return (steps * scale).view(e, -1, n)[:, :k].to(ty)
    t, e, h = c["tokens"], c["experts"], c["hidden"]

    def matrices(name, k, n, chosen=None):
        if op == "step":
            w = s["w" + name]
            return (w if chosen is None else w[chosen]).float()
        q, sc = s["q" + name], s["s" + name]
        return _unpack(*((q, sc) if chosen is None else (q[chosen], sc[chosen])), k, n, c["group"])

    kept = (s["ids"] >= 0) & (s["ids"] < e)
    ids, weights = torch.where(kept, s["ids"], 0).long(), torch.where(kept, s["weights"], 0.0)
    x = s["x"].float()
    if ids.numel() <= e:  # each choice's own matrices
        chosen = ids.flatten()
        rows = x.repeat_interleave(c["top_k"], 0)[:, None]
        factor = weights.view(-1, 1)
    else:                 # every expert for every token, most of them with weight zero
        chosen, rows = None, x.expand(e, t, c["width"])
        factor = torch.zeros(t, e, device="cuda").scatter_add_(1, ids, weights).t()
    hidden = torch.bmm(rows, matrices("1", c["width"], h, chosen))
    hidden = hidden / (1 + torch.exp(-hidden))
    if c["gated"]:
        hidden = hidden * torch.bmm(rows, matrices("3", c["width"], h, chosen))
    out = torch.bmm(hidden, matrices("2", h, c["width"], chosen)) * factor[:, :, None]
    if chosen is None:
        return out.sum(0).to(ty)
    return out.view(t, c["top_k"], -1).sum(1).to(ty)


def _values(q, s, k, n, group):
    """One matrix in 4 bits as 64-bit values, row block by row block."""
    out = torch.empty(k, n, dtype=torch.float64, device=q.device)
    for i, row in enumerate(_ROW_OF_NIBBLE):
        at = torch.arange(row, k, 8, device=q.device)
        nibble = torch.div(q.long() & 0xffffffff, 16 ** i, rounding_mode="floor") % 16
        out[at] = (nibble[at // 8, :n] - 8).double() * s[at // group, :n].double()
    return out


def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows4":
        return s["x"].double() @ _values(s["q"][0], s["s"][0], case["inner"], case["outer"], case["group"])
    if op == "pack4":
        ty = _TYPES[case["type"]]
        out = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        for k0 in range(0, case["inner"], case["group"]):
            w = s["w"][:, k0:k0 + case["group"]].double()
            step = (w.abs().amax(1, keepdim=True) / 7).to(ty).double()
            whole = torch.where(step > 0, w / step, torch.zeros_like(w)).round().clamp(-8, 7)
            out[:, k0:k0 + case["group"]] = whole * step
        return out
    t, c, h = case["tokens"], case["width"], case["hidden"]
    y = torch.zeros(t, c, dtype=torch.float64, device="cuda")

    def matrix(name, e, k, n):
        if op == "step":
            return s["w" + name][e].double()
        return _values(s["q" + name][e], s["s" + name][e], k, n, case["group"])

    for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
        token, j = (s["ids"] == e).nonzero(as_tuple=True)
        x = s["x"][token].double()
        hidden = x @ matrix("1", e, c, h)
        hidden = hidden * torch.sigmoid(hidden)
        if case["gated"]:
            hidden = hidden * (x @ matrix("3", e, c, h))
        y.index_add_(0, token, s["weights"][token, j].double()[:, None] * (hidden @ matrix("2", e, h, c)))
    return y
