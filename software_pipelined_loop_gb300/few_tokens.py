"""The few-token operators for PyTorch: a few rows times a matrix in 4 bits, and
the whole expert layer for a few tokens with weights in 16 or in 4 bits.

    rows4(x, m)                                x @ m
    expert_step(x, ids, weights, w1, w2, w3)   sum over a token's experts e of
        weight * ((silu(x @ w1[e]) * (x @ w3[e])) @ w2[e]), without w3 ungated

For generating token by token: at most 64 rows or tokens a call, no gradients
(expert_layer has them): asking for them, in forward mode too, is an error.  Everything is computed in the CUDA library; torch
supplies memory.  A matrix for many rows is brought back with unpack4.  Graphs
recorded on one stream (torch records all of a process on the same one unless it
is given another) share the library's workspace of that stream where expert_step
uses it: they must not run at the same time.

    m = pack4(w1)                  # once, when the weights are loaded
    y = expert_step(x, ids, weights, m, pack4(w2))
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from software_pipelined_loop_gb300 import gemmpipe as gp
from software_pipelined_loop_gb300.expert_layer import _CODE, _check_devices, _check_ids

GROUPS = (32, 64, 128)


class Packed4(NamedTuple):
    """Matrices in 4 bits: `experts` of inner x outer elements."""
    words: torch.Tensor   # experts x ceil(inner / 8) x outer rounded up to 4, int32
    scales: torch.Tensor  # experts x ceil(inner / group) x outer rounded up to 4
    inner: int
    outer: int
    group: int

    @property
    def experts(self) -> int:
        return self.words.shape[0]

    def expert(self, e: int) -> "Packed4":
        """One of the matrices, without a copy."""
        return self._replace(words=self.words[e:e + 1], scales=self.scales[e:e + 1])


def _no_gradients(*tensors) -> None:
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        raise RuntimeError("the few-token operators have no gradients: use expert_layer, or torch.no_grad()")
    # Forward mode goes by tangents, under no_grad too.  (Outside a dual level there
    # are none; looking at each tensor costs a microsecond.)
    if getattr(forward_ad, "_current_level", 0) >= 0 and not torch.is_inference_mode_enabled() and \
            any(forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError("the few-token operators have no gradients, forward-mode ones neither")


def _check_type(x) -> None:
    if x.dtype not in _CODE:
        raise TypeError(f"x: float16 or bfloat16 is needed, got {x.dtype}")


def _check_packed(name: str, m: Packed4, dtype) -> None:
    if m.words.dtype != torch.int32:
        raise TypeError(f"{name}: int32 words are needed, got {m.words.dtype}")
    if m.scales.dtype != dtype:
        raise TypeError(f"{name}: scales of {dtype} are needed, got {m.scales.dtype}")
    if m.group not in GROUPS:
        raise ValueError(f"{name}: a group of 32, 64 or 128 rows is needed, got {m.group}")
    n4 = (m.outer + 3) // 4 * 4
    e = m.words.shape[0]
    if m.words.shape != (e, -(-m.inner // 8), n4) or m.scales.shape != (e, -(-m.inner // m.group), n4):
        raise ValueError(f"{name}: words {(e, -(-m.inner // 8), n4)} and scales {(e, -(-m.inner // m.group), n4)} are "
                         f"needed, got {tuple(m.words.shape)} and {tuple(m.scales.shape)}")


def _rows(x: torch.Tensor) -> tuple[torch.Tensor, int]:
    """(x, its pitch), a copy where the rows are not each in one piece."""
    if x.shape[0] > 1 and x.shape[1] > 0 and x.stride(1) == 1 and x.shape[1] <= x.stride(0) < 1 << 31:
        return x, x.stride(0)
    return x.contiguous(), x.shape[1]


def pack4(w: torch.Tensor, group: int = 128) -> Packed4:
    """w: experts x inner x outer, or one matrix inner x outer; 16-bit floating point."""
    _check_type(w)
    if w.dim() not in (2, 3):
        raise ValueError(f"w: one matrix, or one per expert, is needed, got {tuple(w.shape)}")
    if group not in GROUPS:
        raise ValueError(f"group: 32, 64 or 128 is needed, got {group}")
    _no_gradients(w)
    _check_devices(w)
    w = w.contiguous()
    e, (k, n) = (w.shape[0] if w.dim() == 3 else 1), w.shape[-2:]
    n4 = (n + 3) // 4 * 4
    words = torch.empty(e, -(-k // 8), n4, dtype=torch.int32, device=w.device)
    scales = torch.empty(e, -(-k // group), n4, dtype=w.dtype, device=w.device)
    gp.gemmpipe_pack4(_CODE[w.dtype], e, k, n, group, w, words, scales)
    return Packed4(words, scales, k, n, group)


def unpack4(m: Packed4) -> torch.Tensor:
    """The matrices (experts x inner x outer), each value rounded to the scales' type."""
    _check_type(m.scales)
    _check_packed("m", m, m.scales.dtype)
    _no_gradients(m.scales)
    _check_devices(m.words, m.scales)
    w = torch.empty(m.experts, m.inner, m.outer, dtype=m.scales.dtype, device=m.words.device)
    gp.gemmpipe_unpack4(_CODE[w.dtype], m.experts, m.inner, m.outer, m.group, m.words.contiguous(),
                        m.scales.contiguous(), w)
    return w


def rows4(x: torch.Tensor, m: Packed4) -> torch.Tensor:
    """x (at most 64 rows) times one matrix in 4 bits."""
    _check_type(x)
    _check_packed("m", m, x.dtype)
    if x.dim() != 2 or x.shape[0] > gp.FEW_ROWS or x.shape[1] != m.inner or m.experts != 1:
        raise ValueError(f"at most {gp.FEW_ROWS} rows of {m.inner} values and one matrix are needed, "
                         f"got {tuple(x.shape)} and {m.experts}")
    _no_gradients(x, m.scales)
    _check_devices(x, m.words, m.scales)
    x, ldx = _rows(x)
    y = torch.empty(x.shape[0], m.outer, dtype=x.dtype, device=x.device)
    gp.gemm_rows4(_CODE[x.dtype], x.shape[0], m.outer, m.inner, m.group, x, ldx, m.words.contiguous(),
                  m.scales.contiguous(), y, m.outer)
    return y


def expert_step(x, ids, weights, w1, w2, w3=None) -> torch.Tensor:
    """x: tokens x c, at most 64; ids: tokens x top_k int32 (outside [0, experts): dropped); weights: tokens x top_k
    fp32; w1, w3: experts x c x h and w2: experts x h x c, tensors of x's type or all Packed4 of one group.  Strided
    tensors are copied to dense ones first; another type, shape or device is refused."""
    _check_type(x)
    _check_ids(ids)
    if weights.dtype != torch.float32:
        raise TypeError(f"weights: float32 is needed, got {weights.dtype}")
    matrices = {"w1": w1, "w2": w2} | ({} if w3 is None else {"w3": w3})
    four = isinstance(w1, Packed4)
    shapes = {}
    for name, w in matrices.items():
        if isinstance(w, Packed4) != four:
            raise TypeError("matrices all in 16 or all in 4 bits are needed")
        if four:
            _check_packed(name, w, x.dtype)
            if w.group != w1.group:
                raise ValueError(f"matrices of one group are needed, got {w1.group} and {w.group}")
            shapes[name] = (w.experts, w.inner, w.outer)
        else:
            if w.dtype != x.dtype:
                raise TypeError(f"{name}: the type of x, {x.dtype}, is needed, got {w.dtype}")
            if w.dim() != 3:
                raise ValueError(f"{name}: one matrix per expert is needed, got {tuple(w.shape)}")
            shapes[name] = tuple(w.shape)
    (t, k), (e, c, h) = ids.shape, shapes["w1"]
    if x.shape != (t, c) or t > gp.FEW_ROWS or weights.shape != (t, k) or shapes["w2"] != (e, h, c) or \
            shapes.get("w3", (e, c, h)) != (e, c, h):
        raise ValueError(f"at most {gp.FEW_ROWS} tokens, x {(t, c)}, weights {(t, k)}, w2 {(e, h, c)} and w3 "
                         f"{(e, c, h)} are needed, got {tuple(x.shape)}, {tuple(weights.shape)} and {shapes}")
    parts = [p for w in matrices.values() for p in ((w.words, w.scales) if four else (w,))]
    _no_gradients(x, weights, *parts)
    _check_devices(x, ids, weights, *parts)
    x, ldx = _rows(x)
    ids, weights = ids.contiguous(), weights.contiguous()
    parts = [p.contiguous() for p in parts] + [None] * (0 if w3 is not None else 2 if four else 1)
    hidden = torch.empty(t * k, (h + 7) // 8 * 8, dtype=x.dtype, device=x.device)
    y = torch.empty(t, c, dtype=x.dtype, device=x.device)
    if four:
        gp.gemmpipe_expert_step4(_CODE[x.dtype], t, k, e, c, h, w1.group, x, ldx, ids, weights, *parts, hidden, y, c)
    else:
        gp.gemmpipe_expert_step(_CODE[x.dtype], t, k, e, c, h, x, ldx, ids, weights, *parts, hidden, y, c)
    return y
