"""Weight gradients whose long sums are split into parts, in every order of
work: experts sorted by length and too many to sort, fewer and more tiles than
the machine has CTA pairs, from 16-bit rows and from rows kept in 8 bits."""
from __future__ import annotations

import pytest
import torch

from software_pipelined_loop_gb300 import gemmpipe as gp

pytestmark = pytest.mark.gpu


def tiles(K, N):  # output tiles of a matrix
    return -(-K // 256) * -(-N // 256)


def plan(counts, head, unused, K, N, pairs):
    """(rows of a part at most, experts that are split, tiles in all), by the documented rule."""
    R = head + sum(counts) + unused
    m = tiles(K, N)
    most = max(2048, -(-(R * m // pairs + 1) // 64) * 64) if m < pairs else 0
    if most and (most + most // 2 >= R or (2 * R // most + 1) * m > 512):
        most = 0
    split = [c for c in counts if most and c - most > most // 2]
    return most, len(split), len(counts) * m + sum(-(-c // most) - 1 for c in split) * m


CASES = [
    # rows per expert, inner, outer, split experts, more tiles than pairs
    ([40] * 300 + [7000, 0, 3500], 64, 128, 2, True),            # too many experts to sort
    ([7000, 40, 0, 3500] + [300] * 30, 768, 880, 1, True),       # sorted, pairs of several tiles
    ([1, 5000] + [17] * 40 + [0] * 3 + [4111], 300, 320, 2, True),
    ([31] * 255 + [9001], 65, 66, 1, True),                      # the most experts that are sorted
    ([31] * 256 + [9001], 65, 66, 1, True),                      # one more
    ([9000, 3073, 15, 8191], 130, 70, 3, False),                 # 3073: just long enough
    ([3400] * 12, 256, 512, 12, False),                          # every expert split
]


@pytest.mark.parametrize("kept8", [False, True])
@pytest.mark.parametrize("ty", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{c[1]}x{c[2]}")
def test_sums_in_parts(case, ty, kept8):
    counts, K, N, split, many = case
    code = gp.F16 if ty == torch.float16 else gp.BF16
    head, unused, E = 5, 37, len(counts)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    most, have, all_tiles = plan(counts, head, unused, K, N, pairs)
    # As the case says.  (A few pairs fewer may be resident at once: neither changes for that.)
    assert have == split and plan(counts, head, unused, K, N, pairs - 6)[1] == split
    assert (all_tiles > pairs) if many else (all_tiles <= pairs - 6), all_tiles
    # Whole numbers: a sum is exact in fp32 in any order, its rounding the only one.
    g = torch.Generator(device="cuda").manual_seed(len(counts) + K)
    R = head + sum(counts) + unused
    X = torch.randint(-2, 3, (R, K), generator=g, device="cuda").to(ty)
    dY = torch.randint(-1, 2, (R, N), generator=g, device="cuda").to(ty)
    X[:head] = X[R - unused:] = dY[:head] = dY[R - unused:] = float("nan")
    bounds = [head]
    for c in counts:
        bounds.append(bounds[-1] + c)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    Q, S = torch.empty(R, K, dtype=torch.int8, device="cuda"), torch.empty(R, -(-K // 32), dtype=torch.uint8, device="cuda")
    if kept8:
        gp.gemmpipe_keep8(code, R, K, X, K, Q, S)  # exact: a group's largest value is 0, 1 or 2
    first = None
    for _ in range(3):
        dW = torch.full((E, K, N), 3.0, dtype=ty, device="cuda")
        if kept8:
            gp.gemm_grouped_dw8(code, R, N, K, E, Q, S, dY, N, off, dW)
        else:
            gp.gemm_grouped_dw(code, R, N, K, E, X, K, dY, N, off, dW)
        assert gp.gemmpipe_get_device_status() == gp.OK
        first = dW if first is None else first
        assert torch.equal(dW, first)
    for e in range(E):
        x, d = X[bounds[e]:bounds[e + 1]].float(), dY[bounds[e]:bounds[e + 1]].float()
        assert torch.equal(first[e], (x.double().t() @ d.double()).to(ty)), e
