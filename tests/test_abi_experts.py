"""Refusals of the expert-layer entry points on the host, before any device call."""
from __future__ import annotations

import pytest

from software_pipelined_loop_gb300 import build, gemmpipe

FAKE = 1 << 20  # never dereferenced
BAD = gemmpipe.ERR_INVALID_VALUE
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gemmpipe.load()


def changed(args, **by_place):
    out = list(args)
    for place, value in by_place.items():
        out[int(place[1:])] = value
    return out


# Valid calls, and which arguments to spoil: {argument: values that are refused}.
CALLS = {
    # T, top_k, E, experts, offsets, slots, rows, stream
    "gemmpipe_route": ([4, 2, 8, FAKE, FAKE, FAKE, FAKE, None],
                       {0: [-1, 1 << 31, BIG], 1: [0, -1, 65], 2: [0, -1, 1025], 3: [None, FAKE + 2],
                        4: [None, FAKE + 1], 5: [None, FAKE + 2], 6: [None, FAKE + 2]}),
    # type, T, top_k, C, X, ldx, rows, weights, Xs, ldxs, stream
    "gemmpipe_dispatch": ([0, 4, 2, 8, FAKE, 8, FAKE, FAKE, FAKE, 8, None],
                          {0: [-1, 2], 1: [-1, 1 << 31], 2: [0, 65], 3: [-1, 9, 1 << 31], 4: [None, FAKE + 1],
                           5: [7, -8, 1 << 31], 6: [None, FAKE + 2], 7: [FAKE + 2], 8: [None, FAKE + 1], 9: [7]}),
    "gemmpipe_combine": ([0, 4, 2, 8, FAKE, 8, FAKE, FAKE, FAKE, 8, None],
                         {0: [-1, 2], 1: [-1, 1 << 31], 2: [0, 65], 3: [-1, 9, 1 << 31], 4: [None, FAKE + 1],
                          5: [7, -8, 1 << 31], 6: [None, FAKE + 2], 7: [FAKE + 2], 8: [None, FAKE + 1], 9: [7]}),
    # type, T, top_k, C, dY, lddy, Ys, ldys, rows, weights, dYs, lddys, dweights, stream
    "gemmpipe_combine_grad": ([1, 4, 2, 8, FAKE, 8, FAKE, 8, FAKE, FAKE, FAKE, 8, FAKE, None],
                              {0: [2], 1: [-1], 2: [0], 3: [-1, 9], 4: [None, FAKE + 1], 5: [7], 6: [None, FAKE + 1],
                               7: [7], 8: [None, FAKE + 2], 9: [FAKE + 2], 10: [None, FAKE + 1], 11: [7],
                               12: [None, FAKE + 2]}),
    # type, R, N, K, E, X, ldx, offsets, W, Y, ldy, stream
    "gemm_grouped": ([0, 4, 8, 16, 2, FAKE, 16, FAKE, FAKE, FAKE, 8, None],
                     {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9, 1 << 31], 3: [-1, 17], 4: [0, 1025],
                      5: [None, FAKE + 1], 6: [15], 7: [None, FAKE + 2], 8: [None, FAKE + 1], 9: [None, FAKE + 1],
                      10: [7, 1 << 31]}),
    "gemm_grouped_dx": ([0, 4, 8, 16, 2, FAKE, 8, FAKE, FAKE, FAKE, 16, None],
                        {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9], 3: [-1, 17], 4: [0, 1025], 5: [None, FAKE + 1],
                         6: [7], 7: [None, FAKE + 2], 8: [None, FAKE + 1], 9: [None, FAKE + 1], 10: [15]}),
    # type, R, N, K, E, X, ldx, dY, lddy, offsets, dW, stream
    "gemm_grouped_dw": ([0, 4, 8, 16, 2, FAKE, 16, FAKE, 8, FAKE, FAKE, None],
                        {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9], 3: [-1, 17], 4: [0, 1025], 5: [None, FAKE + 1],
                         6: [15], 7: [None, FAKE + 1], 8: [7], 9: [None, FAKE + 2], 10: [None, FAKE + 1]}),
    # type, R, N, K, E, Q, S, dY, lddy, offsets, dW, stream
    "gemm_grouped_dw8": ([0, 4, 8, 16, 2, FAKE, FAKE, FAKE, 8, FAKE, FAKE, None],
                         {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9], 4: [0, 1025], 5: [None], 6: [None],
                          7: [None, FAKE + 1], 8: [7], 9: [None, FAKE + 2], 10: [None, FAKE + 1]}),
    # type, R, C, X, ldx, Q, S, stream
    "gemmpipe_keep8": ([0, 4, 8, FAKE, 8, FAKE, FAKE, None],
                       {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9], 3: [None, FAKE + 1], 4: [7], 5: [None], 6: [None]}),
    # type, R, C, Q, S, X, ldx, stream
    "gemmpipe_restore8": ([0, 4, 8, FAKE, FAKE, FAKE, 8, None],
                          {0: [-1, 2], 1: [-1, 1 << 31], 2: [-1, 9], 3: [None], 4: [None], 5: [None, FAKE + 1],
                           6: [7]}),
}


@pytest.mark.parametrize("name", CALLS)
def test_bad_arguments_are_refused(lib, name):
    args, spoilt = CALLS[name]
    for place, values in spoilt.items():
        for v in values:
            assert getattr(lib, name)(*changed(args, **{f"a{place}": v})) == BAD, (place, v)


def test_sizes_past_the_address_range(lib):
    assert lib.gemm_grouped(0, BIG, BIG, 8, 1, FAKE, 8, FAKE, FAKE, FAKE, BIG, None) == BAD      # 2^62 elements of Y
    assert lib.gemm_grouped(0, 8, BIG, BIG, 1, FAKE, BIG, FAKE, FAKE, FAKE, BIG, None) == BAD    # ... of W
    assert lib.gemm_grouped_dw(0, 8, 1 << 23, 1 << 23, 1024, FAKE, 1 << 23, FAKE, 1 << 23, FAKE, FAKE, None) == BAD
    assert lib.gemm_grouped(0, BIG - 1022, 8, 8, 1, FAKE, 8, FAKE, FAKE, FAKE, 8, None) == BAD   # a tile past 2^31
    assert lib.gemmpipe_dispatch(0, 1, 1, (1 << 30) + 1, FAKE, 1 << 31, FAKE, FAKE, FAKE, 1 << 31, None) == BAD
    assert lib.gemmpipe_keep8(0, BIG, BIG, FAKE, BIG, FAKE, FAKE, None) == BAD


def test_empty_outputs_launch_nothing(lib):
    ok = gemmpipe.OK
    n = lib.gemmpipe_launch_count()
    assert lib.gemmpipe_dispatch(0, 0, 2, 8, None, 8, None, None, None, 8, None) == ok
    assert lib.gemmpipe_combine(0, 4, 2, 0, None, 0, None, None, None, 0, None) == ok
    assert lib.gemmpipe_combine_grad(0, 0, 2, 8, None, 8, None, 8, None, None, None, 8, None, None) == ok
    assert lib.gemm_grouped(0, 0, 8, 8, 2, None, 8, None, None, None, 8, None) == ok
    assert lib.gemm_grouped(0, 8, 0, 8, 2, None, 8, None, None, None, 0, None) == ok
    assert lib.gemm_grouped_dx(0, 8, 8, 0, 2, None, 8, None, None, None, 0, None) == ok
    assert lib.gemm_grouped_dw(0, 8, 0, 8, 2, None, 8, None, 0, None, None, None) == ok
    assert lib.gemmpipe_keep8(0, 0, 8, None, 8, None, None, None) == ok
    assert lib.gemmpipe_restore8(0, 8, 0, None, None, None, 0, None) == ok
    assert lib.gemmpipe_launch_count() == n


@pytest.mark.parametrize("name", CALLS)
def test_no_device_is_an_error(lib, name):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert getattr(lib, name)(*CALLS[name][0]) == gemmpipe.ERR_UNSUPPORTED_DEVICE
