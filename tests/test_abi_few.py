"""Refusals of the few-token entry points on the host, before any device call."""
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


# Valid calls, and which arguments to spoil: {argument: values that are refused}.
CALLS = {
    # type, M, N, K, group, X, ldx, Q, S, Y, ldy, stream
    "gemm_rows4": ([0, 4, 9, 16, 32, FAKE, 16, FAKE, FAKE, FAKE, 9, None],
                   {0: [-1, 2], 1: [-1, 65, 1 << 31], 2: [-1, 10, 1 << 31], 3: [-1, 17, 1 << 31],
                    4: [0, 16, 48, 256, -32], 5: [None, FAKE + 1], 6: [15, -16, 1 << 31], 7: [None, FAKE + 8],
                    8: [None, FAKE + 4], 9: [None, FAKE + 1], 10: [8, 1 << 31]}),
    # type, T, top_k, E, C, H, X, ldx, experts, weights, W1, W2, W3, hidden, Y, ldy, stream
    "gemmpipe_expert_step": ([1, 4, 2, 8, 16, 24, FAKE, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 16, None],
                             {0: [-1, 2], 1: [-1, 65], 2: [0, 65], 3: [0, 1025], 4: [-1, 17, 1 << 31],
                              5: [-1, 1 << 31], 6: [None, FAKE + 1], 7: [15, 1 << 31], 8: [None, FAKE + 2],
                              9: [None, FAKE + 2], 10: [None, FAKE + 1], 11: [None, FAKE + 1], 12: [FAKE + 1],
                              13: [None, FAKE + 8], 14: [None, FAKE + 1], 15: [15, 1 << 31]}),
    # type, T, top_k, E, C, H, group, X, ldx, experts, weights, Q1, S1, Q2, S2, Q3, S3, hidden, Y, ldy, stream
    "gemmpipe_expert_step4": ([0, 4, 2, 8, 16, 24, 64, FAKE, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                               FAKE, 16, None],
                              {0: [-1, 2], 1: [-1, 65], 2: [0, 65], 3: [0, 1025], 4: [-1, 17], 5: [-1, 1 << 31],
                               6: [0, 16, 96, 256], 7: [None, FAKE + 1], 8: [15], 9: [None, FAKE + 2],
                               10: [None, FAKE + 2], 11: [None, FAKE + 8], 12: [None, FAKE + 4], 13: [None, FAKE + 8],
                               14: [None, FAKE + 4], 15: [None, FAKE + 8], 16: [None, FAKE + 4],
                               17: [None, FAKE + 8], 18: [None, FAKE + 1], 19: [15]}),
    # type, E, K, N, group, W, Q, S, stream
    "gemmpipe_pack4": ([0, 2, 40, 9, 32, FAKE, FAKE, FAKE, None],
                       {0: [-1, 2], 1: [0, 1025], 2: [-1, 1 << 31], 3: [-1, 1 << 31], 4: [0, 31, 256],
                        5: [None, FAKE + 1], 6: [None, FAKE + 8], 7: [None, FAKE + 4]}),
    # type, E, K, N, group, Q, S, W, stream
    "gemmpipe_unpack4": ([0, 2, 40, 9, 32, FAKE, FAKE, FAKE, None],
                         {0: [-1, 2], 1: [0, 1025], 2: [-1, 1 << 31], 3: [-1, 1 << 31], 4: [0, 31, 256],
                          5: [None, FAKE + 8], 6: [None, FAKE + 4], 7: [None, FAKE + 1]}),
}


@pytest.mark.parametrize("name", CALLS)
def test_bad_arguments_are_refused(lib, name):
    args, spoilt = CALLS[name]
    for place, values in spoilt.items():
        for v in values:
            call = list(args)
            call[place] = v
            assert getattr(lib, name)(*call) == BAD, (place, v)


def test_sizes_past_the_address_range(lib):
    most = BIG - 1023
    assert lib.gemm_rows4(0, 1, most, most, 32, FAKE, BIG, FAKE, FAKE, FAKE, BIG, None) == BAD
    assert lib.gemm_rows4(0, 1, most + 1, 8, 32, FAKE, 8, FAKE, FAKE, FAKE, BIG, None) == BAD
    assert lib.gemmpipe_pack4(0, 1024, 1 << 23, 1 << 23, 32, FAKE, FAKE, FAKE, None) == BAD
    assert lib.gemmpipe_unpack4(0, 1, most + 1, 8, 32, FAKE, FAKE, FAKE, None) == BAD
    assert lib.gemmpipe_expert_step(0, 1, 1, 1024, 1 << 24, 1 << 23, FAKE, 1 << 24, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                                    FAKE, 1 << 24, None) == BAD


def test_empty_outputs_launch_nothing(lib):
    ok, n = gemmpipe.OK, lib.gemmpipe_launch_count()
    assert lib.gemm_rows4(0, 0, 8, 8, 32, None, 8, None, None, None, 8, None) == ok
    assert lib.gemm_rows4(0, 8, 0, 8, 32, None, 8, None, None, None, 0, None) == ok
    assert lib.gemmpipe_expert_step(0, 0, 2, 8, 16, 24, None, 16, None, None, None, None, None, None, None, 16,
                                    None) == ok
    assert lib.gemmpipe_expert_step(0, 4, 2, 8, 0, 24, None, 0, None, None, None, None, None, None, None, 0,
                                    None) == ok
    assert lib.gemmpipe_expert_step4(0, 0, 2, 8, 16, 24, 32, None, 16, None, None, None, None, None, None, None, None,
                                     None, None, 16, None) == ok
    assert lib.gemmpipe_pack4(0, 2, 0, 8, 32, None, None, None, None) == ok
    assert lib.gemmpipe_unpack4(0, 2, 8, 0, 32, None, None, None, None) == ok
    assert lib.gemmpipe_launch_count() == n


@pytest.mark.parametrize("name", CALLS)
def test_no_device_is_an_error(lib, name):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert getattr(lib, name)(*CALLS[name][0]) == gemmpipe.ERR_UNSUPPORTED_DEVICE
