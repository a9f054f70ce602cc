"""TMA multicast loads (quads of CTAs sharing A) are for runs on one GPU alone: bench.py takes them out of the plans of
runs on several ranks (on CPU)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


@pytest.mark.parametrize("world", [2, 4, 8])
def test_ranks_take_pairs_where_one_gpu_takes_quads(world):
    assert bench.rank_override(world, 2) == (-1, 0, 0, 1, -1)
    assert bench.rank_override(world, 2, (0, 256, 5, -1, 1)) == (0, 256, 5, 1, 1)


@pytest.mark.parametrize("cta_pair", [0, 1])
def test_other_plans_stay(cta_pair):
    for world in (1, 2, 8):
        assert bench.rank_override(world, cta_pair) == bench.AUTOMATIC
    assert bench.rank_override(1, 2) == bench.AUTOMATIC
    assert bench.rank_override(1, 2, (0, 256, 0, 2, -1)) == (0, 256, 0, 2, -1)


def test_forced_plans():
    assert bench.parse_force("-1,512,0", 1) == (-1, 512, 0, -1, -1)
    assert bench.parse_force("-1,0,0,2", 1) == (-1, 0, 0, 2, -1)
    assert bench.parse_force("-1,0,0,1,0", 2) == (-1, 0, 0, 1, 0)
    with pytest.raises(ValueError, match="one GPU"):
        bench.parse_force("-1,0,0,2", 2)


@pytest.mark.parametrize("args", [["--force=-1,0,0,2"], ["--ablation"]])
def test_ranks_refuse_what_would_take_quads(args):
    env = dict(os.environ, RANK="0", WORLD_SIZE="2", LOCAL_RANK="0")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *args], capture_output=True, text=True, env=env,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 2 and "one GPU" in r.stderr and r.stdout == ""
