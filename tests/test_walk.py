"""Host check of what the persistent workgroups of the MXFP4 and training
kernels take.

`csrc/rmoe_sched.h` (plain C++, the code that the kernels run) is built with
g++ into `walk_check.cpp`: the item walk must cover every (block with rows,
slice) exactly once and leave out blocks that the table maps elsewhere; the
weight-gradient walk must take every tile exactly once, also where some of a
locality group's workgroups start ahead of the others.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest

import workloads

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("walk") / "walk_check")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-o", exe, os.path.join(HERE, "walk_check.cpp")],
                   check=True)
    return exe


def _run(exe, *words):
    out = subprocess.run([exe], input=" ".join(map(str, words)), capture_output=True, text=True, check=False)
    assert out.returncode == 0 and out.stdout.startswith("ok"), (words[:8], out.stdout, out.returncode)
    return [int(v) for v in out.stdout.split()[1:]]


def _items(exe, gs, NT, grid=256, moved=()):
    return _run(exe, "items", len(gs), NT, grid, *gs, len(moved), *moved)


@pytest.mark.parametrize("name", ["tiny", "decode", "prefill", "fine", "large"])
def test_items_of_the_workloads(checker, name):
    cfg = workloads.CONFIGS[name]
    gs = np.bincount(workloads.draw_routing(cfg).ravel(), minlength=cfg.experts)
    entries = int((-(-gs // 256)).sum())
    for NT in (cfg.intermediate // 128, (cfg.intermediate + 255) // 256, (cfg.hidden + 255) // 256):
        total, most = _items(checker, gs, NT)
        assert total == entries * NT
        assert most <= -(-(-(-total // 8)) // 32)      # no workgroup has an item more than an even deal gives


@pytest.mark.parametrize("gs", [[0], [0, 0, 0, 5], [128, 256, 384], [127, 129, 255, 257], [1] * 33, [4096],
                                [641, 0, 3], [0, 700, 0, 0, 1, 128]])
def test_items_of_edge_groups(checker, gs):
    for NT in (1, 3, 8, 9, 112):
        for grid in (8, 16, 64, 256, 304):
            _items(checker, gs, NT, grid)


def test_items_of_random_groups_and_moved_blocks(checker):
    rng = np.random.default_rng(3)
    for _ in range(150):
        gs = rng.integers(0, 900, int(rng.integers(1, 40)))
        gs[rng.random(gs.size) < 0.3] = 0
        blocks = int((gs // 128 + 1).sum())
        moved = rng.choice(blocks, int(rng.integers(0, min(blocks, 6) + 1)), replace=False)
        _items(checker, gs, int(rng.integers(1, 40)), 8 * int(rng.integers(1, 40)), moved)


def _tiles(exe, E, nh, ni, busy=0, lead=0, grid=256):
    total, most = _run(exe, "tiles", E, nh, ni, grid, busy, lead)
    assert total == 3 * E * nh * ni
    return most


@pytest.mark.parametrize("E,nh,ni", [(1, 1, 1), (4, 1, 1), (64, 8, 6), (8, 16, 56), (3, 9, 7), (5, 17, 3), (2, 1, 30),
                                     (1, 4096, 1), (128, 28, 8)])
def test_weight_gradient_tiles(checker, E, nh, ni):
    most = _tiles(checker, E, nh, ni)
    assert most <= -(-3 * E * nh * ni // 256) + 1
    for busy, lead in ((1, 1), (31, 1), (16, 3), (5, 40), (31, 5461), (1, 5461)):
        _tiles(checker, E, nh, ni, busy, lead)


def test_weight_gradient_tiles_at_random(checker):
    """Heads longer than the list, single workgroups ahead, other grids."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        nl = int(rng.integers(1, 40))
        E, nh, ni = (int(v) for v in rng.integers(1, 12, 3))
        _tiles(checker, E, nh, ni, int(rng.integers(0, nl)), int(rng.integers(0, 30)), 8 * nl)
