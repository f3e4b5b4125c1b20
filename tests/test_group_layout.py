"""CPU checks of group normalisation's layouts (group_layout.hpp, through
tests/layout/group_layout_driver.cpp): every column and row has its thread, every launch
holds fewer than 2^32 threads, and kernels are built for what is asked of them."""
import os
import random
import shutil
import subprocess
from collections import namedtuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("clang++")
ROCM = "/opt/rocm/include"

Layout = namedtuple("Layout", "whole vec block held per_chunk split part chunks lanes slices tile_rows tiles floats")
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    if CXX is None or not os.path.isdir(ROCM):
        pytest.skip("no host compiler or no ROCm headers")
    exe = str(tmp_path_factory.mktemp("layout") / "group_layout")
    r = subprocess.run([CXX, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
                        f"-I{ROCM}", os.path.join(ROOT, "tests", "layout", "group_layout_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(calls):
        """Layouts of (rows, width, groups, samples, ragged, longest, element bytes, backward)."""
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, map(int, c))) for c in calls), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        got = [Layout(*map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(calls)
        return got

    return run


def _calls():
    rng = random.Random(0)
    shapes = [(1, 1), (3, 1), (3, 3), (4, 1), (7, 7), (8, 8), (64, 8), (128, 16), (481, 13), (1312, 8), (1024, 1), (1025, 1), (4096, 1),
              (4097, 1), (9001, 1), (2 ** 24, 1), (2 ** 24, 2 ** 24), (2 ** 24, 64), (999983, 1)]
    calls = []
    for width, groups in shapes:
        for rows, samples in ((0, 0), (0, 3), (1, 1), (418, 1), (5000, 5000), (114688, 1), (114688, 28), (10 ** 6, 999), (MOST, 1),
                              (MOST, MOST // 7)):
            if samples * width * 6 > 2 ** 37:
                continue
            for ragged in (0, 1):
                if not ragged and (rows % samples if samples else rows):
                    continue
                for longest in (0, 1, rows // 3, rows):
                    for size in (2, 4):
                        for back in (0, 1):
                            calls.append((rows, width, groups, samples, ragged, longest, size, back))
    for _ in range(3000):
        c, groups = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 8))
        rows = int(2 ** rng.uniform(0, 22))
        calls.append((rows, c * groups, groups, int(2 ** rng.uniform(0, 12)), 1, rng.choice([0, 5, 100, rows]), rng.choice([2, 4]),
                      rng.randint(0, 1)))
    return calls


def test_layouts_hold(layout):
    calls = _calls()
    for (rows, width, groups, samples, ragged, longest, size, back), y in zip(calls, layout(calls)):
        what = (rows, width, groups, samples, ragged, longest, size, back, y)
        cg = width // groups
        assert y.vec == (4 if width >= 4 else 1), what
        assert 1 <= y.lanes and y.lanes * y.slices <= y.block, what
        if y.split == 1:
            assert y.per_chunk >= 1 and y.lanes * y.vec >= y.per_chunk * cg and y.part == cg, what
            assert (y.chunks - 1) * y.per_chunk < groups <= y.chunks * y.per_chunk, what
        else:
            assert not y.whole and y.per_chunk == 1 and y.chunks == groups * y.split and y.lanes * y.vec >= y.part, what
            assert (y.split - 1) * y.part < cg <= y.split * y.part, what
        if y.whole:
            most = 24 // size if back else 64 // size
            assert y.block in (64, 256) and y.held in (4, most), what
            told = min(longest, rows) if longest else min(rows, 8 * -(-rows // samples) if samples else 0) if ragged else \
                (rows // samples if samples else 0)
            # all of the longest, or half of it, and no more turns than 32
            assert y.slices * y.held * (1 if y.held == 4 else 2) >= told and y.slices * 32 >= told, what
        else:
            assert y.block == 256 and y.tile_rows * y.tiles >= rows and (y.tiles - 1) * y.tile_rows < max(rows, 1), what
            assert y.tiles * y.chunks * y.block < 2 ** 32, what
            assert y.floats >= (y.tiles + samples) * (2 * width if back else 2 * groups * y.split), what
        assert y.floats < 2 ** 40, what


def test_layouts_of_stated_sizes(layout):
    # a short sample alone: its groups in workgroups of their own, down to 32 bytes of a row; many
    # samples: whole rows; long ones: tiles
    short, many, long, tall, last = layout([(418, 64, 8, 1, 0, 0, 4, 0), (40000, 64, 8, 4000, 0, 0, 4, 0), (114688, 128, 16, 1, 0, 0, 2, 0),
                                      (16000, 128, 8, 4, 0, 0, 4, 0), (20060, 481, 13, 48, 1, 1000, 4, 0)])
    assert short.whole and short.per_chunk == 1 and short.chunks == 8 and short.block == 256
    assert many.whole and many.per_chunk == 8 and many.block == 64
    assert not long.whole and 256 <= long.tiles <= 1024
    assert not tall.whole and not last.whole
