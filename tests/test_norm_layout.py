"""CPU checks of the normalisations' launches (norm_layout.hpp, through
tests/layout/norm_layout_driver.cpp): every grid holds fewer than 2^32 threads, for any
rows and terms that the entry points take."""
import os
import shutil
import subprocess

import pytest

from oracle import train_oracle as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("clang++")
ROCM = "/opt/rocm/include"

MOST_ROWS = 2 ** 31 - 1
SPECS = ["1x0e", "3x0e", "8x0e", "16x0e", "1312x0e", "8192x0e", "16384x0e", "+".join(["1x0e"] * 8), "+".join(["1x0o"] * 64),
         "+".join(["3x0e+1x1o"] * 4), "+".join(["3x0e+1x1o"] * 32), "128x0e+64x1o+32x2e+32x3o", "16x0e+16384x0e+9000x1o",
         f"{2 ** 29 - 16384}x0o+16384x0e", f"{2 ** 29 - 1}x0e+1x0e", f"{2 ** 29 // 13}x6e"]


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    if CXX is None or not os.path.isdir(ROCM):
        pytest.skip("no host compiler or no ROCm headers")
    exe = str(tmp_path_factory.mktemp("layout") / "norm_layout")
    r = subprocess.run([CXX, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}",
                        os.path.join(ROOT, "tests", "layout", "norm_layout_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(calls):
        """(threads, workgroups, threads and workgroups of the sums, elements of a lane) of (terms,
        rows, bytes, backward)."""
        text = "\n".join(" ".join(map(str, (rows, size, int(back), len(t), *(
            v for _, m, d, _, b in t for v in (m * d, d, int(b is not None)))))) for t, rows, size, back in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert r.returncode == 0
        got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(calls)
        return got

    return run


def test_grids_hold_fewer_than_2_32_threads(layout):
    rows = [0, 1, 7, 65, 129, 1000, 10 ** 6, 4 * 10 ** 8, 10 ** 9, MOST_ROWS]
    shapes = [T.norm_terms(s) for s in SPECS] + [T.row_terms(2 ** 30 - 1)]
    calls = [(t, n, size, back) for t in shapes for n in rows for size in (2, 4) for back in (False, True)]
    for call, (threads, blocks, sum_threads, sum_blocks, _) in zip(calls, layout(calls)):
        assert threads * blocks < 2 ** 32, (call[1:], threads, blocks)
        assert sum_threads * sum_blocks < 2 ** 32, (call[1:], sum_threads, sum_blocks)
        assert blocks > 0 or all(m * d > 16384 for _, m, d, _, _ in call[0])


def test_layouts_of_stated_sizes(layout):
    # workgroups by cost and by rows, as the header states them: 28 / element bytes turns past the
    # cache, 2048 workgroups of 256 below it, one workgroup where the rows fit four turns
    row = T.row_terms
    got = layout([(row(1312), 114688, 4, False), (row(64), 418, 4, False), (row(64), 300000, 4, False), (row(128), 9, 4, True)])
    assert got[0][:2] == (256, 114688 * 4 // 28)
    assert got[1][:2] == (256, -(-418 // 16))
    assert got[2][:2] == (256, 2048)
    assert got[3][:2] == (256, 1)


def test_workgroups_are_those_that_kernels_are_built_for(layout):
    # more than 8 elements a lane: the forward in 512 (fp32) or 1024 threads, the backward in 256
    # (fp32), 512 (16 bits) or 1024; every lane's elements fit
    shapes = [T.row_terms(w) for w in [*range(1, 1600), *range(1600, 17000, 37), 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385]]
    shapes += [T.norm_terms(f"{w}x0e+{v}x1o+40000x0o") for w in (1, 100, 700, 1100, 5000, 9000) for v in (1, 60, 333, 1400, 2900, 5000)]
    shapes += [t[:-1] for t in shapes[-36:]]
    calls = [(t, n, size, back) for t in shapes for n in (1, 3000) for size in (2, 4) for back in (False, True)]
    for (terms, _, size, back), (threads, _, _, _, most) in zip(calls, layout(calls)):
        assert threads in (128, 256, 512, 1024) and most <= 16
        if most > 8:
            assert threads == 1024 or threads == {(4, False): 512, (4, True): 256, (2, True): 512}.get((size, back)), (terms, size, back, threads)
        longest = max((m * d for _, m, d, _, _ in terms if m * d <= 16 * threads), default=0)
        assert longest <= threads * max(most, 8)
