"""The kernels' walk over experts' segments, csrc/mxq_mm_segments.h compiled for the CPU with
one thread a lane (tests/host/mm_segments.cpp), against a walk in Python's integers: exact
for well-formed offsets, and inside the experts' own rows and the first `most` tiles for
malformed ones, also where the true number of tiles passes 32 bits."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CAP = 2 ** 30 - 1


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("segments") / "segments")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-I",
                    os.path.join(ROOT, "mxfp4_microscaling_quantization_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "mm_segments.cpp"), "-o", exe, "-pthread"], check=True)

    def run(rows, step, offsets, most, indexes):
        text = " ".join(map(str, [rows, step, len(offsets) - 1, most, len(indexes), *offsets, *indexes]))
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=100, check=True).stdout
        lines = [tuple(map(int, x.split())) for x in out.splitlines()]
        return lines[0][0], lines[1:1 + len(indexes)], lines[1 + len(indexes):]

    return run


def check(walk, rows, step, offsets, valid):
    clamped = [min(max(v, 0), rows) for v in offsets]
    counts = [max(b - a, 0) for a, b in zip(clamped, clamped[1:])]
    tiles = [-(-c // step) for c in counts]
    groups, total = len(counts), sum(tiles)
    most = (rows + (step - 1) * groups) // step
    if valid:
        assert total <= most and total <= rows // step + min(rows, groups)
    rng = random.Random(rows)
    indexes = sorted({i for i in [0, 1, total - 1, most - 1, *(rng.randrange(max(most, 1)) for _ in range(12))]
                      if 0 <= i < CAP})
    got, found, segments = walk(rows, step, offsets, most, indexes)
    assert got == min(total, CAP)
    for i, (ok, expert, begin, count, tile) in zip(indexes, found):
        assert ok == (i < total)
        if ok:
            before = 0
            for e, t in enumerate(tiles):
                if before + t > i:
                    break
                before += t
            assert (expert, begin, count, tile) == (e, clamped[e], counts[e], i - before)
            assert 0 <= tile * step < counts[e]
    for g, first, n in segments:
        before = sum(tiles[:g])
        assert first == min(before, CAP)
        assert n >= 0 and (n == 0 or first + n <= most)
        assert n == max(min(tiles[g], most - before), 0)


@pytest.mark.parametrize("step", [16, 64, 128])
@pytest.mark.parametrize("groups", [1, 3, 64, 65, 200])
def test_well_formed(walk, groups, step):
    rng = random.Random(groups)
    for rows in (1, 700, 2 ** 31 - 1):
        check(walk, rows, step, [0, *sorted(rng.randint(0, rows) for _ in range(groups - 1)), rows], True)


@pytest.mark.parametrize("rows,step,groups", [(2 ** 28, 128, 4096), (2 ** 31 - 1, 16, 4096), (2 ** 31 - 1, 16, 70),
                                              (2 ** 24, 64, 4096), (1000, 16, 130)])
def test_segments_that_overlap_many_times(walk, rows, step, groups):
    """Alternating 0 and rows: every second segment is all rows (from 2^28 rows of 4096 groups
    on, their tiles of 128 pass 2^31)."""
    check(walk, rows, step, [rows * (i % 2) for i in range(groups + 1)], False)
    check(walk, rows, step, [(-5, rows + 7, -2 ** 62, 2 ** 62)[i % 4] for i in range(groups + 1)], False)


def test_random_offsets(walk):
    rng = random.Random(0)
    for rows in (50, 2 ** 31 - 1):
        check(walk, rows, 16, [rng.randint(-rows, 2 * rows) for _ in range(301)], False)
