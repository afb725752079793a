"""The sizes that the GPU tests of linear attention run take every kernel of the walk, by the front end's own plan on 256
compute units: a retuned planner cannot leave one untested."""

import os
import shutil
import subprocess

import pytest

from tests.mixer_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES = {"bf16": [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64)],
         "f32": [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)]}


@pytest.fixture(scope="module")
def planned(tmp_path_factory):
    """(tile, segments, tokens of one, whether rows are loaded directly) of the forward and of all gradients."""
    include = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(include, "hip", "hip_runtime.h")):
        pytest.skip("no host compiler or no HIP headers")
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    # the launches' symbols are in other sources and are not reached
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I", include,
                    os.path.join(ROOT, "tests", "mixer_plans.cpp"), "-o", exe, "-Wl,--unresolved-symbols=ignore-all"], check=True)

    def call(cases):
        lines = "\n".join(" ".join(map(str, (*c, int(dtype == "f32"), 256))) for c, dtype in cases)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.splitlines()
        rows = [list(map(int, line.split())) for line in out]
        assert len(rows) == len(cases)
        return [[((dp, nv), segments, each, bool(direct)) for dp, nv, segments, each, direct in (r[:5], r[5:])] for r in rows]
    return call


def test_cases_take_every_kernel(planned):
    cases = [(c, dtype) for c in CASES for dtype in TILES]
    outputs, sums = set(), set()
    for (c, dtype), plans in zip(cases, planned(cases)):
        for tile, segments, each, direct in plans:
            # five chunks in a row use each place of a ring of three again, three that of a ring of two
            if -(-min(each, c[1]) // 64) >= 5:
                outputs.add((dtype, tile, direct))
            if segments > 1 and each // 64 >= 3:
                sums.add((dtype, tile, direct))
    every = {(dtype, tile, direct) for dtype, tiles in TILES.items() for tile in tiles for direct in (False, True)}
    assert outputs == every, every - outputs
    assert sums == every, every - sums


def test_plans_are_within_what_the_kernels_take(planned):
    sizes = [(b, t, h, 1, d, e) for b in (1, 3, 700) for t in (1, 64, 65, 1000, 70000) for h in (1, 5, 64)
             for d, e in ((1, 1), (64, 65), (129, 32), (256, 256), (40, 256))]
    cases = [(c, dtype) for c in sizes for dtype in TILES]
    for (c, dtype), plans in zip(cases, planned(cases)):
        for n, (tile, segments, each, _) in enumerate(plans):
            assert tile in TILES[dtype] and tile[0] >= (max(c[4:]) if n else c[4]), (c, dtype)
            assert each % 64 == 0 and segments * each >= c[1] > (segments - 1) * each, (c, dtype)
