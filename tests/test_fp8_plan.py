"""The kernel choice of the block-scaled e4m3 products (csrc/ar_fp8_plan.h), built with g++
into a small driver (tests/fp8_plan_driver.cpp): the shapes that the GPU tests run
reach the kernels that they name, and every kernel of the library. CPU only."""
import os
import shutil
import subprocess

import pytest

from fp8_shapes import DENSE, GROUPED

HERE = os.path.dirname(os.path.abspath(__file__))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

TILES = ("32x64", "64x64", "64x128", "128x128")
KERNELS = {(t, sets, out) for t in TILES for sets in (1, 2) for out in ("bf16", "f32")} | \
    {("rows", 1, "bf16"), ("rows", 1, "f32"), ("256x256", 1, "bf16")}


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_plan_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
           "-fno-sanitize-recover=all", os.path.join(HERE, "fp8_plan_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(shapes):
        """[(grouped, wide, R, N, K, E)] -> [(tile, K sets)]"""
        text = "\n".join(" ".join(str(int(v)) for v in s) for s in shapes) + "\n"
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        got = [ln.split() for ln in r.stdout.splitlines()]
        assert len(got) == len(shapes)
        return [(t, int(s)) for t, s in got]
    return ask


def test_dense_shapes_reach_every_kernel(plan):
    got = plan([(False, c[2] == "f32", *c[3:], 1) for c in DENSE])
    assert got == [c[:2] for c in DENSE]
    assert {c[:3] for c in DENSE} == KERNELS


def test_shapes_by_expert_reach_every_kernel(plan):
    got = plan([(True, c[2] == "f32", *c[3:]) for c in GROUPED])
    assert got == [c[:2] for c in GROUPED]
    assert {c[:3] for c in GROUPED} == KERNELS


def test_tile_kernels_pass_a_window_of_scales(plan):
    """W's scales are held 64 blocks of K at a time: every tile kernel runs past one
    window, dense or by expert."""
    long = {c[:3] for c in DENSE + GROUPED if c[5] > 64 * 128 * c[1]}
    assert long >= {k for k in KERNELS if k[0] != "rows" and k[1] == 1}
    assert {k[0] for k in long if k[1] == 2} == set(TILES)


@pytest.mark.parametrize("shape", [(True, False, 1, 16, 16, 8192), (True, True, 8000000, 16, 16, 1),
                                   (False, False, 8000000, 8000000, 16, 1),
                                   (False, True, 1, 1, 4194288, 1),
                                   (True, False, 8000000, 8000000, 4194288, 8192)])
def test_extreme_shapes_have_a_plan(plan, shape):
    assert plan([shape])[0][0] in TILES + ("rows", "256x256")
