"""Which kernel the products of the GPU tests run on: the rules of csrc/rz_i8_plan.h,
compiled for the host, on a device of 256 compute units.  A change of the rules that moves
a test to another kernel fails here.  CPU only."""
import functools
import os
import subprocess

import pytest

import test_i8_gpu as basic
import test_i8_shapes_gpu as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_razer_w4a16_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(m, n, k, experts) -> ("stream", row tiles a chunk, chunks a row, X tiles of 16 rows, rows a job)
    or ("tile", rows of W, rows of X, whole tiles, split tiles, slices, tiles done in halves)."""
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang missing")
    exe = str(tmp_path_factory.mktemp("plan") / "i8_plan")
    r = subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-o", exe, os.path.join(CSRC, "i8_plan_print.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    @functools.lru_cache(None)
    def of(m, n, k, experts=0):
        out = subprocess.run([exe, f"{m},{n},{k},{experts}"], capture_output=True, text=True, check=True).stdout.split()
        return (out[0], *map(int, out[1:]))
    return of


# row tiles a chunk, chunks a row, X tiles of 16 rows
FORMS = {(4, 1, 1), (4, 1, 2), (2, 1, 1), (2, 1, 2), (1, 1, 1), (1, 1, 2), (1, 1, 4), (1, 2, 1), (1, 2, 2), (1, 2, 4), (1, 4, 1),
         (1, 4, 2), (1, 8, 1)}


def test_every_form_of_the_stream_kernel(plan):
    assert {p[1:4] for p in (plan(*s) for s in shapes.FEW) if p[0] == "stream"} == FORMS
    assert {p[1:4] for p in (plan(*s) for s in shapes.GROUPS) if p[0] == "stream"} == FORMS


SHAPES = {(256, 256), (256, 128), (128, 128)}  # rows of W and of X of a tile


def test_tiles(plan):
    """Every shape with more tiles than workgroups and with fewer, with K cut (of all tiles, and of the
    last ones alone) and with experts; halves with and without rows."""
    def slots(p):
        return 512 if p[1] == 128 else 256

    got = [plan(*s) for s in shapes.TILES]
    assert {p[0] for p in got} == {"tile"} and {p[1:3] for p in got if p[3] > slots(p)} == SHAPES
    got = [plan(*s) for s in shapes.TILES + shapes.SLICES]
    assert {p[1:3] for p in got if 0 < p[3] <= slots(p) and p[4] == 0} == SHAPES
    got = [plan(*s) for s in shapes.HALVES]
    assert all(p[:3] == ("tile", 256, 256) and p[6] > 0 for p in got)
    assert any(m % 256 in range(1, 129) for m, _, _ in shapes.HALVES)  # a half without rows
    got = [plan(*s) for s in shapes.SLICES]
    assert {p[1:3] for p in got if p[5] > 1} == SHAPES
    assert {p[3] > 0 for p in got if p[5] > 1} == {False, True}
    got = [p for p in (plan(*s) for s in shapes.GROUPS) if p[0] == "tile"]
    assert {p[1:3] for p in got} == SHAPES and {p[1:3] for p in got if p[3] > slots(p)} == SHAPES


def test_both_kernels_in_the_tests_of_values(plan):
    assert {plan(*s)[0] for s in basic.SHAPES} == {"stream", "tile"}


@pytest.mark.parametrize("m,n,k,experts,want", [
    (1, 14336, 4096, 0, ("stream", 1, 2, 1)), (27, 28672, 8192, 0, ("stream", 1, 4, 2)), (1, 4096, 14336, 0, ("stream", 1, 8, 1)),
    (2048, 28672, 8192, 0, ("tile", 256, 256)), (16, 14336, 4096, 8, ("stream", 1, 2, 1)), (8192, 14336, 4096, 8, ("tile", 256, 256)),
    (999, 1503, 2080, 64, ("stream", 1, 2, 2)), (1, 8192, 16384, 0, ("stream", 1, 8, 1)), (1, 8192, 16400, 0, ("tile", 256, 128)),
    (1024, 4096, 4096, 0, ("tile", 128, 128)), (2048, 4096, 4096, 0, ("tile", 256, 128)), (512, 14336, 4096, 0, ("tile", 256, 128)),
])
def test_forms_of_ordinary_sizes(plan, m, n, k, experts, want):
    assert plan(m, n, k, experts)[:len(want)] == want


def test_sizes_at_the_ends_of_their_range(plan):
    for s in ((2 ** 30, 2 ** 30, 131056, 0), (2 ** 30, 2 ** 18, 131056, 4096), (1, 2 ** 30, 16, 0), (2 ** 30, 1, 131056, 0)):
        kind, *rest = plan(*s)
        assert kind in ("stream", "tile") and min(rest) >= 0
