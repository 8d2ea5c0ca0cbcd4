"""Which kernel the MXFP4 products of the GPU tests run on: the rules of
csrc/rz_mx_plan.h, compiled for the host, on a device of 256 compute units.  A change of
the rules that moves a test to another kernel fails here.  CPU only."""
import functools
import os
import subprocess

import pytest

import test_mx_gpu as basic
import test_mx_large_experts_gpu as large
import test_mx_shapes_gpu as shapes
import test_mx_short_gpu as short

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_razer_w4a16_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(m, n, k, experts) -> ("stream", row tiles a chunk, chunks a row, X tiles of 16 rows, rows a job)
    or ("tile", rows, whole tiles, split tiles, slices)."""
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang missing")
    exe = str(tmp_path_factory.mktemp("plan") / "mx_plan")
    r = subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-o", exe, os.path.join(CSRC, "mx_plan_print.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    @functools.lru_cache(None)
    def of(m, n, k, experts=0):
        out = subprocess.run([exe, f"{m},{n},{k},{experts}"], capture_output=True, text=True, check=True).stdout.split()
        return (out[0], *map(int, out[1:]))
    return of


def parameters(test, *names):
    """The values of `names` that one mark of a test parametrises it with."""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0].split(",") == list(names):
            return mark.args[1]
    raise AssertionError(f"{test.__name__} has no parameters {names}")


def test_tiles(plan):
    """Both heights of a tile in every type; more tiles than compute units; K cut or not."""
    got = {s: plan(*s) for s in parameters(shapes.test_tiles, "m", "n", "k")}
    assert {p[:2] for p in got.values()} == {("tile", 128), ("tile", 256)}
    got = {s: plan(*s) for s in parameters(shapes.test_rounds_of_tiles, "m", "n", "k")}
    assert {p[:2] for p in got.values()} == {("tile", 128), ("tile", 256)}
    assert all(p[2] + p[3] > 256 for p in got.values())
    got = [plan(*s) for s in parameters(shapes.test_slices, "m", "n", "k")]
    assert {(p[:2], p[4] > 1) for p in got} == {(("tile", 128), True)}
    got = [plan(*s) for s in large.SPLIT]
    assert {(p[:2], p[4] > 1) for p in got} == {(("tile", 256), True)}


def test_tiles_of_experts(plan):
    got = {plan(sum(z), n, k, len(z))[:2] for n, k, z in large.GROUPS}
    assert got == {("tile", 256)}
    assert any(plan(sum(z), n, k, len(z))[2] > 256 for n, k, z in large.GROUPS)
    got = {plan(sum(z), n, k, len(z))[:2] for n, k, z in parameters(shapes.test_large_experts, "n", "k", "sizes")}
    assert got == {plan(sum(z), n, k, len(z))[:2] for n, k, z in large.TILES_128} == {("tile", 128)}


# row tiles a chunk, chunks a row, X tiles of 16 rows
FORMS = {(4, 1, 1), (4, 1, 2), (2, 1, 1), (2, 1, 2), (1, 1, 1), (1, 1, 2), (1, 1, 4), (1, 2, 1), (1, 2, 2), (1, 2, 4), (1, 4, 1), (1, 4, 2)}


def test_every_form_of_the_stream_kernel(plan):
    got = [plan(m, 4999, k) for m in parameters(shapes.test_few_rows, "m") for k in parameters(shapes.test_few_rows, "k")]
    got += [plan(*s) for s in parameters(short.test_many_short_rows, "m", "n", "k")]
    assert {p[1:4] for p in got if p[0] == "stream"} == FORMS
    got = [plan(sum(z), n, k, len(z)) for t in (shapes.test_small_experts, shapes.test_open_rows, short.test_experts_of_short_rows)
           for n, k, z in parameters(t, "n", "k", "sizes")]
    got += [plan(sum(z), n, k, len(z)) for n, k, z in large.SMALL + basic.GROUPS]
    assert {p[1:4] for p in got if p[0] == "stream"} == FORMS


@pytest.mark.parametrize("m,n,k,experts,want", [
    (1, 14336, 4096, 0, ("stream", 1, 1, 1)), (27, 28672, 8192, 0, ("stream", 1, 2, 2)), (1, 4096, 14336, 0, ("stream", 1, 4, 1)),
    (2048, 28672, 8192, 0, ("tile", 256)), (2041, 4096, 14336, 0, ("tile", 128)), (8192, 14336, 4096, 8, ("tile", 256)),
    (16, 14336, 4096, 8, ("stream", 1, 1, 1)), (999, 1503, 2080, 64, ("stream", 1, 1, 2)),
    (1, 8192, 15360, 0, ("stream", 1, 4, 1)), (1, 8192, 15392, 0, ("tile", 128)),  # longer rows than the stream kernel holds
    (4096, 8192, 480, 0, ("stream", 1, 1, 4)), (4096, 8192, 512, 0, ("tile", 256)),  # shorter rows than a window of scales
])
def test_forms_of_ordinary_sizes(plan, m, n, k, experts, want):
    assert plan(m, n, k, experts)[:len(want)] == want


def test_sizes_at_the_ends_of_their_range(plan):
    for s in ((2 ** 30, 2 ** 30, 2 ** 23, 0), (2 ** 30, 2 ** 18, 2 ** 23, 4096), (1, 2 ** 30, 32, 0), (2 ** 30, 1, 2 ** 23, 0)):
        kind, *rest = plan(*s)
        assert kind in ("stream", "tile") and min(rest) >= 0
