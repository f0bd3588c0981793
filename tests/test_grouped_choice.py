"""Which form a launch of grouped products takes (csrc/qmm_internal.h, built for the
host alone), where one form is many times slower than another."""
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_grouped_contents as contents
import test_gpu_grouped_more as more
import test_gpu_layer_split as split
import test_gpu_lora_contents as adapters
from test_grouped_plan import ROOT, TYPE, _spread, plan  # noqa: F401 (a fixture)


@pytest.mark.parametrize("kind", ["mxfp4", "q4_0", "q8_0"])
def test_many_rows_of_few_outputs_are_not_streamed(plan, kind):  # noqa: F811
    """Streamed, a workgroup of sixteen rows costs its start whatever its work is: such
    launches took two to ten times as long as in tiles."""
    shapes = [(0, 64, 64, 1000000, 8), (0, 64, 64, 32768, 8), (0, 65, 256, 32768, 8), (0, 16, 64, 200000, 8), (0, 33, 96, 100000, 1),
              (1, 64, 64, 32768, 64), (1, 16, 64, 20000, 1), (0, 1024, 128, 4096, 64)]
    shapes += [(pair, M, K, R, E) for pair, M, K, R, E in more.FEW_OUTPUTS]
    plans = plan([f"grouped 256 {TYPE[kind]} {p} {M} {K} {R} {E}" for p, M, K, R, E in shapes])
    assert [s for s, p in zip(shapes, plans) if p["form"] == "0"] == []


def test_no_launch_is_refused_that_some_form_takes(plan):  # noqa: F811
    """The header's limit: fewer than 2^23 tiles of 128 rows and 128 (the pair: 64)
    outputs, whichever form is estimated to be the fastest."""
    shapes = [(p, M, K, R, E) for p in (0, 1) for M in (16, 64, 65, 2048, 1 << 20, 1 << 26) for K in (32, 64, 256, 2048)
              for R in (1, 1000, 1 << 20, 1 << 27, 1 << 28, 1 << 29, (1 << 30) - 1, 1 << 30, (1 << 31) - 1) for E in (1, 8, 1024)]
    shapes += [(p, M, K, R, E) for p, M, K, R, E, *_ in more.MOST_ROWS]
    for kind in ("mxfp4", "q4_0", "q8_0"):
        plans = plan([f"grouped 256 {TYPE[kind]} {p} {M} {K} {R} {E}" for p, M, K, R, E in shapes])
        for (p, M, K, R, E), q in zip(shapes, plans):
            rows, bm = (R + 127 * min(E, R)) // 128, 64 if p else 128
            if rows * -(-M // bm) < 1 << 23:
                assert q["fits"] == "1", (kind, p, M, K, R, E)


def test_shapes_of_the_contents_tests_take_every_form(plan):  # noqa: F811
    for form, shapes in contents.SHAPES.items():
        assert [s[0] for s in shapes] == [0, 1]
        for kind in TYPE:
            got = plan([f"grouped 256 {TYPE[kind]} {p} {M} {K} {R} {contents.E}" for p, M, K, R in shapes])
            assert [p["form"] for p in got] == [form, form], (kind, form)


def test_shapes_of_the_adapters_contents_tests_take_every_form(plan):  # noqa: F811
    shapes = adapters.SHAPES.values()
    plans = plan([f"lora 256 {N} {K} {M} {r} 1" for N, L, r, K, M in shapes])
    got = ["one launch" if p["single"] == "1" else "tiles" if p["tiled"] == "1" else "registers" for p in plans]
    assert got == list(adapters.SHAPES)


def test_second_product_of_a_layer_with_h_in_two_parts(tmp_path):
    """Its rules, and that the GPU tests' shapes take every form."""
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "plan")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                        os.path.join(ROOT, "tests", "plan", "layer_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def forms(launches):
        r = subprocess.run([exe], input="".join(" ".join(map(str, v)) + "\n" for v in launches), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return [v.split() for v in r.stdout.splitlines()]

    rng = random.Random(9)
    launches = [(rng.choice((32, 256, 304)), rng.randint(0, 2), _spread(rng, 1, 1 << 24), _spread(rng, 32, 1 << 21, 32), _spread(rng, 1, 1 << 28),
                 _spread(rng, 1, 1024)) for _ in range(10000)]
    assert len(forms(launches)) == len(launches)
    depths, tiles = set(), set()
    for form, shapes in split.SHAPES.items():
        for E, k, N, F, M in shapes:
            for kind in TYPE:
                (got, depth, per_wave, fits), = forms([(256, TYPE[kind], M, F, N * k, E)])
                assert got == form and fits == "1", (kind, form, E, k, N, F, M)
                if form == "0":
                    depths.add(depth)
                    tiles.add(per_wave)
    assert depths == {"4", "8"} and tiles >= {"1", "2"}
