"""How grouped products and adapters split their work (csrc/qmm_internal.h,
csrc/lora_plan.h), built for the host alone: the rules the kernels rely on over
many sizes and chips, and that the shapes of the GPU tests take every form that
a 256-CU chip takes."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_grouped_paths as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPE = {"mxfp4": 0, "q4_0": 1, "q4_b64": 1, "q8_0": 2, "q8_b64": 2}


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                        os.path.join(ROOT, "tests", "plan", "grouped_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(launches):
        r = subprocess.run([exe], input="".join(l + "\n" for l in launches), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        plans = [dict(f.split("=") for f in l.split()) for l in r.stdout.splitlines()]
        assert len(plans) == len(launches)
        return plans

    return run


def _spread(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step)


@pytest.mark.parametrize("cus", [32, 64, 128, 256, 304])
def test_rules(plan, cus):
    rng = random.Random(cus)
    plan([f"grouped {cus} {rng.randint(0, 2)} {rng.randint(0, 1)} {_spread(rng, 1, 1 << 28)} {rng.choice((0, _spread(rng, 32, 1 << 28, 32)))} "
          f"{_spread(rng, 1, (1 << 31) - 1)} {_spread(rng, 1, 1024)}" for _ in range(10000)])
    plan([f"grouped {cus} {t} {p} {M} {K} {R} {E}" for t in range(3) for p in (0, 1) for M in (1, 1 << 28) for K in (0, 32, 1 << 28)
          for R in (1, (1 << 31) - 1) for E in (1, 1024)])
    plan([f"lora {cus} {_spread(rng, 1, 1 << 24)} {rng.choice((0, _spread(rng, 32, (1 << 23) - 32, 32)))} {_spread(rng, 1, (1 << 24) - 1)} "
          f"{_spread(rng, 8, 128, 8)} {rng.randint(0, 1)}" for _ in range(10000)])
    plan([f"lora {cus} {N} {K} {M} {r} {w}" for N in (1, 256, 257, 512, 513, 1 << 24) for K in (0, 32, (1 << 23) - 32)
          for M in (1, (1 << 24) - 1) for r in (8, 128) for w in (0, 1)])


def test_gpu_shapes_take_every_form(plan):
    launches, kinds = [], []
    for kind in TYPE:
        for pair, M, K, rows, E in P.PRODUCTS:
            K = (K + 63) // 64 * 64 if kind.endswith("b64") or kind == "mxfp4" else K
            launches.append(f"grouped 256 {TYPE[kind]} {pair} {M} {K} {rows} {E}")
            kinds.append((kind, pair))
    got = {(*k, p["form"]) for k, p in zip(kinds, plan(launches))}
    assert got == {(k, pair, form) for k in TYPE for pair in (0, 1) for form in ("0", "1", "2", "2deep", "4", "4deep")}
    depths = {(*k, p["depth"]) for k, p in zip(kinds, plan(launches)) if p["form"] == "0"}
    assert {d for *_, d in depths} == {"4", "8"}
    plans = plan([f"grouped 256 {TYPE[k]} {pair} {M} {K} {rows} {E}" for k, pair, M, K, rows, E in P.STREAMED])
    assert all(p["form"] == "0" for p in plans) and {p["tiles"] for p in plans} == {"2", "4"}
    assert {(TYPE[s[0]], p["tiles"]) for s, p in zip(P.STREAMED, plans)} >= {(0, "2"), (0, "4"), (1, "2"), (1, "4"), (2, "2")}
    assert {p["depth"] for p in plans} == {"4", "8"}


def test_gpu_adapters_take_every_form(plan):
    plans = plan([f"lora 256 {N} {K} {M} {r} {wide}" for N, L, r, K, M, kind, wide in P.ADAPTERS])
    forms = {(p["single"], p["tiled"] if p["single"] == "0" else "-") for p in plans}
    assert forms == {("1", "-"), ("0", "0"), ("0", "1")}
    one = [(p, s) for p, s in zip(plans, P.ADAPTERS) if p["single"] == "1"]
    assert {s[2] for _, s in one} >= {8, 16, 32, 64, 128} and {s[5] for _, s in one} == {"f32", "bf16"}
    assert {p["mt"] for p, _ in one} >= {"1", "2", "3"} and max(s[0] for _, s in one) > 256
    two = [(p, s[5]) for p, s in zip(plans, P.ADAPTERS) if p["single"] == "0"]
    for tiled in "01":
        these = [(p, kind) for p, kind in two if p["tiled"] == tiled]
        assert {p["rt"] for p, _ in these} == {"1", "2", "4", "8"}
        assert {kind for _, kind in these} == {"f32", "bf16"}
        assert {p["chunks"] for p, _ in these} >= {"1", "2", "4"}
    assert {p["mt"] for p, _ in two} == {"1", "2", "4", "8"}
    assert {p["j1"] for p, _ in two} >= {"1", "2", "4", "8", "16"} and {p["j2"] for p, _ in two} >= {"1", "2", "16", "32"}
