"""How the launches over row tiles split their work (csrc/row_plan.h), built for
the host alone: the rules the kernels rely on over many sizes and chips, and
that the shapes of the GPU tests take every path that a 256-CU chip takes."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_moe_paths
import test_gpu_mx_paths
from quantized_matmul_ggml_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                        os.path.join(ROOT, "tests", "plan", "plan_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(launches):
        r = subprocess.run([exe], input="".join(l + "\n" for l in launches), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        plans = [dict(f.split("=") for f in l.split()) for l in r.stdout.splitlines()]
        assert len(plans) == len(launches)
        return plans

    return run


def _spread(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def _gemv(rng, cus, most, batch=True):
    count = rng.choice((1, 1, 2, 3, 5, 8)) if batch else 1
    pair = count == 1 and rng.random() < 0.5
    K = 0 if rng.random() < 0.02 else _spread(rng, 32, 40000, 32)
    return f"mx {cus} {int(pair)} {K} {rng.randint(1, 8)} " + " ".join(str(_spread(rng, 1, most)) for _ in range(count))


def _experts(rng, cus):
    E = _spread(rng, 1, 300)
    return (f"moe {cus} {rng.choice((B.MXFP4, B.Q4_0, B.Q8_0))} {E} {rng.randint(1, 16)} {rng.randint(1, 8)} "
            f"{rng.choice((0, _spread(rng, 32, 100000, 32)))} {rng.choice((0, _spread(rng, 32, 40000, 32)))}")


@pytest.mark.parametrize("cus", [32, 64, 128, 256, 304])
def test_rules(plan, cus):
    rng = random.Random(cus)
    plan([_gemv(rng, cus, 1 << 22) for _ in range(10000)] + [_experts(rng, cus) for _ in range(5000)])
    plan([f"mx {cus} 0 {K} {N} {M}" for K in (0, 32, 1 << 26) for N in (1, 8) for M in (1, (1 << 31) - 1)])


def _gemv_path(p):
    return tuple(p[f] for f in ("tg", "pair", "half", "depth", "passes", "loops", "halved", "more"))


def test_gpu_shapes_take_every_gemv_path(plan):
    rng = random.Random(5)
    taken = {_gemv_path(p) for p in plan([f"mx 256 {pair} {K} {N} {M}" for pair, M, K, N in test_gpu_mx_paths.PATHS])}
    every = {_gemv_path(p) for p in plan([_gemv(rng, 256, 120000, batch=False) for _ in range(30000)])}
    assert len(every) > 90 and every <= taken, every - taken
    # all instantiations: two token groups or one, alone or a pair, four depths;
    # eight-row tiles with three
    assert len({p[:4] for p in taken}) == 2 * 2 * 4 + 3


def test_gpu_shapes_take_every_experts_path(plan):
    types = {"mxfp4": B.MXFP4, "q4_0": B.Q4_0, "q8_0": B.Q8_0, "q4_b64": B.Q4_0, "q8_b64": B.Q8_0}
    rng = random.Random(6)
    path = lambda p: (p["type"], p["depth"], p["passes"])
    taken = {path(p) for p in plan([f"moe 256 {types[t]} {E} {k} {N} {F} {K}" for t, E, k, N, K, F, M in test_gpu_moe_paths.PATHS])}
    every = {path(p) for p in plan([_experts(rng, 256) for _ in range(20000)])}
    assert every <= taken, every - taken
