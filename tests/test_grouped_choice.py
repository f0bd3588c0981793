"""Which form a launch of grouped products takes (csrc/qmm_internal.h, built for the
host alone), where one form is many times slower than another."""
import pytest

import test_gpu_grouped_more as more
from test_grouped_plan import TYPE, plan  # noqa: F401 (a fixture)


@pytest.mark.parametrize("kind", ["mxfp4", "q4_0", "q8_0"])
def test_many_rows_of_few_outputs_are_not_streamed(plan, kind):  # noqa: F811
    """Streamed, a workgroup of sixteen rows costs its start whatever its work is: such
    launches took two to ten times as long as in tiles."""
    shapes = [(0, 64, 64, 1000000, 8), (0, 64, 64, 32768, 8), (0, 65, 256, 32768, 8), (0, 16, 64, 200000, 8), (0, 33, 96, 100000, 1),
              (1, 64, 64, 32768, 64), (1, 16, 64, 20000, 1), (0, 1024, 128, 4096, 64)]
    shapes += [(pair, M, K, R, E) for pair, M, K, R, E in more.FEW_OUTPUTS]
    plans = plan([f"grouped 256 {TYPE[kind]} {p} {M} {K} {R} {E}" for p, M, K, R, E in shapes])
    assert [s for s, p in zip(shapes, plans) if p["form"] == "0"] == []
