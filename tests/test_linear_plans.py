"""The linear layers' plans, on the host: the sizes that the GPU tests compare reach every kernel."""
import pytest

import self_attention_gb300 as sa
import _linear_plans as plans
from self_attention_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sa.load_library(build())


@pytest.mark.parametrize("what", plans.REQUIRED)
def test_the_sizes_reach_every_kernel(what):
    missing = plans.REQUIRED[what] - plans.reached()[what]
    assert not missing, f"{what}: no size of tests/_linear_plans.py reaches {sorted(missing)}"


def test_refusals_and_ranges():
    f = sa.attn_debug_linear_plan
    for bad in (lambda: f(3, 1, 1, 16, 64, 32), lambda: f(-1, 1, 1, 16, 64, 32), lambda: f(0, 1, 1, 16, 60, 32),
                lambda: f(0, 1, 1, 0, 64, 32), lambda: f(1, 1, 1, 16, 72, 32), lambda: f(1, 2, 2, 16, 64, 32),
                lambda: f(0, 2, 2, 16, 64, 32, 1), lambda: f(0, 2, 2, 16, 96, 32), lambda: f(2, 1, 1, 16, 64, 32, 9),
                lambda: f(0, 1, 1, (1 << 31) - 1, 8, 8)):
        with pytest.raises(sa.AttnError):
            bad()
    assert sa.load_library().attn_debug_linear_plan(0, 1, 1, 16, 64, 32, 0, None) == 1
    for M in (1, 100, 10_000):
        rows, splits, bn, dw, bias = f(0, 1, 1, M, 512, 512)
        assert (rows in (16, 32, 64, 128) and splits in (1, 2, 4, 8) and bn == 0) or (rows == splits == 0 and bn in (128, 256))
        assert dw == bias == 0
        rows, splits, bn, dw, bias = f(2, 1, 1, M, 512, 512, 2)
        assert bn in (128, 256) and 1 <= dw <= 16 and bias == 0      # dz is made first, and its sums with it
