"""sdv_linear_attn where a query is infinite or NaN: its own row is not finite, every
other row and the state are what they are without it (test_gpu_linear_attn's bounds)."""
import numpy as np
import pytest
import torch

from tests import test_gpu_linear_attn as lin
from tests.test_gpu_linear_attn import BF16, F16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [1, 3, 20, 90, 300])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_is_not_finite_reaches_its_own_row_alone(sdv, dt, T, value):
    q, k, v, g, s = lin.make(dt, 2, T, 4, 2, 128, 64, 95)
    ref = lin.oracle(q, k, v, g, None, s)
    at = T // 2
    q[1, at, 0, 7] = value  # of value heads 0 and 1
    o, state = lin.call(sdv, q, k, v, g, None, s)
    got = f64(o)
    assert not np.isfinite(got[1, at, :2]).any()
    got[1, at, :2] = ref["o"][1, at, :2]
    lin.check(dt, ref, torch.from_numpy(got), state, T)
