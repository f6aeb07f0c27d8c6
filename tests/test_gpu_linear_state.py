"""States of sdv_linear_attn are fp32: terms kept to more bits than their type has.

A term e^{G_T - G_t} k_t v_t of the state may be off by 2^-20 of itself: decayed keys are
held to 2^-22, the exponential is good to 2^-22, its argument, below 16 for the terms that
count, is rounded at 2^-21.  Errors of different terms are independent, so with q the sum
of the terms' squares (the oracle's state of squared keys and values under the doubled
decay) the errors' root mean square is below 2^-20 sqrt(q)'s; sums of fp32 add 2^-24 of
the state for each of the additions it goes through, a chunk of 128 tokens or a token:
  rms(M - ref) <= 2^-20 rms(sqrt(q)) + (additions + 16) 2^-24 rms(ref).
"""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests import test_gpu_linear_attn as lin
from tests.rounding_checks import rms
from tests.test_gpu_linear_attn import BF16, F16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("B,T,H,hqk,dk,dv,n", [
    (2, 20, 2, 1, 128, 128, [20, 7]), (2, 100, 2, 2, 128, 128, None), (2, 200, 2, 1, 64, 64, [200, 130]),
    (1, 515, 4, 2, 64, 128, None), (1, 1500, 2, 1, 128, 128, None), (2, 400, 2, 1, 128, 64, [400, 129]),
    (1, 4100, 1, 1, 64, 128, None), (1, 6000, 1, 1, 128, 128, None), (1, 50, 2, 1, 96, 40, None)])
@pytest.mark.parametrize("rate", [0.0, 0.02, 0.4])
@pytest.mark.parametrize("outputs", [True, False])
def test_states_are_held_in_fp32(sdv, dt, B, T, H, hqk, dk, dv, n, rate, outputs):
    q, k, v, g, s = lin.make(dt, B, T, H, hqk, dk, dv, 96, rate=rate)
    _, state = lin.call(sdv, q if outputs else None, k, v, g, n, s, want_o=outputs)
    count = n or [T] * B
    ref = mixing.linear(None, f64(k), f64(v), f64(g), 1.0, count, f64(s))["state"]
    squares = mixing.linear(None, f64(k) ** 2, f64(v) ** 2, 2 * f64(g), 1.0, count, f64(s) ** 2)["state"]
    additions = T if T <= 32 or dk not in (64, 128) or dv not in (64, 128) else -(-T // 128)
    for b in range(B):
        limit = 2.0 ** -20 * rms(np.sqrt(squares[b])) + (additions + 16) * 2.0 ** -24 * rms(ref[b])
        err = rms(f64(state)[b] - ref[b])
        assert err <= limit, f"{err:.3e} where {limit:.3e} is the most, of {rms(ref[b]):.3e}"
