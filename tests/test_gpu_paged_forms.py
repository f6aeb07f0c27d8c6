"""sdv_paged_attn: sides of its choices beside those of tests/test_gpu_paged_attn.py."""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests.test_gpu_paged_attn import BF16, F16, as_i32, call, check, f64, make, sdv, words  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,masked", [(F16, 80, 2, 8, 4, 96, 16, True), (BF16, 400, 1, 4, 1, 40, 5, False),
                                                         (F16, 52, 9, 16, 2, 72, 16, True)])
def test_many_units_in_the_form_for_other_sizes(sdv, dt, B, S, hq, hkv, d, page, masked):  # noqa: F811
    """More units than CTAs: their partials are joined by the CTAs' ranges.  A few long sequences among short
    ones, so that units begin and end inside ranges and some span several."""
    ctx = [1500 if b % 29 == 3 else (37 * b) % 120 for b in range(B)]
    n = [S - b % (S + 1) if b % 7 == 0 else S for b in range(B)]
    q, kp, vp, table = make(dt, B, S, hq, hkv, d, page, ctx, n, d)
    mask = words(np.random.default_rng(d), B, S) if masked else None
    im = None if mask is None else as_i32(mask)
    out, lse, ws = call(sdv, q, kp, vp, table, ctx, n, im, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    check(dt, mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, mask, d ** -0.5), out, lse, d)
    again, _, _ = call(sdv, q, kp, vp, table, ctx, n, im, d ** -0.5, ws=ws)
    assert torch.equal(again, out)
