"""The bounded-wait timeout path of the attention behind a shared prefix, made to run on purpose without
faulting or hanging anything (as test_gpu_mixing_timeout does for the other token mixers): one copy of
each CTA is not asked for, the roles waiting for it give up after 2 ms, the CTA waits for the copies
that it did ask for and ends.  The status read returns SDV_ERR_TIMEOUT once, the workspace's head is
zero again, and the next call on that workspace is the one before."""
import pytest
import torch

from tests import test_gpu_prefix_attn as att
from tests.test_gpu_paged_attn import BF16, F16
from tests.test_gpu_timeout import fault

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("stage", [0, 1, 2, 5])
@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,prefix,ctx", [
    (F16, 4, 1, 32, 8, 128, 16, 1201, 90),        # one row tile, few tiles
    (BF16, 64, 1, 32, 8, 128, 16, 9000, 300),     # two row tiles a unit
    (F16, 24, 9, 16, 2, 256, 64, 3000, 200),      # wide heads
    (BF16, 33, 4, 8, 2, 64, 32, 700, 40),         # an odd number of row tiles
    (F16, 6, 5, 32, 8, 128, 16, 500, 200),        # two warps for a sequence's own positions
    (BF16, 4, 16, 16, 4, 64, 16, 500, 300)])      # four
def test_timeout_reported_then_next_call_correct(sdv, dt, B, S, hq, hkv, d, page, prefix, ctx, stage):
    ctx, n = [ctx] * B, [S] * B
    made = [x.cuda() for x in att.make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, 70)]
    args = (*made[:4], prefix, made[4], ctx, n, None, d ** -0.5)
    want, lse, ws = att.call(sdv, *args)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    with fault(sdv, stage):
        att.call(sdv, *args, ws=ws)
        status = sdv.sdv_last_device_status(ws)
    if stage == 0:  # every CTA with work has a first copy
        assert status == sdv.SDV_ERR_TIMEOUT
    assert status in (sdv.SDV_OK, sdv.SDV_ERR_TIMEOUT)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    assert not ws[:256].any()
    for _ in range(2):
        got, lse2, _ = att.call(sdv, *args, ws=ws)
        assert torch.equal(got, want) and torch.equal(lse2, lse) and sdv.sdv_last_device_status(ws) == sdv.SDV_OK
