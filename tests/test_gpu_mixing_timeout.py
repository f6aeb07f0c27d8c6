"""The bounded-wait timeout path of the token mixers' tensor-core kernels, made to run
on purpose without faulting or hanging anything (as test_gpu_timeout does for the heads).

sdv_debug_fault keeps one copy of each CTA from being asked for: the roles waiting for
it find a barrier that nothing completes, give up after 2 ms, and the CTA waits for the
copies that it did ask for, frees its tensor memory and ends.  The status read returns
SDV_ERR_TIMEOUT once, the workspace's head is zero again (arrivals that a dead CTA owed
its shared units among them), and the next call on that workspace is the one before.
"""
import pytest
import torch

from tests import test_gpu_linear_attn as lin
from tests import test_gpu_paged_attn as att
from tests.test_gpu_paged_attn import BF16, F16
from tests.test_gpu_timeout import fault

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("stage", [0, 1, 2, 6])
@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,ctx", [
    (F16, 2, 1, 32, 8, 128, 16, [5003, 700]),          # units joined by their last CTA, 1 to 3 tiles a CTA
    (BF16, 1, 1, 8, 1, 64, 16, [90000]),
    (F16, 60, 1, 8, 8, 128, 64, [31 * i % 900 for i in range(60)]),  # many units a CTA
    (F16, 2, 20, 8, 2, 128, 16, [3000, 40]),            # rows that fill the tile, a join of its own
    (BF16, 40, 17, 16, 2, 256, 64, [17 * i for i in range(40)]),
    (F16, 6, 8, 8, 2, 64, 32, [9000, 1, 0, 300, 64, 5])])
def test_attention_timeout_reported_then_next_call_correct(sdv, dt, B, S, hq, hkv, d, page, ctx, stage):
    n = [S] * B
    q, kp, vp, table = (x.cuda() for x in att.make(dt, B, S, hq, hkv, d, page, ctx, n, 70))
    want, _, ws = att.call(sdv, q, kp, vp, table, ctx, n, None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    with fault(sdv, stage):
        att.call(sdv, q, kp, vp, table, ctx, n, None, d ** -0.5, ws=ws)
        status = sdv.sdv_last_device_status(ws)
    tiles = sum((c + S + 127) // 128 for c in ctx) * hkv
    if stage == 0 or tiles > 152 * (stage + 3):  # every CTA has that many
        assert status == sdv.SDV_ERR_TIMEOUT
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    assert not ws[:256].any()
    for _ in range(2):
        got, _, _ = att.call(sdv, q, kp, vp, table, ctx, n, None, d ** -0.5, ws=ws)
        assert torch.equal(got, want) and sdv.sdv_last_device_status(ws) == sdv.SDV_OK


@pytest.mark.parametrize("stage", [0, 1, 3])
@pytest.mark.parametrize("dt,B,T,H,hqk,dk,dv,parts", [
    (F16, 1, 5000, 8, 4, 128, 128, "both"),             # heads that many CTAs share: both launches
    (BF16, 2, 3000, 30, 10, 64, 128, "both"),
    (F16, 3, 100, 60, 60, 64, 64, "both"),              # one chunk a head: the second launch alone
    (BF16, 2, 4000, 24, 24, 128, 64, "state"),
    (F16, 2, 4000, 24, 24, 128, 128, "outputs")])
def test_linear_timeout_reported_then_next_call_correct(sdv, dt, B, T, H, hqk, dk, dv, parts, stage):
    q, k, v, g, s = lin.make(dt, B, T, H, hqk, dk, dv, 71, rate=0.01)
    want, want_s = lin.call(sdv, q, k, v, g, None, s)
    ws = sdv.linear_attn_workspace(k, v)

    def call():
        o = torch.full_like(want, float("nan")) if parts != "state" else None
        state = torch.full_like(want_s, float("nan")) if parts != "outputs" else None
        sdv.sdv_linear_attn(q, k, v, g, 0.3, None, s, state, o, ws)
        return o, state, sdv.sdv_last_device_status(ws)

    with fault(sdv, stage):
        status = call()[2]
    if stage == 0 or B * H * (-(-T // 128)) > 152 * (stage + 1):
        assert status == sdv.SDV_ERR_TIMEOUT
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK and not ws[:256].any()
    for _ in range(2):
        o, state, status = call()
        assert status == sdv.SDV_OK
        assert o is None or torch.equal(o, want)
        assert state is None or torch.equal(state, want_s)
