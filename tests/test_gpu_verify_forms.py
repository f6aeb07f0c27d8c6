"""sdv_verify_drafts: forms and limits beside those of tests/test_gpu_verify_drafts.py."""
import pytest
import torch

from tests.test_gpu_verify_drafts import F32, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("B,S,V,probs", [(1, 5, 30000, False), (30, 3, 9000, True), (200, 1, 5000, False)])
def test_inputs_that_the_launch_in_front_writes(sdv, B, S, V, probs):
    real = make(F32, B, S, V, probs, 16)
    want = call(sdv, real)[:2]
    mine = [None if x is None else torch.zeros_like(x) for x in real]
    ws = sdv.verify_drafts_workspace(real[0])
    given = [i for i, x in enumerate(real) if x is not None]
    for last in given:
        for _ in range(8):
            for i in given:
                mine[i].zero_()
            for i in [i for i in given if i != last] + [last]:
                mine[i].copy_(real[i])
            accepted, token, _ = call(sdv, mine, ws)
            assert torch.equal(accepted, want[0]) and torch.equal(token, want[1]), last
