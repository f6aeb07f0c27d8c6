"""sdv_prefix_attn reads what the launch in front of it in the stream writes, and its last launch what
its first ones do: every form that has launches of its own for the prefix and the own positions."""
import pytest
import torch

from tests.test_gpu_prefix_attn import BF16, F16, call, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,prefix,own,width", [
    (F16, 40, 1, 32, 8, 128, 16, 700, 90, 0),      # the own positions in parts, a launch that joins
    (BF16, 300, 2, 32, 8, 64, 16, 300, 30, 0),     # joined where the own positions are computed
    (F16, 12, 9, 16, 2, 256, 16, 500, 100, 0),     # several row groups of wide heads
    (BF16, 6, 4, 16, 2, 128, 16, 500, 200, 40000),  # the paged attention for the own positions
    (F16, 6, 4, 16, 2, 96, 16, 300, 60, 0),        # head sizes outside the tensor-core kernel's
])
def test_inputs_that_the_launch_in_front_writes(sdv, dt, B, S, hq, hkv, d, page, prefix, own, width):
    ctx, n = [own - i % 7 for i in range(B)], [S - i % 2 for i in range(B)]
    q, kp, vp, ptable, table = make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, 61)
    if width:
        wide = torch.full((B, width // page), -1, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    q, kp, vp, ptable, table = (x.cuda() for x in (q, kp, vp, ptable, table))
    want, wl, ws = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, None, d ** -0.5)
    real = (q, kp, vp, ptable, dev([prefix]), table, dev(ctx), dev(n))
    mine = [torch.zeros_like(x) for x in real]
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    for last in range(len(real)):
        for _ in range(8):
            for x in mine:
                x.zero_()
            # every input is once the one whose copy is directly in front
            for i in [*range(last + 1, len(real)), *range(last + 1)]:
                mine[i].copy_(real[i])
            sdv.sdv_prefix_attn(*mine, None, d ** -0.5, out, lse, ws)
            assert torch.equal(out, want) and torch.equal(lse, wl), last
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
