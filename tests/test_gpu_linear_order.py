"""sdv_linear_attn reads what the launch in front of it in the stream writes, in the form of two launches
whose second runs beside the first, and in those of one."""
import pytest
import torch

from tests.test_gpu_linear_attn import BF16, F16, make, sdv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,B,T,H,hqk,dk,dv", [(F16, 1, 3000, 32, 16, 128, 128), (BF16, 5, 700, 12, 12, 64, 128),
                                                (F16, 2, 129, 4, 2, 128, 64), (BF16, 3, 100, 8, 4, 64, 64)])
def test_inputs_that_the_launch_in_front_writes(sdv, dt, B, T, H, hqk, dk, dv):  # noqa: F811
    q, k, v, g, s = (x.cuda() for x in make(dt, B, T, H, hqk, dk, dv, 71))
    n = torch.tensor([T - 3 * b for b in range(B)], dtype=torch.int32).cuda()
    ws = sdv.linear_attn_workspace(k, v)
    real = (q, k, v, g, n, s)
    mine = [torch.zeros_like(x) for x in real]

    def call(x, o, state):
        sdv.sdv_linear_attn(x[0], x[1], x[2], x[3], 0.3, x[4], x[5], state, o, ws)

    want, ws_out = torch.zeros_like(v), torch.zeros_like(s)
    call(real, want, ws_out)
    o, state = torch.empty_like(want), torch.empty_like(ws_out)
    for last in range(len(real)):
        for _ in range(6):
            for x in (*mine, o, state):
                x.zero_()
            for i in [*range(last + 1, len(real)), *range(last + 1)]:
                mine[i].copy_(real[i])
            call(mine, o, state)
            assert torch.equal(o, want) and torch.equal(state, ws_out), last
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
