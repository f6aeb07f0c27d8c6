"""Workspaces of the token mixers: one that holds a window (or a prompt) holds every
shorter one of the same heads, so a program allocates once for its largest."""
import pytest
import torch

from tests import test_gpu_linear_attn as lin
from tests import test_gpu_paged_attn as att


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


@pytest.mark.parametrize("heads", [1, 2, 8])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 8, 12, 16, 33, 64, 100, 128, 129])
@pytest.mark.parametrize("dim", [8, 64, 96, 128, 256])
def test_attention_windows_fit_the_largest_ones_workspace(sdv, heads, group, dim):
    sizes = [sdv.sdv_paged_attn_workspace_bytes(2, S, heads * group, heads, dim) for S in range(1, 33)]
    assert sizes == sorted(sizes) and sizes[0] >= 256


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,dim,page,most,shorter", [(6, 1, 128, 16, 32, (1, 17, 21, 22)),
                                                          (16, 2, 256, 64, 17, (1, 10, 16)),
                                                          (6, 1, 96, 16, 32, (17, 2))])
def test_one_workspace_serves_shorter_windows(sdv, hq, hkv, dim, page, most, shorter):
    ctx = [3000]
    q, kp, vp, table = (x.cuda() for x in att.make(torch.float16, 1, most, hq, hkv, dim, page, ctx, [most], 1))
    ws = sdv.paged_attn_workspace(q, kp, table)
    for S in shorter:
        part = q[:, :S].contiguous()
        want, _, _ = att.call(sdv, part, kp, vp, table, ctx, [S], None, 0.1)
        got, _, _ = att.call(sdv, part, kp, vp, table, ctx, [S], None, 0.1, ws=ws)
        assert torch.equal(got, want) and sdv.sdv_last_device_status(ws) == sdv.SDV_OK


@pytest.mark.parametrize("B,H,dk,dv", [(1, 2, 128, 128), (40, 7, 64, 64), (300, 4096, 64, 128), (2, 3, 96, 128)])
def test_linear_prompts_fit_the_longest_ones_workspace(sdv, B, H, dk, dv):
    lengths = [1, 6, 31, 32, 33, 128, 129, 3000, 100000, 2 ** 22, 2 ** 25, 2 ** 30, 2 ** 31 - 1]
    sizes = [sdv.sdv_linear_attn_workspace_bytes(B, T, H, dk, dv) for T in lengths]
    assert sizes == sorted(sizes) and sizes[0] >= 256
    more = [sdv.sdv_linear_attn_workspace_bytes(b, 5000, H, dk, dv) for b in (1, 2, 100, 5000, 65535)]
    assert more == sorted(more)


@pytest.mark.gpu
def test_one_workspace_serves_shorter_prompts(sdv):
    big = lin.make(torch.bfloat16, 3, 900, 4, 2, 128, 64, 2)
    ws = sdv.linear_attn_workspace(big[1], big[2])
    for B, T in ((3, 130), (1, 900), (2, 33), (3, 8), (1, 1)):
        q, k, v, g, s = lin.make(torch.bfloat16, B, T, 4, 2, 128, 64, 3)
        want, want_s = lin.call(sdv, q, k, v, g, None, s)
        o, state = torch.empty_like(want), torch.empty_like(want_s)
        sdv.sdv_linear_attn(q, k, v, g, 0.3, None, s, state, o, ws)
        assert torch.equal(o, want) and torch.equal(state, want_s)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
