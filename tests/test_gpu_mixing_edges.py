"""Paged and linear attention where they can go wrong: values that are not finite,
states updated in place, heads that many CTAs share, one workspace for all.

Tolerances are those of test_gpu_paged_attn and test_gpu_linear_attn; where the
oracle's value is infinite or NaN, so is the operator's.
"""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests import test_gpu_linear_attn as lin
from tests import test_gpu_paged_attn as att
from tests.test_gpu_linear_attn import BF16, F16, U, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def same_kind(got, want, tol):
    """Within tol where `want` is finite, otherwise the same infinity or NaN too."""
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert np.all(np.abs(got[fin] - want[fin]) <= tol[fin])


def check_any(dt, ref, o, state, T):
    ot = (3.1 * U[dt] + (T + 64) * 2.0 ** -22) * ref["o_abs"] + 2.0 ** -25
    st = (2.0 ** -16 + (T + 64) * 2.0 ** -22) * ref["state_abs"] + 2.0 ** -126
    same_kind(f64(o), ref["o"], ot)
    same_kind(f64(state), ref["state"], st)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [1, 20, 90, 300, 1500])
@pytest.mark.parametrize("where", ["value", "key", "state", "nan"])
def test_infinities_reach_what_the_formula_lets_them_reach(sdv, dt, T, where):
    # a token's infinity reaches its own and later outputs of its head, until a decay of
    # zero drops the state
    H = 2
    q, k, v, g, s = lin.make(dt, 1, T, H, H, 64, 128, 50)
    at, drop = T // 3, T // 3 + T // 4 + 1
    if where == "value":
        v[0, at, 1, 5] = float("inf")
    elif where == "nan":
        v[0, at, 1, 77] = float("nan")
    elif where == "key":
        k[0, at, 1, 9] = float("-inf")
    else:
        s[0, 1, 3, 8] = float("inf")
    if drop < T:
        g[0, drop, 1] = float("-inf")
    o, state = lin.call(sdv, q, k, v, g, None, s)
    with np.errstate(invalid="ignore"):
        ref = lin.oracle(q, k, v, g, None, s)
    assert np.isfinite(ref["o"][0, :, 0]).all() and (T == 1 or np.isfinite(ref["o"][0, drop:, 1]).all())
    with np.errstate(invalid="ignore"):
        check_any(dt, ref, o, state, T)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T,H", [(1, 2), (25, 2), (128, 3), (129, 1), (2000, 1), (1300, 5)])
@pytest.mark.parametrize("odd", [None, 0.1, 0.95])
def test_a_state_updated_in_place(sdv, dt, T, H, odd):
    q, k, v, g, s = lin.make(dt, 1, T, H, 1, 128, 64, 51)
    if odd is not None:
        v[0, int(odd * T), 0, 0] = float("inf")
    want_o, want = lin.call(sdv, q, k, v, g, None, s)
    for _ in range(3):
        state = s.clone()
        o, _ = lin.call(sdv, q, k, v, g, None, state, s_out=state)
        assert torch.equal(o.view(torch.int16), want_o.view(torch.int16))
        assert torch.equal(state.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("dt,B,T,H,hqk,dk,dv,n", [
    (F16, 3, 385, 60, 20, 64, 64, [385, 256, 130]),       # several heads in a CTA's share, and parts of two
    (BF16, 40, 140, 7, 7, 64, 64, [(37 * i) % 141 for i in range(40)]),
    (F16, 1, 4100, 1, 1, 64, 64, [4097]),                 # one chunk a CTA
    (BF16, 2, 257, 1, 1, 128, 128, [256, 257]),
    (F16, 2, 128, 2, 2, 128, 128, [128, 127])])
def test_shares_of_the_gpu(sdv, dt, B, T, H, hqk, dk, dv, n):
    q, k, v, g, s = lin.make(dt, B, T, H, hqk, dk, dv, 52, rate=0.02)
    o, state = lin.call(sdv, q, k, v, g, n, s)
    lin.check(dt, lin.oracle(q, k, v, g, n, s), o, state, T)
    again, state2 = lin.call(sdv, q, k, v, g, n, s)
    assert torch.equal(o, again) and torch.equal(state, state2)


def test_one_workspace_for_every_operation(sdv):
    # others leave anything behind the head of 256 bytes, which is zero between calls
    q, kp, vp, table = att.make(F16, 1, 1, 8, 1, 128, 64, [5003], [1], 53)
    lq, lk, lv, lg, ls = lin.make(F16, 2, 700, 2, 2, 128, 128, 54)
    want, _, _ = att.call(sdv, q, kp, vp, table, [5003], [1], None, 0.1)
    lin_o, lin_s = lin.call(sdv, lq, lk, lv, lg, None, ls)
    kp, vp, q, table = kp.cuda(), vp.cuda(), q.cuda(), table.cuda()
    size = max(sdv.paged_attn_workspace(q, kp, table).numel(), sdv.linear_attn_workspace(lk, lv).numel())
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    for _ in range(2):
        got, _, _ = att.call(sdv, q, kp, vp, table, [5003], [1], None, 0.1, ws=ws)
        assert torch.equal(got, want)
        o, s = torch.empty_like(lin_o), torch.empty_like(lin_s)
        sdv.sdv_linear_attn(lq, lk, lv, lg, 0.3, None, ls, s, o, ws)
        assert torch.equal(o, lin_o) and torch.equal(s, lin_s)
        torch.cuda.synchronize()
        assert not ws[:256].any()


@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,ctx,n", [
    (F16, 2, 1, 136, 1, 64, 16, [300, 4], [1, 1]),        # more query heads a cache head than a tile's rows
    (BF16, 1, 3, 128, 1, 128, 16, [900], [3]),            # exactly as many
    (F16, 1, 32, 5, 1, 128, 64, [640], [32]),             # 160 rows: a tile of 32 words cut
    (BF16, 2, 32, 65, 1, 64, 16, [129, 0], [32, 31]),
    (F16, 1, 4, 8, 2, 128, 512, [1000], [4]),
    # few rows, on both sides of 2048 elements of an output and of 32 rows
    (F16, 3, 2, 8, 2, 256, 64, [0, 63, 700], [2, 1, 2]),
    (BF16, 3, 3, 6, 2, 256, 32, [1, 64, 500], [3, 0, 3]),
    (F16, 2, 4, 8, 1, 128, 16, [126, 2000], [4, 4]),
    (BF16, 2, 17, 2, 2, 128, 16, [127, 400], [17, 9]),
    (F16, 2, 8, 8, 2, 64, 16, [300, 0], [8, 8]),
    (BF16, 2, 11, 3, 1, 64, 16, [300, 5], [11, 8])])
def test_rows_past_a_tile(sdv, dt, B, S, hq, hkv, d, page, ctx, n):
    q, kp, vp, table = att.make(dt, B, S, hq, hkv, d, page, ctx, n, 55)
    mask = att.words(np.random.default_rng(5), B, S)
    out, lse, ws = att.call(sdv, q, kp, vp, table, ctx, n, att.as_i32(mask), d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, mask, d ** -0.5)
    att.check(dt, ref, out, lse, d)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,S,page,ctx", [(256, 13, 64, 33), (128, 20, 16, 120), (64, 16, 32, 126)])
def test_infinite_values_in_windows_of_few_rows(sdv, dt, d, S, page, ctx):
    hq, hkv, j = 4, 2, 2
    q, kp, vp, table = att.make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 56)
    where = (table[0, (ctx + j) // page], slice(None), (ctx + j) % page)
    clean = vp.clone()
    v = vp[where].clone()
    v[..., 0], v[..., d - 1] = float("inf"), float("-inf")
    vp[where] = v
    out, lse, _ = att.call(sdv, q, kp, vp, table, [ctx], [S], None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(clean), table.tolist(), [ctx], [S], None, d ** -0.5)
    att.check(dt, {k: x[:, :j] for k, x in ref.items()}, out[:, :j], lse[:, :j], d)
    o = f64(out)[:, j:]
    assert np.all(np.isposinf(o[..., 0])) and np.all(np.isneginf(o[..., -1]))
    inner = {k: (x[:, j:, :, 1:-1] if x.ndim == 4 else x[:, j:]) for k, x in ref.items()}
    att.check(dt, inner, out[:, j:, :, 1:-1], lse[:, j:], d)
