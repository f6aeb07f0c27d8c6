"""sdv_paged_attn where values are infinite, NaN or close to the type's largest.

What is not finite among a position's values reaches every row that sees the
position, however small the row's weight of it is (a weight is above zero in the
formula, whatever it is in 32 bits), and no other: infinities of one sign give
that infinity, of both signs or with a NaN a NaN.  The other columns keep
test_gpu_paged_attn's tolerances, with the oracle's values of the odd places 0
(they have columns of their own).
"""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests import test_gpu_paged_attn as att
from tests.test_gpu_paged_attn import BF16, F16, f64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def check_odd(dt, ref, out, lse, d, odd, rows=slice(None)):
    """Columns `odd` {column: value} hold that value in every row, the others the oracle's."""
    got = f64(out)
    for c, want in odd.items():
        assert np.array_equal(got[:, rows, :, c], np.full_like(got[:, rows, :, c], want), equal_nan=True), (c, want)
    kept = [c for c in range(d) if c not in odd]
    part = {k: (x[:, rows][..., kept] if x.ndim == 4 else x[:, rows]) for k, x in ref.items()}
    att.check(dt, part, out[:, rows][..., kept], lse[:, rows], d)


# (d, page, S, heads, cache heads, ctx): one token and more rows, rows that stand four times in a
# tile and rows that do not, units in one share and in many, the CUDA-core form
FORMS = [(128, 16, 1, 8, 2, 613), (128, 16, 1, 1, 1, 3), (64, 64, 1, 8, 1, 200), (256, 32, 1, 8, 1, 130),
         (128, 64, 1, 8, 1, 30011), (128, 16, 4, 8, 2, 613), (64, 16, 16, 4, 2, 126), (256, 64, 13, 4, 2, 300),
         (128, 16, 20, 8, 2, 5003), (256, 64, 17, 16, 2, 777), (128, 16, 32, 16, 1, 3000),
         (40, 16, 3, 4, 2, 500), (128, 12, 1, 4, 1, 900), (248, 20, 5, 4, 2, 4001)]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_odd_values_of_the_context_reach_every_row(sdv, dt, form):
    d, page, S, hq, hkv, ctx = FORMS[form]
    q, kp, vp, table = att.make(dt, 2, S, hq, hkv, d, page, [ctx, ctx // 2], [S, S], 60 + form)
    clean = vp.clone()
    at = lambda b, p, c: (int(table[b, p // page]), hkv - 1, p % page, c)  # noqa: E731
    first, mid, last = 0, ctx // 3, ctx - 1
    odd = {0: INF, 9: -INF, 18: NAN, 27: NAN, d - 1: INF}
    for p, c, x in ((mid, 0, INF), (first, 9, -INF), (last, 18, NAN), (first, 27, INF), (last, 27, -INF),
                    (last, d - 1, INF), (mid, d - 1, INF)):
        vp[at(0, p, c)] = x
        clean[at(0, p, c)] = 0.0
    out, lse, ws = att.call(sdv, q, kp, vp, table, [ctx, ctx // 2], [S, S], None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    ref = mixing.attention(f64(q), f64(kp), f64(clean), table.tolist(), [ctx, ctx // 2], [S, S], None, d ** -0.5)
    own = hq // hkv * (hkv - 1)  # the query heads of the cache head that holds them
    pick = lambda b, h: {k: x[b:b + 1, :, h] for k, x in ref.items()}  # noqa: E731
    check_odd(dt, pick(0, slice(own, None)), out[:1, :, own:], lse[:1, :, own:], d, odd)
    if own:
        att.check(dt, pick(0, slice(0, own)), out[:1, :, :own], lse[:1, :, :own], d)
    att.check(dt, pick(1, slice(None)), out[1:], lse[1:], d)
    again, _, _ = att.call(sdv, q, kp, vp, table, [ctx, ctx // 2], [S, S], None, d ** -0.5, ws=ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,page,S,hq,hkv,ctx", [
    (128, 16, 1, 8, 1, 100), (128, 16, 1, 8, 1, 9000), (64, 16, 5, 4, 2, 400), (256, 64, 17, 16, 2, 777),
    (128, 16, 20, 8, 1, 5003), (40, 16, 3, 4, 2, 500), (128, 12, 2, 4, 2, 3000)])
@pytest.mark.parametrize("where", ["before", "behind"])
def test_odd_values_of_positions_with_hardly_any_weight(sdv, dt, d, page, S, hq, hkv, ctx, where):
    # scores of one half lie 400 below the other's: its weights are 0 in 32 bits
    q, kp, vp, table = att.make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 90)
    q[...] = 1.0
    high = 20.0 / d ** 0.5
    low = [p for p in range(ctx) if (p < ctx // 2) == (where == "before")]
    faint = set(low)
    for p in range(ctx + S):
        kp[table[0, p // page], :, p % page] = -high * 19 if p in faint else high
    clean = vp.clone()
    for p, c, x in ((low[0], 0, INF), (low[-1], 1, -INF), (low[len(low) // 2], 2, NAN)):
        vp[table[0, p // page], :, p % page, c] = x
        clean[table[0, p // page], :, p % page, c] = 0.0
    out, lse, _ = att.call(sdv, q, kp, vp, table, [ctx], [S], None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(clean), table.tolist(), [ctx], [S], None, d ** -0.5)
    check_odd(dt, ref, out, lse, d, {0: INF, 1: -INF, 2: NAN})


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,page,S,hq,hkv,ctx", [(128, 16, 5, 8, 2, 300), (256, 64, 17, 16, 2, 777),
                                                 (64, 32, 20, 8, 2, 126), (40, 16, 6, 4, 2, 77)])
def test_odd_values_of_the_context_and_of_the_window(sdv, dt, d, page, S, hq, hkv, ctx):
    # the rows before the window position see the context's alone
    q, kp, vp, table = att.make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 91)
    clean, j = vp.clone(), 2
    for p, c, x in ((5, 0, INF), (ctx + j, 0, -INF), (7, 1, -INF), (ctx + j, 1, -INF), (ctx + j, 2, INF)):
        vp[table[0, p // page], :, p % page, c] = x
        clean[table[0, p // page], :, p % page, c] = 0.0
    out, lse, _ = att.call(sdv, q, kp, vp, table, [ctx], [S], None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(clean), table.tolist(), [ctx], [S], None, d ** -0.5)
    check_odd(dt, ref, out, lse, d, {0: INF, 1: -INF}, slice(0, j))
    check_odd(dt, ref, out, lse, d, {0: NAN, 1: -INF, 2: INF}, slice(j, None))


@pytest.mark.parametrize("d,page,S,hq,hkv,ctx", [(128, 16, 1, 8, 2, 613), (64, 16, 5, 8, 2, 300), (256, 64, 17, 16, 2, 777),
                                                 (128, 64, 1, 8, 1, 9000), (40, 16, 3, 4, 2, 500)])
@pytest.mark.parametrize("std", [0.0, 1.7])
def test_values_close_to_the_largest_of_the_type(sdv, d, page, S, hq, hkv, ctx, std):
    # a mean of values is no larger than they are: 2^120 in bf16 stays finite
    q, kp, vp, table = att.make(BF16, 1, S, hq, hkv, d, page, [ctx], [S], 92, std=std)
    vp = (vp.float() * 2.0 ** 116).to(BF16)
    out, lse, _ = att.call(sdv, q, kp, vp, table, [ctx], [S], None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), [ctx], [S], None, d ** -0.5)
    att.check(BF16, ref, out, lse, d)
