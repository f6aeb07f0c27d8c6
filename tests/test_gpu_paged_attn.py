"""sdv_kv_append and sdv_paged_attn on the GPU against the 64-bit oracle.

Tolerances, from the operation alone (u: unit roundoff of the 16-bit type):
weights may be rounded to the type before their product with the values (u per
weight), the result is rounded once (u), scores carry the fp32 error of a
dim-long dot product (delta, from the row's sum |q k|), sums run in fp32:
  |out - ref| <= (2.1 u + 2 delta + (count + 16) 2^-23) sum p|v| + 2^-24 sum|v|
(the last term: weights below the type's normal range), plus half the smallest
subnormal of the output.  lse: delta + (count + 16) 2^-23 + 2^-20 + |lse| 2^-22.
"""
import numpy as np
import pytest
import torch

from oracle import mixing

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def f64(t):
    return t.detach().cpu().double().numpy()


def make(dt, B, S, hq, hkv, d, page, ctx, n, seed, std=1.7, spare=3):
    """A cache of randomly placed pages with NaN in every slot no sequence uses."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-(c + r) // page) for c, r in zip(ctx, n)]
    pages, width = sum(need) + spare, max(max(need), 1)
    ids = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    kp = torch.full((pages, hkv, page, d), float("nan"), dtype=dt)
    vp = kp.clone()
    at = 0
    for b in range(B):
        for j in range(need[b]):
            table[b, j] = ids[at]
            used = min(page, ctx[b] + n[b] - j * page)
            kp[ids[at], :, :used] = torch.randn((hkv, used, d), generator=gen).to(dt)
            vp[ids[at], :, :used] = torch.randn((hkv, used, d), generator=gen).to(dt)
            at += 1
    q = (torch.randn((B, S, hq, d), generator=gen) * std).to(dt)
    return q, kp, vp, table


def call(sdv, q, kp, vp, table, ctx, n, mask, scale, want_lse=True, stream=None, ws=None):
    dev = lambda x: None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, kp, vp, table = (x if x.is_cuda else x.cuda() for x in (q, kp, vp, table))
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda") if want_lse else None
    ws = sdv.paged_attn_workspace(q, kp, table) if ws is None else ws
    sdv.sdv_paged_attn(q, kp, vp, table, dev(ctx), dev(n), dev(mask), scale, out, lse, ws, stream)
    return out, lse, ws


def check(dt, ref, out, lse, d):
    u = U[dt]
    delta = (d + 4) * 2.0 ** -24 * ref["dot"]
    sums = (ref["count"] + 16) * 2.0 ** -23
    tol = (2.1 * u + 2 * delta + sums)[..., None] * ref["weight"] + 2.0 ** -24 * ref["total"] + 2.0 ** -25
    err = np.abs(f64(out) - ref["out"])
    assert np.all(err <= tol), f"out: worst {np.max(err / tol):.3f} of the bound"
    if lse is None:
        return
    got = f64(lse)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(got), empty)
    assert not f64(out)[empty].any()
    lt = delta + sums + 2.0 ** -20 + np.abs(np.where(empty, 0.0, ref["lse"])) * 2.0 ** -22
    le = np.abs(np.where(empty, 0.0, got) - np.where(empty, 0.0, ref["lse"]))
    assert np.all(le <= lt), f"lse: worst {np.max(le / lt):.3f} of the bound"


def words(rng, B, S):
    """Random visibility words, some empty, bits past the window set at random."""
    w = rng.integers(0, 2 ** 32, (B, S), dtype=np.uint64)
    w[rng.random((B, S)) < 0.2] = 0
    return w


def as_i32(w):
    return np.asarray(w, dtype=np.uint64).astype(np.uint32).view(np.int32)


SHAPES = [
    # dtype, B, S, Hq, Hkv, D, page, ctx, n, mask
    (F16, 1, 1, 1, 1, 128, 16, [0], [1], False),              # one token, no context
    (F16, 1, 1, 8, 2, 128, 16, [613], [1], False),
    (BF16, 4, 1, 8, 2, 128, 16, [126, 127, 128, 129], [1] * 4, False),
    (BF16, 5, 1, 4, 4, 64, 64, [0, 63, 64, 255, 511], [1] * 5, False),
    (F16, 3, 1, 6, 1, 256, 32, [62, 63, 700], [1] * 3, False),
    (F16, 1, 17, 16, 2, 256, 64, [777], [17], False),         # 136 rows of a kv head
    (BF16, 1, 32, 16, 2, 128, 128, [300], [32], True),        # 256 rows
    (F16, 2, 32, 4, 4, 64, 16, [0, 100], [32, 32], True),
    (BF16, 3, 9, 12, 2, 128, 8, [5, 119, 250], [9, 9, 9], False),
    (F16, 4, 13, 6, 2, 128, 256, [0, 243, 244, 513], [13, 0, 12, 1], True),
    (BF16, 2, 31, 2, 2, 256, 128, [97, 0], [31, 30], True),
    (F16, 40, 1, 4, 2, 64, 16, [7 * i % 97 for i in range(40)], [1] * 40, False),
    (BF16, 35, 3, 4, 1, 128, 32, [31 * i % 211 for i in range(35)], [i % 4 for i in range(35)], True),
    (F16, 1, 1, 8, 1, 128, 64, [5003], [1], False),           # split over the GPU and joined
    (BF16, 1, 8, 32, 4, 128, 16, [2999], [8], True),
    (F16, 1, 2, 8, 8, 256, 16, [1500], [2], False),
    # head and page sizes outside the tensor-core kernel's
    (F16, 2, 3, 4, 2, 40, 16, [33, 500], [3, 2], True),
    (BF16, 2, 1, 4, 1, 8, 5, [0, 77], [1, 1], False),
    (F16, 2, 5, 4, 2, 128, 1, [70, 3], [5, 5], False),
    (BF16, 1, 20, 4, 1, 96, 48, [400], [20], True),
    (F16, 2, 4, 2, 2, 248, 20, [39, 41], [4, 4], True),
    (BF16, 1, 7, 8, 2, 256, 48, [95], [7], False),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention_matches_the_oracle(sdv, case):
    dt, B, S, hq, hkv, d, page, ctx, n, masked = SHAPES[case]
    q, kp, vp, table = make(dt, B, S, hq, hkv, d, page, ctx, n, 100 + case)
    mask = words(np.random.default_rng(case), B, S) if masked else None
    scale = d ** -0.5
    out, lse, ws = call(sdv, q, kp, vp, table, ctx, n, None if mask is None else as_i32(mask), scale)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, mask, scale)
    check(dt, ref, out, lse, d)
    # the same call again, and without lse: the same bits
    out2, _, _ = call(sdv, q, kp, vp, table, ctx, n, None if mask is None else as_i32(mask), scale, want_lse=False, ws=ws)
    assert torch.equal(out2, out)
    # n_rows left out means full windows
    if all(r == S for r in n):
        out3, _, _ = call(sdv, q, kp, vp, table, ctx, None, None if mask is None else as_i32(mask), scale)
        assert torch.equal(out3, out)


@pytest.mark.parametrize("dt,B,S,hq,hkv,d,most", [
    (F16, 64, 1, 16, 8, 64, 400), (BF16, 48, 1, 16, 8, 128, 300), (F16, 30, 5, 12, 6, 256, 200),
    (BF16, 20, 32, 20, 4, 128, 150)])
def test_many_sequences_per_cta(sdv, dt, B, S, hq, hkv, d, most):
    # several units in a CTA's share, of one tile and of more
    rng = np.random.default_rng(B)
    ctx, n = [int(x) for x in rng.integers(0, most, B)], [int(x) for x in rng.integers(0, S + 1, B)]
    q, kp, vp, table = make(dt, B, S, hq, hkv, d, 16, ctx, n, B)
    mask = words(rng, B, S) if S > 1 else None
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, mask, d ** -0.5)
    first = None
    for _ in range(5):
        out, lse, ws = call(sdv, q, kp, vp, table, ctx, n, None if mask is None else as_i32(mask), d ** -0.5)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        first = out if first is None else first
        assert torch.equal(out, first)
    check(dt, ref, out, lse, d)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("std", [0.0, 1e-3, 60.0])
def test_flat_and_sharp_softmax(sdv, dt, std):
    ctx, n, d = [1029, 400], [5, 5], 128
    q, kp, vp, table = make(dt, 2, 5, 8, 2, d, 16, ctx, n, 7, std=std)
    out, lse, _ = call(sdv, q, kp, vp, table, ctx, n, None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, None, d ** -0.5)
    check(dt, ref, out, lse, d)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256, 48])
@pytest.mark.parametrize("scale", [0.0, -0.11, 1e-30, -3.0])
def test_scales_of_any_sign(sdv, dt, d, scale):
    ctx, n = [300], [4]
    q, kp, vp, table = make(dt, 1, 4, 4, 2, d, 16, ctx, n, 15)
    out, lse, _ = call(sdv, q, kp, vp, table, ctx, n, None, scale)
    ref = mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, None, scale)
    check(dt, ref, out, lse, d)


@pytest.mark.parametrize("d,page", [(128, 16), (64, 64), (256, 32), (40, 16), (128, 12)])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_scores_that_rise_or_fall_along_the_cache(sdv, d, page, order):
    # the running maximum moves at every tile, or never again after the first
    ctx, n = [1900], [3]
    q, kp, vp, table = make(F16, 1, 3, 4, 2, d, page, ctx, n, 8)
    L = ctx[0] + n[0]
    q[...] = 1.0
    for p in range(L):
        x = (p if order == "rising" else L - p) / L * 60.0 / d ** 0.5 - 2.0
        kp[table[0, p // page], :, p % page] = x
    out, lse, _ = call(sdv, q, kp, vp, table, ctx, n, None, d ** -0.5)
    check(F16, mixing.attention(f64(q), f64(kp), f64(vp), table.tolist(), ctx, n, None, d ** -0.5), out, lse, d)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,page,ctx", [(128, 16, 0), (128, 16, 120), (256, 64, 33), (64, 32, 127), (40, 16, 29)])
def test_unseen_positions_may_hold_anything(sdv, dt, d, page, ctx):
    # window position 1 holds infinities and NaN, position 3 the type's largest
    # values: rows that do not see them are the same as if they were zero
    S, hq, hkv = 6, 4, 2
    q, kp, vp, table = make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 9)
    mask = np.array([[0b000001, 0b000011, 0b000101, 0b001101, 0b010101, 0b100000]], dtype=np.uint64)
    at = lambda j: (table[0, (ctx + j) // page], slice(None), (ctx + j) % page)  # noqa: E731
    clean_k, clean_v = kp.clone(), vp.clone()
    for j in (1, 3):
        clean_k[at(j)] = 0
        clean_v[at(j)] = 0
    kp[at(1)] = float("nan")
    vp[at(1)] = float("inf")
    vp[at(1)][..., ::3] = float("nan")
    kp[at(3)] = torch.finfo(dt).max
    vp[at(3)] = torch.finfo(dt).min
    out, lse, _ = call(sdv, q, kp, vp, table, [ctx], [S], as_i32(mask), d ** -0.5)
    ref = mixing.attention(f64(q), f64(clean_k), f64(clean_v), table.tolist(), [ctx], [S], mask, d ** -0.5)
    rows = [0, 2, 4, 5]
    check(dt, {k: v[:, rows] for k, v in ref.items()}, out[:, rows], lse[:, rows], d)
    assert torch.isnan(out[:, 1].float()).any() and torch.isnan(lse[:, 1]).all()


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,page,ctx", [(128, 16, 0), (128, 16, 300), (256, 64, 33), (64, 32, 126), (40, 16, 29)])
def test_infinite_values_reach_the_rows_that_see_them_alone(sdv, dt, d, page, ctx):
    S, hq, hkv = 5, 4, 2
    q, kp, vp, table = make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 10)
    j, cols = 2, [0, d - 1]
    where = (table[0, (ctx + j) // page], slice(None), (ctx + j) % page)
    ref_v = vp.clone()
    v = vp[where].clone()
    v[..., cols[0]], v[..., cols[1]] = float("inf"), float("-inf")
    vp[where] = v
    out, lse, _ = call(sdv, q, kp, vp, table, [ctx], [S], None, d ** -0.5)
    ref = mixing.attention(f64(q), f64(kp), f64(ref_v), table.tolist(), [ctx], [S], None, d ** -0.5)
    check(dt, {k: v[:, :2] for k, v in ref.items()}, out[:, :2], lse[:, :2], d)
    o = f64(out)[:, 2:]
    assert np.all(np.isposinf(o[..., 0])) and np.all(np.isneginf(o[..., -1]))
    finite = {k: (v[:, 2:, :, 1:-1] if v.ndim == 4 else v[:, 2:]) for k, v in ref.items()}
    check(dt, finite, out[:, 2:, :, 1:-1], lse[:, 2:], d)


def test_rows_of_a_fused_projection_and_another_stream(sdv):
    B, S, hq, hkv, d, page = 2, 4, 8, 2, 128, 16
    ctx, n = [50, 131], [4, 3]
    q, kp, vp, table = make(F16, B, S, hq, hkv, d, page, ctx, n, 11)
    want, _, _ = call(sdv, q, kp, vp, table, ctx, n, None, 0.1)
    fused = torch.full((B, S, (hq + 2 * hkv) * d), float("nan"), dtype=F16, device="cuda")
    fused[..., :hq * d] = q.cuda().reshape(B, S, -1)
    view = fused[..., :hq * d].view(B, S, hq, d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, _, _ = call(sdv, view, kp.cuda(), vp.cuda(), table.cuda(), ctx, n, None, 0.1)
        s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("d,page", [(128, 16), (40, 16)])
def test_bad_tables_and_lengths_are_reported(sdv, d, page):
    ctx, n = [40, 20], [2, 2]
    q, kp, vp, table = make(F16, 2, 2, 2, 1, d, page, ctx, n, 12)
    good, _, ws = call(sdv, q, kp, vp, table, ctx, n, None, 0.1)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    for entry in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[0, 1] = entry
        out, _, _ = call(sdv, q, kp, vp, bad, ctx, n, None, 0.1, ws=ws)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        assert torch.equal(out[1], good[1])  # the other sequence is untouched
        # positions 16 .. 31 are absent: the same as a cache without them
        keep = [p for p in range(42) if p // page != 1]
        pos = f64(kp)[table[0].tolist()].transpose(0, 2, 1, 3).reshape(-1, d)[keep]
        val = f64(vp)[table[0].tolist()].transpose(0, 2, 1, 3).reshape(-1, d)[keep]
        s = pos @ f64(q)[0, 1].T * 0.1
        w = np.exp(s - s.max(0))
        ref = (w / w.sum(0)).T @ val
        np.testing.assert_allclose(f64(out)[0, 1], ref, atol=4e-3)
    # a context longer than the table holds, and a negative one
    for c in (table.shape[1] * page + 1, 2 ** 31 - 1, -5):
        call(sdv, q, kp, vp, torch.zeros_like(table), [c, ctx[1]], n, None, 0.1, ws=ws)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [128, 24])
def test_offsets_past_32_bits(sdv, d):
    # a cache of more than 2^32 elements a tensor; the sequence lives in its last pages
    page, hkv = 256, 8
    pages = 2 ** 32 // (page * hkv * d) + 40
    q, kp, vp, table = make(BF16, 1, 3, 8, hkv, d, page, [900], [3], 13)
    big = [torch.empty((pages, hkv, page, d), dtype=BF16, device="cuda") for _ in range(2)]
    ids = table[0].long()
    moved = (pages - 1 - torch.arange(len(ids))).to(torch.int32)
    for x, src in zip(big, (kp, vp)):
        x[moved.long().cuda()] = src[ids].cuda()
    want, _, _ = call(sdv, q, kp, vp, table, [900], [3], None, 0.1)
    got, _, ws = call(sdv, q, big[0], big[1], moved[None], [900], [3], None, 0.1)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    assert torch.equal(got, want)
    # and the append reaches them
    rows = torch.randn((1, 3, hkv, d)).to(BF16).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    sdv.sdv_kv_append(rows, rows, big[0], big[1], moved[None].cuda(), i32([510]), None, None)
    for t, p in enumerate((510, 511, 512)):
        assert torch.equal(big[1][int(moved[p // page]), :, p % page], rows[0, t])
    del big
    torch.cuda.empty_cache()


# ---- append ----------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("B,T,hkv,d,page,ctx,n", [
    (1, 1, 8, 128, 16, [15], None), (1, 1, 1, 8, 1, [0], None), (3, 17, 2, 64, 16, [0, 15, 100], [17, 0, 5]),
    (2, 300, 4, 128, 32, [3, 250], [300, 299]), (4, 9, 3, 40, 7, [1, 2, 3, 4], [9, 8, 1, 0]),
    (2, 33, 2, 256, 128, [127, 128], None)])
def test_append(sdv, dt, B, T, hkv, d, page, ctx, n):
    live = n or [T] * B
    _, kp, vp, table = make(dt, B, 1, hkv, hkv, d, page, ctx, live, 20)
    kv = torch.randn((B, T, 2 * hkv + 1, d)).to(dt).cuda()
    k, v = kv[:, :, :hkv], kv[:, :, hkv:2 * hkv]  # slices of a fused projection
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gk, gv = kp.cuda(), vp.cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sdv.sdv_kv_append(k, v, gk, gv, table.cuda(), i32(ctx), None if n is None else i32(n), ws)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    for got, before, rows in ((gk, kp, k), (gv, vp, v)):
        want = mixing.append(f64(before), f64(rows), table.tolist(), ctx, live)
        np.testing.assert_array_equal(f64(got), want)


def test_append_leaves_the_cache_alone_outside_its_table(sdv):
    _, kp, vp, table = make(F16, 2, 1, 2, 2, 64, 16, [20, 20], [4, 4], 21)
    rows = torch.ones((2, 30, 2, 64), dtype=F16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for ctx, bad in (([20, 20], None), ([-3, 0], None), ([2 ** 31 - 5, 0], None), ([0, 0], kp.shape[0]), ([0, 0], -7)):
        gk, gv, t = kp.cuda(), vp.cuda(), table.clone()
        if bad is not None:
            t[0, 1] = bad
        sdv.sdv_kv_append(rows, rows, gk, gv, t.cuda(), i32(ctx), None, ws)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        want = f64(kp)
        for b in range(2):
            for j in range(30):
                p = ctx[b] + j
                if 0 <= p < 32 and 0 <= int(t[b, p // 16]) < kp.shape[0]:
                    want[int(t[b, p // 16]), :, p % 16] = 1.0
        np.testing.assert_array_equal(f64(gk), want)
    sdv.sdv_kv_append(rows, rows, kp.cuda(), vp.cuda(), table.cuda(), i32([20, 20]), None, None)  # unrecorded


def test_append_then_attend_equals_a_cache_built_at_once(sdv):
    B, S, hq, hkv, d, page, ctx = 2, 6, 8, 2, 128, 16, [30, 77]
    n = [6, 4]
    q, kp, vp, table = make(BF16, B, S, hq, hkv, d, page, ctx, n, 22)
    k, v = torch.zeros((B, S, hkv, d), dtype=BF16), torch.zeros((B, S, hkv, d), dtype=BF16)
    ek, ev = kp.clone(), vp.clone()
    for b in range(B):
        for t in range(n[b]):
            p = ctx[b] + t
            k[b, t], v[b, t] = kp[table[b, p // page], :, p % page], vp[table[b, p // page], :, p % page]
            ek[table[b, p // page], :, p % page] = float("inf")
            ev[table[b, p // page], :, p % page] = float("inf")
    want, _, _ = call(sdv, q, kp, vp, table, ctx, n, None, 0.09)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gk, gv = ek.cuda(), ev.cuda()
    sdv.sdv_kv_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), i32(ctx), i32(n), None)
    got, _, _ = call(sdv, q, gk, gv, table, ctx, n, None, 0.09)
    assert torch.equal(got, want)
