"""sdv_prefix_attn on the GPU against the 64-bit oracle: attention over a shared prefix and each
sequence's own positions is attention over both.

Tolerances as for sdv_paged_attn (tests/test_gpu_paged_attn.py): from the operation alone, with
one merge more of the same kind.
"""
import numpy as np
import pytest
import torch

from oracle import rounds
from tests.test_gpu_paged_attn import as_i32, check, f64, words

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, seed, std=1.7):
    """A cache of randomly placed pages with NaN in every slot that nothing uses."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-(c + r) // page) for c, r in zip(ctx, n)]
    front = -(-prefix // page)
    pages, width = sum(need) + front + 3, max(max(need), 1)
    ids = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    ptable = torch.tensor(ids[:front] + [-1], dtype=torch.int32)
    kp = torch.full((pages, hkv, page, d), float("nan"), dtype=dt)
    vp = kp.clone()
    at = front

    def fill(page_id, used):
        for x in (kp, vp):
            x[page_id, :, :used] = torch.randn((hkv, used, d), generator=gen).to(dt)

    for j in range(front):
        fill(ids[j], min(page, prefix - j * page))
    for b in range(B):
        for j in range(need[b]):
            table[b, j] = ids[at]
            fill(ids[at], min(page, ctx[b] + n[b] - j * page))
            at += 1
    q = (torch.randn((B, S, hq, d), generator=gen) * std).to(dt)
    return q, kp, vp, ptable, table


def dev(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()


def call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, mask, scale, want_lse=True, ws=None, stream=None):
    q, kp, vp, ptable, table = (x if x.is_cuda else x.cuda() for x in (q, kp, vp, ptable, table))
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda") if want_lse else None
    ws = sdv.prefix_attn_workspace(q, kp, table) if ws is None else ws
    sdv.sdv_prefix_attn(q, kp, vp, ptable, dev([prefix]), table, dev(ctx), dev(n), dev(mask), scale, out, lse, ws,
                        stream)
    return out, lse, ws


def reference(q, kp, vp, ptable, prefix, table, ctx, n, mask, scale):
    return rounds.prefix_attention(f64(q), f64(kp), f64(vp), ptable.tolist(), prefix, table.tolist(), ctx, n, mask,
                                   scale)


SHAPES = [
    # dtype, B, S, Hq, Hkv, D, page, prefix, ctx, n, mask
    (F16, 1, 1, 1, 1, 128, 16, 1, [0], [1], False),
    (F16, 2, 1, 8, 2, 128, 16, 129, [0, 5], [1, 1], False),
    (BF16, 3, 1, 8, 2, 128, 16, 1000, [17, 0, 300], [1, 1, 1], False),
    (BF16, 5, 1, 4, 4, 64, 64, 127, [0, 63, 64, 255, 511], [1] * 5, False),
    (F16, 3, 1, 6, 1, 256, 32, 64, [62, 63, 700], [1] * 3, False),
    (F16, 4, 9, 16, 2, 256, 64, 801, [7, 0, 90, 33], [9, 6, 3, 9], True),
    (BF16, 40, 5, 8, 2, 128, 32, 640, [3 * i for i in range(40)], [5] * 40, False),   # 800 rows of a kv head
    (F16, 33, 1, 28, 4, 128, 8, 300, [i for i in range(33)], [1] * 33, False),        # a group of 7
    (BF16, 20, 32, 4, 1, 64, 16, 333, [i * 7 for i in range(20)], [32 - i for i in range(20)], True),
    (F16, 70, 1, 64, 1, 128, 128, 500, [0] * 70, [1] * 70, False),                    # rows of 64 heads
    (F16, 2, 2, 128, 1, 128, 16, 200, [0, 9], [2, 1], False),                         # a token a row tile
    (BF16, 6, 4, 24, 8, 64, 16, 15, [0] * 6, [4, 0, 1, 2, 3, 4], True),
    (BF16, 2, 3, 8, 2, 128, 16, 0, [40, 0], [3, 3], False),                           # no prefix
    (F16, 1, 1, 8, 1, 128, 64, 5003, [3], [1], False),
    (BF16, 9, 2, 8, 8, 256, 16, 1500, [1] * 9, [2] * 9, False),
    # head and page sizes outside the tensor-core kernel's, a group of more than 128
    (F16, 2, 3, 4, 2, 40, 16, 100, [33, 200], [3, 2], True),
    (BF16, 2, 1, 4, 1, 8, 5, 33, [0, 77], [1, 1], False),
    (F16, 3, 5, 4, 2, 128, 1, 70, [30, 3, 0], [5, 5, 5], False),
    (BF16, 4, 6, 4, 1, 96, 48, 400, [40, 0, 1, 2], [6] * 4, True),
    (F16, 2, 2, 2, 2, 248, 20, 61, [39, 41], [2, 2], True),
    (F16, 1, 2, 130, 1, 64, 16, 70, [5], [2], False),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_matches_the_oracle(sdv, case):
    dt, B, S, hq, hkv, d, page, prefix, ctx, n, masked = SHAPES[case]
    q, kp, vp, ptable, table = make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, 300 + case)
    mask = words(np.random.default_rng(case), B, S) if masked else None
    im = None if mask is None else as_i32(mask)
    scale = d ** -0.5
    out, lse, ws = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, im, scale)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    ref = reference(q, kp, vp, ptable, prefix, table, ctx, n, mask, scale)
    check(dt, ref, out, lse, d)
    # the same call again, and without lse: the same bits
    out2, _, _ = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, im, scale, want_lse=False, ws=ws)
    assert torch.equal(out2, out)


@pytest.mark.parametrize("d,page", [(128, 16), (256, 16), (64, 128), (96, 16)])
def test_every_length_around_a_tile(sdv, d, page):
    B, S, hq, hkv = 3, 2, 4, 1
    for prefix in (1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257):
        ctx, n = [0, 1, 30], [2, 1, 2]
        q, kp, vp, ptable, table = make(F16, B, S, hq, hkv, d, page, prefix, ctx, n, prefix)
        out, lse, _ = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, None, 0.2)
        check(F16, reference(q, kp, vp, ptable, prefix, table, ctx, n, None, 0.2), out, lse, d)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(sdv, scale):
    ctx, n = [20, 3], [2, 2]
    q, kp, vp, ptable, table = make(BF16, 2, 2, 8, 2, 128, 16, 300, ctx, n, 7, std=1.0)
    out, lse, _ = call(sdv, q, kp, vp, ptable, 300, table, ctx, n, None, scale)
    check(BF16, reference(q, kp, vp, ptable, 300, table, ctx, n, None, scale), out, lse, 128)


@pytest.mark.parametrize("d", [64, 128, 256, 96])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_infinities_and_nan_of_seen_values_arrive(sdv, dt, d):
    """Every live row sees the whole prefix: what is not finite there reaches all of them, in
    its column, however small its weight; the rows of dead windows stay 0."""
    ctx, n = [20, 3, 0], [2, 1, 0]
    q, kp, vp, ptable, table = make(dt, 3, 2, 8, 2, d, 16, 400, ctx, n, 8, std=20.0)
    at = lambda p: (int(ptable[p // 16]), p % 16)  # noqa: E731
    for p, h, c, x in ((3, 0, 1, float("inf")), (390, 0, 5, float("nan")), (140, 1, 7, float("-inf")),
                       (5, 1, 9, float("inf")), (391, 1, 9, float("-inf"))):
        page, slot = at(p)
        vp[page, h, slot, c] = x
    out, lse, _ = call(sdv, q, kp, vp, ptable, 400, table, ctx, n, None, d ** -0.5)
    out = out.float().cpu()
    for b, i in ((0, 0), (0, 1), (1, 0)):
        for h in range(8):
            row = out[b, i, h]
            odd = {1: float("inf"), 5: float("nan")} if h < 4 else {7: float("-inf"), 9: float("nan")}
            for c in range(d):
                if c not in odd:
                    assert torch.isfinite(row[c])
                elif odd[c] != odd[c]:
                    assert torch.isnan(row[c])
                else:
                    assert row[c] == odd[c]
    assert not out[1, 1].any() and not out[2].any()


def test_large_values_do_not_overflow(sdv):
    """bf16 values near the type's largest, weights spread over many positions."""
    ctx, n = [20, 3], [1, 1]
    q, kp, vp, ptable, table = make(BF16, 2, 1, 8, 2, 128, 16, 700, ctx, n, 9, std=0.1)
    vp = torch.where(torch.isnan(vp), vp, torch.full_like(vp, 2.0 ** 127))
    out, _, _ = call(sdv, q, kp, vp, ptable, 700, table, ctx, n, None, 0.1)
    assert torch.all((out.float() / 2.0 ** 127 - 1.0).abs() <= 2.0 ** -6)


def test_absent_pages_and_lengths_out_of_range(sdv):
    """Positions behind an entry that is not a page are absent, and reported, lengths clamped."""
    ctx, n = [20, 3], [2, 2]
    for d in (128, 96):
        q, kp, vp, ptable, table = make(F16, 2, 2, 8, 2, d, 16, 320, ctx, n, 10)
        bad = ptable.clone()
        bad[5], bad[19] = -1, kp.shape[0]
        out, lse, ws = call(sdv, q, kp, vp, bad, 320, table, ctx, n, None, 0.1)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        keep = torch.cat([ptable[:5], ptable[6:19]])
        ref = reference(q, kp, vp, keep, 288, table, ctx, n, None, 0.1)
        check(F16, ref, out, lse, d)
        # the table names 21 pages, the last of which is none: 336 positions at most
        out, lse, ws = call(sdv, q, kp, vp, ptable, 5000, table, ctx, n, None, 0.1)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        check(F16, reference(q, kp, vp, ptable, 320, table, ctx, n, None, 0.1), out, lse, d)
        out, lse, ws = call(sdv, q, kp, vp, ptable, -3, table, ctx, n, None, 0.1)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        check(F16, reference(q, kp, vp, ptable, 0, table, ctx, n, None, 0.1), out, lse, d)


def test_queries_of_a_fused_projection_and_nan_of_dead_rows(sdv):
    ctx, n = [20, 3, 0], [2, 1, 0]
    q, kp, vp, ptable, table = make(F16, 3, 2, 8, 2, 128, 16, 400, ctx, n, 11)
    want, wl, _ = call(sdv, q, kp, vp, ptable, 400, table, ctx, n, None, 0.1)
    wide = torch.full((3, 2, 14, 128), float("nan"), dtype=F16, device="cuda")
    wide[:, :, 3:11] = q.cuda()
    wide[1, 1], wide[2] = float("nan"), float("inf")
    out, lse, _ = call(sdv, wide[:, :, 3:11], kp, vp, ptable, 400, table, ctx, n, None, 0.1)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_one_workspace_captured_and_shared(sdv):
    """Two captured calls of other shapes on one workspace, replayed in turn; the same bits."""
    calls = []
    for dt, B, S, d, prefix, seed in ((F16, 3, 2, 128, 500, 1), (BF16, 30, 3, 64, 1000, 2), (F16, 2, 2, 96, 90, 3)):
        ctx, n = [5 * i for i in range(B)], [S] * B
        made = make(dt, B, S, 8, 2, d, 16, prefix, ctx, n, seed)
        made = [x.cuda() for x in made]
        calls.append((made, prefix, ctx, n, call(sdv, *made[:4], prefix, made[4], ctx, n, None, 0.1)[0]))
    size = max(sdv.prefix_attn_workspace(c[0][0], c[0][1], c[0][4]).numel() for c in calls)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    graphs = []
    for made, prefix, ctx, n, want in calls:
        q, kp, vp, ptable, table = made
        out = torch.zeros_like(q)
        fixed = (dev([prefix]), table, dev(ctx), dev(n), None, 0.1, out, None, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sdv.sdv_prefix_attn(q, kp, vp, ptable, *fixed)
        graphs.append((graph, out, want, fixed))
    for _ in range(3):
        for graph, out, want, _ in graphs:
            out.zero_()
            graph.replay()
        for _, out, want, _ in graphs:
            assert torch.equal(out, want)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK


def test_the_binding_refuses_layouts_and_shapes(sdv):
    q, kp, vp, ptable, table = (x.cuda() for x in make(F16, 2, 2, 8, 2, 64, 16, 100, [0, 3], [2, 2], 12))
    i, out = dev([0, 3]), torch.zeros_like(q)
    ws = sdv.prefix_attn_workspace(q, kp, table)
    ok = dict(q=q, k_pages=kp, v_pages=vp, prefix_table=ptable, prefix_len=dev([100]), table=table, ctx=i, n_rows=None,
              mask=None, scale=0.1, out=out, lse=None, ws=ws)
    sdv.sdv_prefix_attn(**ok)
    for kw in (dict(prefix_table=ptable[None]), dict(prefix_len=i), dict(table=table[:1]), dict(ctx=i[:1]),
               dict(prefix_table=ptable[::2]), dict(out=out[..., :32])):
        with pytest.raises(ValueError):
            sdv.sdv_prefix_attn(**{**ok, **kw})
    for kw in (dict(prefix_len=dev([100]).long()), dict(prefix_table=ptable.float()), dict(q=q.bfloat16())):
        with pytest.raises(TypeError):
            sdv.sdv_prefix_attn(**{**ok, **kw})
    with pytest.raises(sdv.SdvError) as e:
        sdv.sdv_prefix_attn(**{**ok, "ws": ws[:ws.numel() // 2]})
    assert e.value.status == sdv.SDV_ERR_WORKSPACE


@pytest.mark.parametrize("case", [2, 4, 5, 6, 8])
def test_tables_for_long_sequences(sdv, case):
    """A table row that could hold more positions than one warp should walk sends the own positions through
    the paged attention, which deals any lengths evenly: the same result to the tolerances."""
    dt, B, S, hq, hkv, d, page, prefix, ctx, n, masked = SHAPES[case]
    q, kp, vp, ptable, table = make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, 300 + case)
    wide = torch.full((B, 40000 // page), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    mask = words(np.random.default_rng(case), B, S) if masked else None
    im = None if mask is None else as_i32(mask)
    out, lse, ws = call(sdv, q, kp, vp, ptable, prefix, wide, ctx, n, im, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    check(dt, reference(q, kp, vp, ptable, prefix, table, ctx, n, mask, d ** -0.5), out, lse, d)


@pytest.mark.parametrize("d,page", [(64, 8), (128, 16), (128, 32), (256, 128)])
def test_own_lengths_around_a_slice(sdv, d, page):
    """Own positions of every length around the slices, parts and pages of their kernel."""
    ctx = [0, 1, 7, 30, 31, 32, 33, 62, 63, 64, 65, 95, 127, 128, 190, 511]
    n = [1 + i % 3 for i in range(len(ctx))]
    q, kp, vp, ptable, table = make(BF16, len(ctx), 3, 8, 2, d, page, 40, ctx, n, d + page)
    out, lse, ws = call(sdv, q, kp, vp, ptable, 40, table, ctx, n, None, 0.1)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    check(BF16, reference(q, kp, vp, ptable, 40, table, ctx, n, None, 0.1), out, lse, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_positions_that_are_not_finite_or_absent(sdv, d):
    """A window row's infinities and NaN reach the rows that see it and no others, the context's reach all
    rows of their sequence; a page of a sequence's own that is none is absent, and reported."""
    ctx, n = [20, 40, 0], [3, 3, 2]
    q, kp, vp, ptable, table = make(F16, 3, 3, 8, 2, d, 16, 100, ctx, n, 30)
    at = lambda b, p: (int(table[b, p // 16]), p % 16)  # noqa: E731
    page, slot = at(0, 21)  # window row 1 of sequence 0
    vp[page, 0, slot, 3], vp[page, 0, slot, 9] = float("inf"), float("nan")
    page, slot = at(1, 5)   # a context position of sequence 1
    vp[page, 1, slot, 4] = float("-inf")
    out, _, ws = call(sdv, q, kp, vp, ptable, 100, table, ctx, n, None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    out = out.float().cpu()
    odd = ~torch.isfinite(out)
    want = torch.zeros_like(odd)
    want[0, 1:, :4, 3] = want[0, 1:, :4, 9] = True
    want[1, :, 4:, 4] = True
    assert torch.equal(odd, want)
    assert torch.isposinf(out[0, 1:, :4, 3]).all() and torch.isneginf(out[1, :, 4:, 4]).all()
    bad = table.clone()
    bad[1, 1] = kp.shape[0] + 5
    vp = torch.where(torch.isinf(vp), torch.zeros_like(vp), vp)
    vp[at(0, 21)[0], 0, at(0, 21)[1], 9] = 0.0
    out, lse, ws = call(sdv, q, kp, vp, ptable, 100, bad, ctx, n, None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
    # positions 16 .. 31 of sequence 1 are gone: pages 0 and 2 as its first two
    short = table.clone()
    short[1, 1] = table[1, 2]
    ref = reference(q, kp, vp, ptable, 100, short, [20, 24, 0], n, None, d ** -0.5)
    check(F16, ref, out, lse, d)


def forms(ptable, page):
    """The prefix's table as it is, and with room for more positions than few rows take in parts: what is
    asked for is the same, the kernel is another."""
    wide = torch.full((9000 // page + 1,), -1, dtype=torch.int32)
    wide[:len(ptable)] = ptable
    return ptable, wide


@pytest.mark.parametrize("dt,d,page", [(F16, 128, 16), (BF16, 64, 64), (BF16, 128, 8), (F16, 64, 32)])
@pytest.mark.parametrize("prefix", [1, 31, 32, 33, 63, 64, 65, 129, 2047, 2049, 4100, 8192])
def test_a_prefix_before_few_rows(sdv, dt, d, page, prefix):
    ctx, n = [0, 70], [2, 1]
    q, kp, vp, ptable, table = make(dt, 2, 2, 8, 2, d, page, prefix, ctx, n, prefix + d)
    ref = reference(q, kp, vp, ptable, prefix, table, ctx, n, None, d ** -0.5)
    for pt in forms(ptable[:-1], page):
        out, lse, ws = call(sdv, q, kp, vp, pt, prefix, table, ctx, n, None, d ** -0.5)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        check(dt, ref, out, lse, d)


@pytest.mark.parametrize("dt,d", [(F16, 128), (BF16, 64)])
def test_odd_values_and_absent_pages_before_few_rows(sdv, dt, d):
    ctx, n = [20, 3], [2, 1]
    q, kp, vp, ptable, table = make(dt, 2, 2, 8, 2, d, 16, 400, ctx, n, 8, std=20.0)
    for pt in forms(ptable[:-1], 16):
        bad = pt.clone()
        bad[5], bad[19] = -1, kp.shape[0]
        out, lse, ws = call(sdv, q, kp, vp, bad, 400, table, ctx, n, None, d ** -0.5)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
        keep = torch.cat([ptable[:5], ptable[6:19], ptable[20:25]])
        check(dt, reference(q, kp, vp, keep, 368, table, ctx, n, None, d ** -0.5), out, lse, d)
    at = lambda p: (int(ptable[p // 16]), p % 16)  # noqa: E731
    want = {}
    for p, h, c, x in ((3, 0, 1, float("inf")), (390, 0, d - 1, float("nan")), (140, 1, 7, float("-inf")),
                       (5, 1, 9, float("inf")), (391, 1, 9, float("-inf"))):
        page, slot = at(p)
        vp[page, h, slot, c] = x
        want[h, c] = float("nan") if (h, c) in want else x
    for pt in forms(ptable[:-1], 16):
        out, _, ws = call(sdv, q, kp, vp, pt, 400, table, ctx, n, None, d ** -0.5)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        out = out.float().cpu()
        for b, i in ((0, 0), (0, 1), (1, 0)):
            for h in range(8):
                for c in range(d):
                    x, y = float(out[b, i, h, c]), want.get((h // 4, c), 0.0)
                    assert np.isfinite(x) if y == 0.0 else (np.isnan(x) if np.isnan(y) else x == y)
        assert not out[1, 1].any()


def test_a_prefix_before_few_rows_behind_the_launch_that_writes_it(sdv):
    """A call reads what the launch in front of it in the stream writes: queries, cache and lengths."""
    ctx, n = [20, 3], [2, 2]
    q, kp, vp, ptable, table = (x.cuda() for x in make(F16, 2, 2, 8, 2, 128, 16, 1000, ctx, n, 31))
    want, _, ws = call(sdv, q, kp, vp, ptable, 1000, table, ctx, n, None, 0.1)
    out, c, m, ln = torch.zeros_like(q), dev(ctx), dev(n), dev([1000])
    q2, k2, v2, l2 = torch.zeros_like(q), torch.zeros_like(kp), torch.zeros_like(vp), torch.zeros_like(ln)
    for _ in range(50):
        out.zero_()
        for x in (q2, k2, v2, l2):
            x.zero_()
        for x, y in ((v2, vp), (k2, kp), (q2, q), (l2, ln)):
            x.copy_(y)
        sdv.sdv_prefix_attn(q2, k2, v2, ptable, l2, table, c, m, None, 0.1, out, None, ws)
        assert torch.equal(out, want)


def test_what_padding_rows_hold_before_few_rows(sdv):
    """Rows behind a window's end hold anything: the live rows' bits are the same, the others 0."""
    ctx, n = [20, 3], [2, 1]
    q, kp, vp, ptable, table = make(F16, 2, 2, 8, 2, 128, 16, 400, ctx, n, 32)
    want, wl, _ = call(sdv, q, kp, vp, ptable, 400, table, ctx, n, None, 0.1)
    for x in (float("nan"), float("inf"), 60000.0):
        other = q.clone()
        other[1, 1] = x
        out, lse, ws = call(sdv, other, kp, vp, ptable, 400, table, ctx, n, None, 0.1)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        assert torch.equal(out, want) and torch.equal(lse, wl) and not out[1, 1].any()


@pytest.mark.parametrize("S,d,page", [(5, 128, 16), (8, 64, 8), (9, 128, 32), (16, 64, 16), (16, 128, 128), (20, 64, 32)])
def test_own_lengths_of_wide_windows(sdv, S, d, page):
    """Windows of 20 to 80 rows a kv head, several warps to a sequence: lengths around the slices, parts and
    pages, windows with rows left out, some of whole warps."""
    ctx = [0, 1, 12, 27, 31, 32, 60, 64, 95, 128, 300]
    n = [S - (3 * i) % (S + 1) for i in range(len(ctx))]
    mask = words(np.random.default_rng(S), len(ctx), S)
    q, kp, vp, ptable, table = make(F16, len(ctx), S, 8, 2, d, page, 40, ctx, n, d + page + S)
    out, lse, ws = call(sdv, q, kp, vp, ptable, 40, table, ctx, n, as_i32(mask), 0.1)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    check(F16, reference(q, kp, vp, ptable, 40, table, ctx, n, mask, 0.1), out, lse, d)


@pytest.mark.parametrize("S,d", [(6, 128), (6, 64), (12, 128), (16, 64)])
def test_odd_values_and_absent_pages_of_wide_windows(sdv, S, d):
    """As for narrow windows above: what is not finite reaches the rows that see it, whichever warp they are in."""
    ctx, n = [20, 40, 0], [S, S, S - 1]
    q, kp, vp, ptable, table = make(F16, 3, S, 8, 2, d, 16, 100, ctx, n, 33)
    at = lambda b, p: (int(table[b, p // 16]), p % 16)  # noqa: E731
    i = S - 2
    page, slot = at(0, 20 + i)  # a window row that only the last two rows see
    vp[page, 0, slot, 3], vp[page, 0, slot, 9] = float("inf"), float("nan")
    page, slot = at(1, 5)       # a context position of sequence 1
    vp[page, 1, slot, 4] = float("-inf")
    out, _, ws = call(sdv, q, kp, vp, ptable, 100, table, ctx, n, None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    out = out.float().cpu()
    want = torch.zeros_like(out, dtype=torch.bool)
    want[0, i:, :4, 3] = want[0, i:, :4, 9] = True
    want[1, :, 4:, 4] = True
    assert torch.equal(~torch.isfinite(out), want)
    assert torch.isposinf(out[0, i:, :4, 3]).all() and torch.isneginf(out[1, :, 4:, 4]).all()
    bad = table.clone()
    bad[1, 1] = kp.shape[0] + 5
    vp = torch.where(torch.isinf(vp), torch.zeros_like(vp), vp)
    page, slot = at(0, 20 + i)
    vp[page, 0, slot, 9] = 0.0
    out, lse, ws = call(sdv, q, kp, vp, ptable, 100, bad, ctx, n, None, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
    short = table.clone()  # positions 16 .. 31 of sequence 1 are gone: pages 0 and 2 as its first two
    short[1, 1:-1] = table[1, 2:]
    ref = reference(q, kp, vp, ptable, 100, short, [20, 24, 0], n, None, d ** -0.5)
    check(F16, ref, out, lse, d)


MANY = [  # so many rows that the prefix's partials of a row are few, tables of one tile: joined on the spot
    (F16, 450, 1, 32, 8, 128, 16, 200, False),
    (BF16, 60, 8, 32, 8, 128, 32, 129, True),
    (F16, 32, 16, 32, 8, 64, 8, 300, True),
    (F16, 200, 2, 16, 8, 256, 16, 65, False),
    (BF16, 230, 2, 32, 8, 64, 64, 0, False),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows_and_short_tables(sdv, case):
    dt, B, S, hq, hkv, d, page, prefix, masked = MANY[case]
    n = [S - (5 * i) % (S + 1) for i in range(B)]
    ctx = [min((11 * i) % 64, 64 - n[i]) for i in range(B)]
    q, kp, vp, ptable, table = make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, 50 + case)
    mask = words(np.random.default_rng(case), B, S) if masked else None
    im = None if mask is None else as_i32(mask)
    out, lse, ws = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, im, d ** -0.5)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
    check(dt, reference(q, kp, vp, ptable, prefix, table, ctx, n, mask, d ** -0.5), out, lse, d)
    out2, _, _ = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, im, d ** -0.5, want_lse=False, ws=ws)
    assert torch.equal(out2, out)
    # what is not finite: in the prefix (all live rows of its head), in a context, in a window row
    want = torch.zeros(out.shape, dtype=torch.bool)
    b = next(i for i in range(B) if ctx[i] > 3 and n[i] > 0)
    group = hq // hkv
    if prefix:
        vp[int(ptable[0]), 1, 3 % min(page, prefix), 5] = float("inf")
        for i in range(B):
            want[i, :n[i], group:2 * group, 5] = True
    vp[int(table[b, 2 // page]), 0, 2 % page, 7] = float("nan")
    want[b, :n[b], :group, 7] = True
    if not masked:
        at = ctx[b] + n[b] - 1
        vp[int(table[b, at // page]), 2, at % page, 9] = float("-inf")
        want[b, n[b] - 1, 2 * group:3 * group, 9] = True
    odd, _, _ = call(sdv, q, kp, vp, ptable, prefix, table, ctx, n, im, d ** -0.5, ws=ws)
    odd = odd.float().cpu()
    assert torch.equal(~torch.isfinite(odd), want)
    assert torch.isnan(odd[b, :n[b], :group, 7]).all()
    if prefix:
        assert all(torch.isposinf(odd[i, :n[i], group:2 * group, 5]).all() for i in range(B))
    if not masked:
        assert torch.isneginf(odd[b, n[b] - 1, 2 * group:3 * group, 9]).all()
    assert torch.equal(odd[~want], out.float().cpu()[~want])


@pytest.mark.parametrize("dt,B,S,hq,hkv,d,page,prefix", [
    (F16, 5, 3, 8, 2, 80, 16, 333), (BF16, 9, 4, 12, 3, 112, 24, 129), (F16, 40, 2, 8, 1, 72, 5, 95), (BF16, 3, 1, 4, 4, 8, 16, 31),
    (F16, 30, 5, 6, 2, 192, 16, 200), (BF16, 70, 1, 16, 2, 136, 3, 64), (F16, 2, 32, 9, 1, 24, 1, 33), (BF16, 17, 2, 200, 2, 64, 16, 65)])
def test_other_head_and_page_sizes(sdv, dt, B, S, hq, hkv, d, page, prefix):
    ctx, n = [(7 * i) % 40 for i in range(B)], [S - i % (S + 1) for i in range(B)]
    q, kp, vp, ptable, table = make(dt, B, S, hq, hkv, d, page, prefix, ctx, n, d)
    for length in (prefix, max(prefix - page, 0)):
        out, lse, ws = call(sdv, q, kp, vp, ptable, length, table, ctx, n, None, d ** -0.5)
        assert sdv.sdv_last_device_status(ws) == sdv.SDV_OK
        check(dt, reference(q, kp, vp, ptable, length, table, ctx, n, None, d ** -0.5), out, lse, d)
