"""sdv_page_assign on the GPU against the oracle: every value equal."""
import random

import pytest
import torch

from oracle import rounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, sdv, B, T, n_pages, page, width, seed=0):
        self.sdv, self.B, self.T, self.page = sdv, B, T, page
        rng = random.Random(seed)
        self.free = list(range(n_pages))
        rng.shuffle(self.free)
        self.n_free, self.table, self.held = n_pages, [[-1] * width for _ in range(B)], [0] * B
        self.dev = [ints(self.free), ints([n_pages]), ints(self.table), ints(self.held)]
        self.ws = sdv.page_assign_workspace(ints([0] * B))
        self.out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B,), (B, T), (B, T))]

    def call(self, ctx, n, maps=True, stream=None):
        g, p, s = self.out
        self.sdv.sdv_page_assign(*self.dev, self.page, ints(ctx), None if n is None else ints(n), g,
                                 p if maps else None, s if maps else None, self.ws, stream, T=self.T)

    def check(self, ctx, n, maps=True):
        n = [self.T] * self.B if n is None else n
        want = rounds.assign(self.free, self.n_free, self.table, self.held, self.page, ctx, n, self.T)
        self.call(ctx, n, maps)
        self.free, self.n_free, self.table, self.held = (want[k] for k in ("free", "n_free", "table", "held"))
        for got, key in zip(self.dev, ("free", "n_free", "table", "held")):
            assert got.tolist() == ([want[key]] if key == "n_free" else want[key]), key
        assert self.out[0].tolist() == want["granted"]
        if maps:
            assert self.out[1].tolist() == want["positions"] and self.out[2].tolist() == want["slots"]
        return want


@pytest.mark.parametrize("B,T,page,width", [(1, 1, 16, 4), (1, 1, 1, 3), (3, 17, 16, 9), (48, 17, 16, 40),
                                            (31, 300, 7, 60), (33, 5, 64, 3), (300, 9, 16, 5), (700, 33, 8, 12),
                                            (1025, 3, 4, 6), (2100, 2, 16, 2), (5, 5000, 16, 320)])
def test_random_rounds(sdv, B, T, page, width):
    rng = random.Random(B * 1000 + T)
    most = width * page
    # too few pages for everyone, so that some calls run short
    pool = Pool(sdv, B, T, max(1, B * width * 2 // 3), page, width, seed=B)
    ctx = [0] * B
    for step in range(6):
        n = [rng.choice([0, 1, T, rng.randint(0, T)]) for _ in range(B)]
        n = [min(x, most - c) for x, c in zip(n, ctx)]
        want = pool.check(ctx, n, maps=step != 4)
        assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_OK
        # some requests end, some keep a part of what they were granted
        ctx = [0 if rng.random() < 0.3 else c + rng.randint(0, g) for c, g in zip(ctx, want["granted"])]
    pool.check([0] * B, [0] * B)
    assert pool.n_free == len(pool.free) and sorted(pool.free) == list(range(len(pool.free)))


def test_rows_left_out_mean_all(sdv):
    pool = Pool(sdv, 3, 20, 40, 16, 4)
    pool.check([0, 5, 30], None)


def test_giving_back_what_was_taken(sdv):
    pool = Pool(sdv, 300, 40, 4000, 16, 12)
    pool.check([0] * 300, [i % 40 for i in range(300)])
    before = [t.clone() for t in pool.dev]
    ctx = [i % 40 for i in range(300)]
    pool.check(ctx, [40] * 300)
    pool.check(ctx, [0] * 300)
    assert all(torch.equal(a, b) for a, b in zip(pool.dev, before))


def test_rows_in_place_and_values_out_of_range(sdv):
    """granted may be n_rows; lengths out of range are clamped and reported."""
    pool = Pool(sdv, 4, 8, 16, 4, 3)
    n = ints([8, -2, 100, 3])
    ctx = ints([0, 0, 0, -5])
    pool.sdv.sdv_page_assign(*pool.dev, 4, ctx, n, n, pool.out[1], pool.out[2], pool.ws, T=8)
    assert n.tolist() == [8, 0, 8, 3]
    assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_ERR_INVALID_ARG
    assert pool.dev[3].tolist() == [2, 0, 2, 1]
    # past the table's row: the rows that fit have places
    pool.sdv.sdv_page_assign(*pool.dev, 4, ints([10, 0, 8, 3]), ints([8, 0, 0, 0]), n, pool.out[1], pool.out[2],
                             pool.ws, T=8)
    assert n.tolist() == [2, 0, 0, 0] and pool.dev[3].tolist() == [3, 0, 2, 1]
    assert pool.out[1][0].tolist() == [10, 11] + [-1] * 6
    assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_ERR_INVALID_ARG


def test_a_damaged_list_is_reported(sdv):
    pool = Pool(sdv, 1, 8, 4, 4, 3)
    pool.dev[0][:] = ints([0, 1, 99, -7])
    pool.call([0], [8])
    assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_ERR_INVALID_ARG
    assert pool.out[2].tolist() == [[-1] * 8]  # neither is a page
    # more given back than there are pages: the rest is dropped
    pool.dev[1][:] = 4
    pool.call([0], [0])
    assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_ERR_INVALID_ARG
    assert pool.dev[1].tolist() == [4] and pool.dev[3].tolist() == [0]


def test_captured_rounds_and_streams(sdv):
    B, T = 40, 9
    pool = Pool(sdv, B, T, 600, 4, 16)
    ctx, n = ints([3 * i % 20 for i in range(B)]), ints([T] * B)
    none = ints([0] * B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = [t.clone() for t in pool.dev]
    g, p, s = pool.out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sdv.sdv_page_assign(*pool.dev, 4, ctx, n, g, p, s, pool.ws)
        sdv.sdv_page_assign(*pool.dev, 4, none, none, None, None, None, pool.ws, T=T)
    torch.cuda.current_stream().wait_stream(side)
    first = [t.clone() for t in pool.out]
    assert torch.equal(pool.dev[3], none)
    for t, b in zip(pool.dev, before):
        t.copy_(b)
    with torch.cuda.graph(graph):
        sdv.sdv_page_assign(*pool.dev, 4, ctx, n, g, p, s, pool.ws)
        sdv.sdv_page_assign(*pool.dev, 4, none, none, None, None, None, pool.ws, T=T)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(pool.out, first))
    want = rounds.assign(pool.free, pool.n_free, pool.table, pool.held, 4, ctx.tolist(), n.tolist(), T)
    assert g.tolist() == want["granted"] and s.tolist() == want["slots"]
