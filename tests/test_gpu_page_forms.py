"""sdv_page_assign: sides of its choices beside those of tests/test_gpu_page_assign.py."""
import random

import pytest

from tests.test_gpu_page_assign import Pool, sdv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,page,width", [(255, 1, 16, 3), (256, 1, 16, 3), (255, 10, 4, 5), (256, 10, 4, 5),
                                            (80, 32, 16, 4), (197, 13, 8, 4), (1, 2560, 16, 170), (1, 2561, 16, 170),
                                            (1024, 2, 2, 4), (1025, 2, 2, 4)])
def test_around_the_borders_of_the_forms(sdv, B, T, page, width):  # noqa: F811
    rng = random.Random(B + T)
    pool = Pool(sdv, B, T, max(1, B * width * 2 // 3), page, width, seed=B)
    ctx = [0] * B
    for step in range(4):
        n = [min(rng.choice([0, 1, T, rng.randint(0, T)]), width * page - c) for c in ctx]
        want = pool.check(ctx, n, maps=step != 2)
        assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_OK
        ctx = [0 if rng.random() < 0.3 else c + rng.randint(0, g) for c, g in zip(ctx, want["granted"])]
    pool.check([0] * B, [0] * B)
    assert sorted(pool.free[:pool.n_free]) == list(range(len(pool.free)))


@pytest.mark.parametrize("B,page,width,maps", [(255, 16, 300, False), (255, 16, 300, True), (3, 1, 20000, False),
                                               (200, 8, 1000, False), (9, 4, 9000, True),
                                               (64, 2, 1024, True), (64, 2, 1025, True)])
def test_long_tables_are_taken_and_given_back(sdv, B, page, width, maps):  # noqa: F811
    """Whole tables of entries in a call, with few rows to place or none."""
    pool = Pool(sdv, B, 4, B * width + 7, page, width, seed=B)
    pool.T = width * page
    full = [width * page - 4 - b % 3 for b in range(B)]
    pool.check(full, [0] * B, maps=False)  # (contexts that another program has filled)
    pool.T = 4
    pool.check([c // 2 for c in full], [b % 5 for b in range(B)], maps=maps)
    pool.check(full, [0] * B, maps=maps)
    before = [t.clone() for t in pool.dev]
    pool.check([0] * B, [0] * B, maps=maps)
    pool.check(full, [0] * B, maps=maps)
    # (what lies behind the list's end is of no meaning)
    assert pool.dev[0][:pool.n_free].equal(before[0][:pool.n_free])
    assert all(x.equal(y) for x, y in zip(pool.dev[1:], before[1:]))
    assert sdv.sdv_last_device_status(pool.ws) == sdv.SDV_OK
