"""sdv_verify_drafts: forms and limits beside those of tests/test_gpu_verify_drafts.py."""
import pytest
import torch

from tests.test_gpu_verify_drafts import BF16, F32, call, check, make

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


@pytest.mark.parametrize("dt,B,S,V", [(F32, 60, 2, 40001), (F32, 130, 3, 9001), (BF16, 200, 2, 40001),
                                      (F32, 256, 2, 20011)])
def test_drafters_probabilities_of_many_sequences(sdv, dt, B, S, V):
    """The more sequences, the fewer CTAs look through the probabilities of one: four, two and one here,
    several chunks a warp."""
    args = make(dt, B, S, V, True, 600 + B)
    accepted, token, ws = call(sdv, args)
    check(args, accepted, token)
    again, token2, _ = call(sdv, args, ws)
    assert torch.equal(again, accepted) and torch.equal(token2, token)
    args[3] = None
    accepted, token, _ = call(sdv, args, ws)
    check(args, accepted, token)


@pytest.mark.parametrize("B,V", [(1, 151936), (3, 300), (60, 40001), (256, 9001)])
def test_a_drafter_that_leaves_nothing(sdv, B, V):
    """Probabilities that are nowhere below the target's: a draft that is not kept leaves no weight, and
    the next token is drawn from the target's own row, the draft's token among the rest."""
    args = make(F32, B, 2, V, True, 700 + B)
    logits, t, drafts, n, q, u = args
    n.fill_(1)
    t.fill_(1.0)
    q.fill_(1.0)
    p = torch.softmax(logits[:, 0].double(), -1)
    drafts[:, 0] = p.argmin(-1).to(torch.int32)  # its probability is far below u
    u[:, 0] = 0.75
    accepted, token, _ = call(sdv, args)
    assert not accepted.any()
    check(args, accepted, token)
    running = torch.cumsum(p, -1)
    want = (running <= (u[:, 1].double() * running[:, -1])[:, None]).sum(-1)
    assert (token.long() - want).abs().max() <= 1 and (token.long() == want).float().mean() >= 0.99
    # beside sequences of which something is left
    q[::2] = make(F32, B, 2, V, True, 800 + B)[4][::2]
    accepted, token, _ = call(sdv, args)
    check(args, accepted, token)


def test_greedy_drafts_at_a_tie(sdv):
    """The lowest index of the maximum is kept, one behind it and one below the maximum are not."""
    args = make(BF16, 4, 2, 9000, False, 8)
    args[0].fill_(1.0)
    args[0][1, :, :3000] = 0.5
    args[0][3, :, :3000] = 0.5
    args[1].zero_()
    args[2][:] = torch.tensor([[0], [3000], [5], [2999]], dtype=torch.int32)
    args[3].fill_(1)
    accepted, token, _ = call(sdv, args)
    assert accepted.tolist() == [1, 1, 0, 0] and token.tolist() == [0, 3000, 0, 3000]
    check(args, accepted, token)
