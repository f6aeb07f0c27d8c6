"""sdv_verify_drafts on the GPU against the 64-bit oracle: every value equal, but where the oracle's
own margin is below what the documentation allows (fp32 sums of a test: 2^-18 of a probability; the
draw: held to 2^-34 of all weights here, a sixteenth of it)."""
import numpy as np
import pytest
import torch

from oracle import rounds

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def make(dt, B, S, V, probs, seed, pad=0, std=2.2, lead=0):
    """Logits as a slice of wider rows (pad elements more each), `lead` elements past an aligned address."""
    gen = torch.Generator().manual_seed(seed)
    logits = torch.randn((B, S, V), generator=gen) * std
    q = torch.softmax(logits[:, :S - 1] + 0.7 * torch.randn((B, S - 1, V), generator=gen), -1)
    if probs:
        drafts = torch.stack([torch.multinomial(x, 1, generator=gen)[:, 0] for x in q]) if S > 1 else None
    else:
        best = logits[:, :S - 1].argmax(-1)
        other = torch.randint(0, V, (B, S - 1), generator=gen)
        drafts = torch.where(torch.rand((B, S - 1), generator=gen) < 0.7, best, other)
    store = torch.full((B * S * (V + pad) + lead,), float("nan"), dtype=dt, device="cuda")
    view = store[lead:].view(B, S, V + pad)[:, :, :V]
    view.copy_(logits.to(dt))
    t = torch.tensor([[0.7, 1.0, 0.0, 1.3, 0.2][i % 5] for i in range(B)])
    u = torch.rand((B, S), generator=gen)
    n = torch.tensor([max(0, S - 1 - i % 3) for i in range(B)], dtype=torch.int32)
    return [view, t.cuda(), None if S == 1 else drafts.to(torch.int32).cuda(), n.cuda(),
            q.contiguous().cuda() if probs else None, u.cuda()]


def call(sdv, args, ws=None, stream=None):
    B = args[0].shape[0]
    accepted, token = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = sdv.verify_drafts_workspace(args[0]) if ws is None else ws
    sdv.sdv_verify_drafts(*args, accepted, token, ws, stream)
    return accepted, token, ws


def check(args, accepted, token):
    logits, t, drafts, n, q, u = (None if x is None else x.detach().cpu().float().numpy() for x in args)
    B, S = logits.shape[:2]
    tight = 0
    for b in range(B):
        k = S - 1 if n is None else int(n[b])
        want = rounds.verify(logits[b], float(t[b]), drafts[b] if drafts is not None else [], k,
                             None if q is None else q[b], u[b])
        if want[2] < 2.0 ** -34:
            tight += 1
            continue
        assert (int(accepted[b]), int(token[b])) == want[:2], (b, want)
    assert tight <= 1


SHAPES = [
    # dtype, B, S, V, probs, pad, lead
    (F32, 1, 1, 1, False, 0, 0),
    (F32, 3, 4, 2, True, 0, 0),
    (F32, 1, 5, 151936, False, 0, 0),
    (F32, 4, 3, 32000, True, 0, 0),
    (BF16, 7, 1, 50257, False, 0, 0),          # rows of odd length, one behind the other
    (F16, 5, 3, 50257, True, 0, 0),
    (F32, 5, 3, 2049, True, 3, 1),             # every alignment of a row
    (BF16, 9, 2, 4095, True, 1, 3),
    (F16, 6, 2, 7, True, 0, 5),
    (F32, 40, 2, 300, False, 0, 0),
    (F32, 2, 32, 1000, True, 0, 0),
    (BF16, 2, 32, 5000, False, 24, 0),
    (F32, 200, 1, 5000, False, 0, 0),
    (F16, 3, 2, 300000, True, 0, 0),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_against_the_oracle(sdv, case):
    dt, B, S, V, probs, pad, lead = SHAPES[case]
    args = make(dt, B, S, V, probs, 500 + case, pad, lead=lead)
    accepted, token, ws = call(sdv, args)
    check(args, accepted, token)
    again, token2, _ = call(sdv, args, ws)
    assert torch.equal(again, accepted) and torch.equal(token2, token)
    args[3] = None  # all drafts
    accepted, token, _ = call(sdv, args, ws)
    check(args, accepted, token)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_draws_over_the_whole_row(sdv, dt):
    """Random numbers from 0 to just below 1 at a flat and a steep row: every draw is the oracle's."""
    B, V = 256, 20011
    gen = torch.Generator().manual_seed(5)
    for std in (0.1, 4.0):
        row = (torch.randn((1, 1, V), generator=gen) * std).to(dt)
        u = torch.arange(B, dtype=F32)[:, None] / B
        u[-1] = 1.0 - 2.0 ** -24
        args = [row.expand(B, 1, V).contiguous().cuda(), torch.ones(B, device="cuda"), None, None, None, u.cuda()]
        accepted, token, _ = call(sdv, args)
        check(args, accepted, token)
        assert token[0] == 0


def test_filtered_rows(sdv):
    """-inf takes tokens out, NaN too; a row with nothing left gives -1; +inf takes everything."""
    args = make(F32, 8, 3, 5000, False, 6)
    x = args[0]
    x[0, :, 10:] = float("-inf")
    x[1, 0] = float("-inf")
    x[2] = float("nan")
    x[3, :, ::2] = float("nan")
    x[4, :, 77] = float("inf")
    x[5, 0, :] = float("-inf")
    x[5, 0, 4999] = -3.0e38
    x[6, :, :] = float("-inf")
    x[6, :, 2048] = 0.0
    accepted, token, _ = call(sdv, args)
    check(args, accepted, token)
    assert token[1] == -1 and accepted[1] == 0 and token[2] == -1
    args[1].fill_(0.0)  # greedy
    accepted, token, _ = call(sdv, args)
    check(args, accepted, token)


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), 1e-42, float("inf"), 1e30, 1e-4, 1e-6, 1e-37, 3e-38])
def test_temperatures(sdv, t):
    args = make(F32, 4, 3, 3001, True, 7)
    args[1].fill_(t)
    accepted, token, _ = call(sdv, args)
    if t == 1e-42:  # log2(e) / T overflows: greedy
        args[1].fill_(0.0)
    check(args, accepted, token)


def test_greedy_ties_go_to_the_lowest(sdv):
    args = make(BF16, 3, 2, 9000, False, 8)
    args[0].fill_(1.0)
    args[0][1, :, :3000] = 0.5
    args[1].zero_()
    args[2][:] = torch.tensor([[0], [3000], [5]], dtype=torch.int32)
    accepted, token, _ = call(sdv, args)
    assert accepted.tolist() == [1, 1, 0] or args[3].tolist() != [1, 1, 1]
    check(args, accepted, token)


def test_drafts_and_probabilities_at_their_limits(sdv):
    args = make(F32, 6, 2, 4000, True, 9)
    args[3].fill_(1)
    args[1].fill_(1.0)
    logits, _, drafts, _, q, u = args
    u[:, 0] = 0.0
    drafts[0], drafts[1] = -1, 4000          # outside: never kept
    q[2] = 0.0                               # a drafter that gives nothing: kept wherever p > 0
    q[3] = torch.softmax(logits[3, 0].double(), 0).float()  # the target's own: kept with u < 1
    u[3, 0] = 0.999
    q[4] = float("nan")                      # counts as 0
    q[5] = -1.0
    accepted, token, _ = call(sdv, args)
    assert accepted.tolist() == [0, 0, 1, 1, 1, 1]
    check(args, accepted, token)
    # the same draft twice, and a count of drafts out of range
    args = make(F32, 2, 4, 4000, False, 10)
    args[2][:] = args[2][:, :1]
    args[3][:] = torch.tensor([99, -4], dtype=torch.int32)
    accepted, token, _ = call(sdv, args)
    args[3][:] = torch.tensor([3, 0], dtype=torch.int32)
    check(args, accepted, token)


def test_a_rejected_draft_that_has_nearly_all_weight(sdv):
    """What is left without it is far below it: its own digits count."""
    B, V = 64, 30000
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((B, 2, V), generator=gen)
    x[:, :, 123] = 30.0
    u = torch.rand((B, 2), generator=gen)
    u[:, 0] = 1.0 - 2.0 ** -24  # p(123) is 1 - 5e-9 of about 1: rejected where it is below
    x[:, :, 123] = 24.0
    args = [x.cuda(), torch.ones(B, device="cuda"), torch.full((B, 1), 123, dtype=torch.int32, device="cuda"), None,
            None, u.cuda()]
    accepted, token, _ = call(sdv, args)
    assert not accepted.any() and not (token == 123).any()
    check(args, accepted, token)


def test_the_accept_follows_the_probabilities(sdv):
    """Over many random numbers a draft of probability p against q is kept in min(1, p / q) of the cases and
    the next token follows what is left (three tokens, within 5 standard deviations)."""
    B = 20000
    p, q = torch.tensor([0.5, 0.3, 0.2]), torch.tensor([0.2, 0.2, 0.6])
    gen = torch.Generator().manual_seed(12)
    drafts = torch.multinomial(q, B, replacement=True, generator=gen).to(torch.int32)[:, None]
    u = torch.rand((B, 2), generator=gen)
    args = [p.log().expand(B, 2, 3).contiguous().cuda(), torch.ones(B, device="cuda"), drafts.cuda(), None,
            q.expand(B, 1, 3).contiguous().cuda(), u.cuda()]
    accepted, token, _ = call(sdv, args)
    first = torch.where(accepted == 1, drafts.cuda()[:, 0], token)
    share = torch.bincount(first.long(), minlength=3).double().cpu() / B
    assert torch.all((share - p).abs() <= 5 * (p * (1 - p) / B).sqrt())


def test_captured_with_a_shared_workspace_and_a_side_stream(sdv):
    a, b = make(F32, 6, 3, 9000, True, 13), make(BF16, 20, 1, 50257, False, 14)
    want = [call(sdv, x)[:2] for x in (a, b)]
    size = max(sdv.verify_drafts_workspace(x[0]).numel() for x in (a, b))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (a, b):
        out = [torch.zeros(x[0].shape[0], dtype=torch.int32, device="cuda") for _ in range(2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sdv.sdv_verify_drafts(*x, *out, ws)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    for (_, out), w in zip(graphs, want):
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    acc, token, _ = call(sdv, a, stream=side)
    side.synchronize()
    assert torch.equal(acc, want[0][0]) and torch.equal(token, want[0][1])


def test_the_binding_refuses(sdv):
    args = make(F32, 4, 3, 100, True, 15)
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = sdv.verify_drafts_workspace(args[0])
    sdv.sdv_verify_drafts(*args, i, i.clone(), ws)
    for k, bad in ((0, args[0][..., ::2]), (0, args[0].transpose(0, 1)), (0, args[0][0]), (2, args[2][:, :1]),
                   (4, args[4][..., :50]), (5, args[5][:, :2]), (1, args[1][:2])):
        with pytest.raises(ValueError):
            sdv.sdv_verify_drafts(*args[:k], bad, *args[k + 1:], i, i.clone(), ws)
    for k, bad in ((1, args[1].double()), (2, args[2].long()), (4, args[4].half()), (0, args[0].double())):
        with pytest.raises(TypeError):
            sdv.sdv_verify_drafts(*args[:k], bad, *args[k + 1:], i, i.clone(), ws)
    with pytest.raises(sdv.SdvError) as e:
        sdv.sdv_verify_drafts(*args, i, i.clone(), ws[:256])
    assert e.value.status == sdv.SDV_ERR_WORKSPACE
