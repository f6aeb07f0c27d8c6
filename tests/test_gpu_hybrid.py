"""The hybrid example: speculative rounds over caches and states.

A window of S rows and single-row windows differ by roundings of 2^-11 in each
layer's mixer and projection inputs, about ten of them: 1e-3 of the hidden rows'
norm, so 4e-3 (one sigma) on logits of size 4, 0.02 over all the tokens compared.
Tokens are compared while the plain stream's top-2 gap is above 0.05.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
GAP = 0.05


@pytest.fixture(scope="module")
def hybrid():
    from speculative_decode_verify_sdv_gb300 import build, hybrid as _hybrid, sdv
    build.build()
    sdv.load()
    return _hybrid


def plain(hybrid, prompt, count, **kw):
    """Single-token decoding: the tokens, the target, and how many steps kept the gap."""
    target = hybrid.HybridTarget(**kw)
    logits = torch.empty((1, target.embed.shape[0]), dtype=torch.float32, device="cuda")
    out, gaps = [target.prefill(prompt, logits)], []
    for _ in range(count - 1):
        top = logits[0].topk(2).values
        gaps.append(float(top[0] - top[1]))
        out.append(target.round(out[-1], [], 0, logits)[1])
    safe = next((i for i, g in enumerate(gaps) if g < GAP), len(gaps))
    return out, target, safe


@pytest.mark.parametrize("length", [5, 40, 333])
def test_rounds_commit_the_accepted_rows_alone(hybrid, length):
    gen = torch.Generator().manual_seed(length)
    prompt = torch.randint(0, 4096, (length,), generator=gen).tolist()
    rounds = 0
    for seed in range(6):
        want, _, safe = plain(hybrid, prompt, 40, seed=seed)
        target = hybrid.HybridTarget(seed=seed)
        got, k, at = [target.prefill(prompt)], 6, 0
        while len(got) - 1 + k < safe:
            right = at % (k + 1)  # drafts that are right, then a wrong one
            drafts = want[len(got):len(got) + k]
            if right < k:
                drafts[right] = (drafts[right] + 1) % 4096
            accepted, a0 = target.round(got[-1], drafts, k)
            assert accepted == right
            got += drafts[:accepted] + [a0]
            assert got == want[:len(got)]
            at += 1
        rounds += at
        # the state and the context of having decoded those tokens alone (the last is not in yet)
        alone = hybrid.HybridTarget(seed=seed)
        alone.prefill(prompt)
        for t in got[:-1]:
            alone.round(t, [], 0)
        assert int(target.ctx) == int(alone.ctx) == length + len(got) - 1
        for x, y in zip(target.layers, alone.layers):
            if hasattr(x, "state"):
                err = (x.state - y.state).abs().max() / y.state.abs().max()
                assert float(err) < 2.0 ** -7
        assert target.status() == alone.status() == 0
    assert rounds >= 6


def test_generate(hybrid):
    prompt = [7, 8, 9] * 20
    tokens, rounds = hybrid.generate(hybrid.HybridTarget(), prompt, 60)
    assert len(tokens) == 60 and 0 < rounds < 60
    want, _, safe = plain(hybrid, prompt, 60)
    assert tokens[:safe] == want[:safe]


def test_windows_past_the_limit_are_refused(hybrid):
    target = hybrid.HybridTarget()
    target.prefill([1, 2, 3])
    with pytest.raises(ValueError):
        target.round(1, [2] * 32, 32)
    with pytest.raises(ValueError):
        target.round(1, [2, 3], 1)
