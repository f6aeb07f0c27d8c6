"""What a round of the hybrid example commits, exactly: the accepted rows and no other.

Rows of one window do not depend on the ones behind them, so two rounds that differ in
rejected drafts alone leave the same bits; and the new state is the old one advanced by
the accepted rows' keys and values, to the tolerance of the operator's own tests.
"""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests.test_gpu_hybrid import plain
from tests.test_gpu_linear_attn import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hybrid():
    from speculative_decode_verify_sdv_gb300 import build, hybrid as _hybrid, sdv
    build.build()
    sdv.load()
    return _hybrid


def cached(layer, ctx):
    """The layer's keys and values of the first ctx positions."""
    p = torch.arange(ctx, device=layer.table.device)
    at = layer.table[0].long()[p // layer.k.shape[2]], slice(None), p % layer.k.shape[2]
    return layer.k[at], layer.v[at]


@pytest.mark.parametrize("length,right,k", [(5, 0, 4), (40, 3, 6), (300, 5, 6), (77, 1, 20)])
def test_a_round_commits_the_accepted_rows_to_the_bit(hybrid, length, right, k):
    prompt = torch.randint(0, 4096, (length,), generator=torch.Generator().manual_seed(length)).tolist()
    for seed in range(20):
        want, _, safe = plain(hybrid, prompt, right + 3, seed=seed)
        if safe >= right + 2:
            break
    after = []
    for tail in (1, 1000):
        target = hybrid.HybridTarget(seed=seed)
        a0 = target.prefill(prompt)
        before = [x.state.clone() for x in target.layers if hasattr(x, "state")]
        drafts = want[1:1 + right] + [(want[1 + right] + tail) % 4096] + [(7 * tail + j) % 4096 for j in range(k - 1 - right)]
        accepted, nxt = target.round(a0, drafts, k)
        assert accepted == right and nxt == want[1 + right]
        n = accepted + 1
        assert int(target.ctx) == length + n
        linear = [x for x in target.layers if hasattr(x, "state")]
        for x, old in zip(linear, before):
            kk, vv = x.kv
            g = np.broadcast_to(f64(x.decay), (1, kk.shape[1], x.h))
            ref = mixing.linear(None, f64(kk), f64(vv), g, 1.0, [n], f64(old))
            tol = (2.0 ** -16 + (kk.shape[1] + 64) * 2.0 ** -22) * ref["state_abs"] + 2.0 ** -126
            assert np.all(np.abs(f64(x.state) - ref["state"]) <= tol)
        after.append([x.state for x in linear] +
                     [t for x in target.layers if not hasattr(x, "state") for t in cached(x, int(target.ctx))])
        assert target.status() == 0
    assert len(after[0]) == 4
    for x, y in zip(*after):
        assert torch.equal(x, y)
