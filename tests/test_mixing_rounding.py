"""The token mixers' outputs against the roundings that they are allowed, and mistakes
planted in the oracle's arithmetic (CPU) that the check has to find."""
import numpy as np
import pytest
import torch

from oracle import mixing
from tests import test_gpu_linear_attn as lin
from tests import test_gpu_paged_attn as att
from tests.rounding_checks import check_roundings
from tests.test_gpu_linear_attn import BF16, F16, U, f64

CHUNK = 128


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


# ---- on the CPU: the roundings as the operators may make them, and mistakes -----------

def rounded(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dt).double().numpy()


def chunked(q, k, v, g, scale, state, dt, mistake=None):
    """One head in chunks, scores, states and outputs rounded to the type; no batch."""
    T = v.shape[0]
    o, m = np.zeros_like(v), state.copy()
    for t in range(0, T, CHUNK):
        at = slice(t, min(t + CHUNK, T))
        gc = g[at] * (1.03 if mistake == "decay" else 1.0)
        run = np.cumsum(gc)
        p = np.tril(q[at] @ k[at].T * np.exp(np.minimum(run[:, None] - run[None, :], 0.0)))
        if mistake == "left out":
            p[np.subtract.outer(np.arange(len(p)), np.arange(len(p))) == 32] = 0.0
        y = rounded(p, dt) @ v[at] + np.exp(run)[:, None] * (q[at] @ rounded(m, dt))
        o[at] = rounded(scale * y, dt)
        m = np.exp(run[-1]) * m + (k[at] * np.exp(run[-1] - run)[:, None]).T @ v[at]
    return o


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [17, 200, 515])
@pytest.mark.parametrize("mistake", [None, "decay", "left out"])
def test_planted_mistakes_in_linear_attention(dt, T, mistake):
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(s, generator=gen).to(dt).double().numpy()  # noqa: E731
    q, k, v = r(T, 128), r(T, 128) / 8.0, r(T, 64)
    k = rounded(k, dt)
    g = -0.1 * torch.rand(T, generator=gen).double().numpy()
    s = torch.randn((128, 64), generator=gen).double().numpy()
    four = lambda x: x[None, :, None]  # noqa: E731
    ref = mixing.linear(four(q), four(k), four(v), g[None, :, None], 0.3, [T], s[None, None])
    o, squares = mixing.linear_squares(four(q), four(k), four(v), g[None, :, None], 0.3, [T], s[None, None], CHUNK)
    assert np.allclose(o, ref["o"], rtol=1e-10, atol=1e-10)
    got = four(chunked(q, k, v, g, 0.3, s, dt, mistake))
    if mistake is None or (mistake == "left out" and T <= 32):
        check_roundings(U[dt], got, ref["o"], squares, ref["o_abs"])
    else:
        with pytest.raises(AssertionError):
            check_roundings(U[dt], got, ref["o"], squares, ref["o_abs"])


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("N", [40, 613, 3000])
@pytest.mark.parametrize("mistake", [None, "left out", "seen twice", "scale"])
def test_planted_mistakes_in_attention(dt, N, mistake):
    d, hq = 64, 16
    gen = torch.Generator().manual_seed(N)
    r = lambda *s: torch.randn(s, generator=gen).to(dt).double().numpy()  # noqa: E731
    q, kp, vp = r(1, 1, hq, d) * 1.5, r(1, 1, N, d), r(1, 1, N, d)
    args = (kp, vp, [[0]], [N - 1], [1], None, 0.125)
    ref = mixing.attention(q, *args)
    squares = mixing.attention_squares(q, *args)
    scale = 0.125 * (1.02 if mistake == "scale" else 1.0)
    s = q[0, 0] @ kp[0, 0].T * scale
    w = np.exp(s - s.max(1, keepdims=True))
    if mistake == "left out":
        w[:, N // 2] = 0.0
    elif mistake == "seen twice":
        w[:, N // 2] *= 2.0
    got = rounded(rounded(w, dt) @ vp[0, 0] / w.sum(1, keepdims=True), dt)[None, None]
    if mistake is None:
        check_roundings(U[dt], got, ref["out"], squares, ref["weight"])
    else:
        with pytest.raises(AssertionError):
            check_roundings(U[dt], got, ref["out"], squares, ref["weight"])


# ---- on the GPU -----------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("B,T,H,hqk,dk,dv,n", [
    (2, 1, 4, 2, 128, 128, None), (3, 5, 4, 2, 64, 128, [5, 1, 4]), (2, 17, 4, 2, 128, 128, None),
    (2, 32, 2, 1, 64, 64, [32, 19]), (3, 33, 2, 2, 128, 64, None), (2, 200, 2, 1, 128, 128, [200, 131]),
    (1, 515, 4, 2, 64, 128, None), (1, 1500, 2, 1, 128, 128, None), (2, 90, 2, 1, 96, 40, [90, 33])])
@pytest.mark.parametrize("rate", [0.0, 0.01, 0.3])
def test_linear_outputs_are_off_by_their_roundings_alone(sdv, dt, B, T, H, hqk, dk, dv, n, rate):
    q, k, v, g, s = lin.make(dt, B, T, H, hqk, dk, dv, 80, rate=rate)
    o, _ = lin.call(sdv, q, k, v, g, n, s)
    ref = lin.oracle(q, k, v, g, n, s)
    _, squares = mixing.linear_squares(f64(q), f64(k), f64(v), f64(g), 0.3, n or [T] * B, f64(s), CHUNK)
    for b, m in enumerate(n or [T] * B):
        check_roundings(U[dt], f64(o)[b, :m], ref["o"][b, :m], squares[b, :m], ref["o_abs"][b, :m])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("S,hq,hkv,d,page,ctx,masked", [
    (1, 8, 2, 128, 16, 613, False), (1, 8, 1, 64, 64, 5003, False), (17, 16, 2, 256, 64, 777, False),
    (20, 8, 1, 128, 16, 3000, True), (6, 8, 2, 256, 32, 130, True), (32, 4, 4, 64, 16, 100, True),
    (5, 4, 2, 96, 48, 400, False), (3, 4, 2, 128, 16, 2, False)])
def test_attention_outputs_are_off_by_their_roundings_alone(sdv, dt, S, hq, hkv, d, page, ctx, masked):
    q, kp, vp, table = att.make(dt, 1, S, hq, hkv, d, page, [ctx], [S], 81)
    mask = att.words(np.random.default_rng(S), 1, S) if masked else None
    out, _, _ = att.call(sdv, q, kp, vp, table, [ctx], [S], None if mask is None else att.as_i32(mask), d ** -0.5)
    args = (f64(q), f64(kp), f64(vp), table.tolist(), [ctx], [S], mask, d ** -0.5)
    ref = mixing.attention(*args)
    check_roundings(U[dt], f64(out), ref["out"], mixing.attention_squares(*args), ref["weight"])
