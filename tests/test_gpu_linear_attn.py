"""sdv_linear_attn on the GPU against the 64-bit oracle.

Tolerances, from the operation alone (u: unit roundoff of the 16-bit type).
Outputs: the score matrix and the state may be rounded to the type once for
their products (u each) and the result is rounded once (u):
  |o - ref| <= (3.1 u + (T + 64) 2^-22) sum |q||terms of the state| + 2^-25.
States are fp32: products of decayed keys are held to 2^-17 at least, decays to
2^-20, sums run in fp32:  |M - ref| <= (2^-16 + (T + 64) 2^-22) sum |terms|.
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


def make(dt, B, T, H, hqk, dk, dv, seed, rate=0.1, per_token=True):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn((B, T, hqk, dk), generator=gen).to(dt)
    k = (torch.randn((B, T, hqk, dk), generator=gen) / dk ** 0.5).to(dt)
    v = torch.randn((B, T, H, dv), generator=gen).to(dt)
    g = -rate * torch.rand((B, T, H) if per_token else (H,), generator=gen)
    s = torch.randn((B, H, dk, dv), generator=gen) * 0.5
    return [x.cuda() for x in (q, k, v, g, s)]


def call(sdv, q, k, v, g, n, s_in, want_state=True, want_o=True, scale=0.3, s_out=None, stream=None):
    B, T, H, dv = v.shape
    o = torch.full((B, T, H, dv), float("nan"), dtype=v.dtype, device="cuda") if want_o else None
    if want_state and s_out is None:
        s_out = torch.full((B, H, k.shape[3], dv), float("nan"), device="cuda")
    ws = sdv.linear_attn_workspace(k, v)
    nt = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    sdv.sdv_linear_attn(q, k, v, g, scale, nt, s_in, s_out if want_state else None, o, ws, stream)
    assert sdv.sdv_last_device_status(ws, stream) == sdv.SDV_OK
    return o, s_out


def oracle(q, k, v, g, n, s, scale=0.3):
    B, T, H, dv = v.shape
    gg = f64(g) if g.dim() == 3 else np.broadcast_to(f64(g), (B, T, H))
    state = np.zeros((B, H, k.shape[3], dv)) if s is None else f64(s)
    return mixing.linear(f64(q), f64(k), f64(v), gg, scale, n or [T] * B, state)


def check(dt, ref, o, state, T):
    if o is not None:
        tol = (3.1 * U[dt] + (T + 64) * 2.0 ** -22) * ref["o_abs"] + 2.0 ** -25
        err = np.abs(f64(o) - ref["o"])
        assert np.all(err <= tol), f"o: worst {np.max(err / tol):.3f} of the bound"
    if state is not None:
        tol = (2.0 ** -16 + (T + 64) * 2.0 ** -22) * ref["state_abs"] + 2.0 ** -126
        err = np.abs(f64(state) - ref["state"])
        assert np.all(err <= tol), f"state: worst {np.max(err / tol):.3f} of the bound"


SHAPES = [
    # dtype, B, T, H, Hqk, Dk, Dv, n, decay per token
    (F16, 1, 1, 1, 1, 128, 128, None, True),
    (BF16, 3, 1, 4, 2, 128, 128, [1, 0, 1], True),
    (F16, 2, 1, 2, 2, 64, 64, None, False),
    (BF16, 2, 2, 4, 1, 64, 128, [2, 1], True),
    (F16, 2, 9, 2, 1, 128, 64, None, False),
    (F16, 4, 17, 4, 2, 128, 128, [17, 0, 5, 16], True),
    (BF16, 3, 31, 3, 3, 64, 128, [31, 30, 1], True),
    (BF16, 2, 32, 2, 2, 128, 128, None, True),
    (F16, 2, 33, 2, 1, 128, 128, [33, 32], True),
    (F16, 1, 63, 2, 2, 64, 64, None, True),
    (BF16, 2, 64, 2, 1, 128, 128, [64, 63], False),
    (F16, 2, 65, 2, 2, 128, 64, None, True),
    (BF16, 3, 200, 2, 1, 128, 128, [200, 129, 0], True),
    (F16, 1, 515, 2, 1, 128, 128, None, True),
    (BF16, 1, 1100, 1, 1, 64, 128, None, False),
    (F16, 2, 700, 2, 2, 64, 64, [1, 700], True),
    # head sizes outside the tensor-core form's
    (F16, 2, 5, 2, 1, 8, 8, [5, 3], True),
    (BF16, 1, 70, 2, 2, 40, 72, None, True),
    (F16, 1, 20, 2, 1, 256, 256, None, True),
    (BF16, 2, 40, 1, 1, 200, 136, [40, 11], False),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_matches_the_oracle(sdv, case):
    dt, B, T, H, hqk, dk, dv, n, per_token = SHAPES[case]
    q, k, v, g, s = make(dt, B, T, H, hqk, dk, dv, 200 + case, per_token=per_token)
    o, state = call(sdv, q, k, v, g, n, s)
    ref = oracle(q, k, v, g, n, s)
    check(dt, ref, o, state, T)
    for b, r in enumerate(n or []):
        assert not f64(o)[b, r:].any()
    # again: the same bits; verify alone, commit alone and in place: the same as together
    o2, state2 = call(sdv, q, k, v, g, n, s)
    assert torch.equal(o, o2) and torch.equal(state, state2)
    only_o, _ = call(sdv, q, k, v, g, n, s, want_state=False)
    check(dt, ref, only_o, None, T)
    _, only_s = call(sdv, None, k, v, g, n, s, want_o=False)
    check(dt, ref, None, only_s, T)
    place = s.clone()
    o3, _ = call(sdv, q, k, v, g, n, place, s_out=place)
    check(dt, ref, o3, place, T)
    # no state in: zeros
    o4, state4 = call(sdv, q, k, v, g, n, None)
    check(dt, oracle(q, k, v, g, n, None), o4, state4, T)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [1, 17, 300])
@pytest.mark.parametrize("kind", ["none", "slow", "fast", "mixed", "resets"])
def test_decays(sdv, dt, T, kind):
    B, H = 2, 3
    q, k, v, g, s = make(dt, B, T, H, 1, 128, 128, 31)
    if kind == "none":
        g.zero_()
    elif kind == "slow":
        g *= 1e-4
    elif kind == "fast":
        g = g * 300 - 5.0
    elif kind == "mixed":
        g[:, ::3] *= 100
        g[:, 1::7] = 0.5  # above 0: taken as 0
        g[:, 2::11] = -1e4
    else:
        g[:, 5::13] = float("-inf")
        s[0] = float("inf")  # dropped by a reset before the first token
        g[0, 0] = float("-inf")
    ref_s = torch.nan_to_num(s, posinf=0.0) if kind == "resets" else s
    o, state = call(sdv, q, k, v, g, None, s)
    check(dt, oracle(q, k, v, g, None, ref_s), o, state, T)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [1, 20, 130])
def test_large_magnitudes_do_not_overflow(sdv, dt, T):
    # scores and states beyond fp16's range, as unnormalised keys give them
    q, k, v, g, s = make(dt, 1, T, 2, 1, 128, 128, 32)
    k, q, v, s = k * 300, q * 20, v * 40, s * 3e6
    o, state = call(sdv, q, k, v, g, None, s, scale=1e-5)
    check(dt, oracle(q, k, v, g, None, s, scale=1e-5), o, state, T)
    # and far below its normal range
    k, q, v, s = k * 1e-5, q, v * 1e-2, s * 1e-15
    o, state = call(sdv, q, k, v, g, None, s, scale=1.0)
    ref = oracle(q, k, v, g, None, s, scale=1.0)
    check(dt, ref, o, state, T)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T,n", [(17, [6, 0]), (150, [70, 129])])
def test_tokens_past_the_count_may_hold_anything(sdv, dt, T, n):
    q, k, v, g, s = make(dt, 2, T, 2, 1, 128, 128, 33)
    want = call(sdv, q, k, v, g, n, s)
    for x in (q, k, v, g):
        for b in range(2):
            x[b, n[b]:] = float("nan")
    got = call(sdv, q, k, v, g, n, s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 12, 100])
def test_counts_are_clamped(sdv, T):
    q, k, v, g, s = make(F16, 2, T, 1, 1, 128, 128, 34)
    want = call(sdv, q, k, v, g, [T, 0], s)
    got = call(sdv, q, k, v, g, [T + 1000, -3], s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("T", [1, 21, 260])
def test_slices_of_a_fused_projection_and_another_stream(sdv, dt, T):
    B, H, hqk, d = 2, 4, 2, 128
    q, k, v, g, s = make(dt, B, T, H, hqk, d, d, 35)
    want = call(sdv, q, k, v, g, None, s)
    fused = torch.cat([x.reshape(B, T, -1) for x in (q, k, v)], -1)
    a, b = hqk * d, 2 * hqk * d
    views = fused[..., :a].view(B, T, hqk, d), fused[..., a:b].view(B, T, hqk, d), fused[..., b:].view(B, T, H, d)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = call(sdv, *views, g, None, s, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cuts", [[100, 1, 1, 17, 64, 130], [1] * 9, [32, 33, 64]])
def test_pieces_of_a_sequence_equal_the_whole(sdv, cuts):
    # a prompt, single tokens and windows, the state carried from call to call
    T = sum(cuts)
    q, k, v, g, s = make(F16, 2, T, 2, 1, 128, 128, 36)
    ref = oracle(q, k, v, g, None, s)
    state, at, outs = s, 0, []
    for c in cuts:
        part = [x[:, at:at + c].contiguous() for x in (q, k, v, g)]
        o, state = call(sdv, *part, None, state)
        outs.append(o)
        at += c
    check(F16, ref, torch.cat(outs, 1), state, T)


def test_a_round_commits_the_accepted_rows_alone(sdv):
    # verify a window, commit the accepted rows: the state of decoding them alone
    B, T = 3, 9
    acc = [9, 1, 4]
    q, k, v, g, s = make(BF16, B, T, 2, 1, 128, 128, 37)
    before = s.clone()
    o, _ = call(sdv, q, k, v, g, None, s, want_state=False)
    assert torch.equal(s, before)
    _, committed = call(sdv, None, k, v, g, acc, s, want_o=False)
    ref = oracle(q, k, v, g, acc, s)
    check(BF16, ref, None, committed, T)
    check(BF16, oracle(q, k, v, g, None, s), o, None, T)
