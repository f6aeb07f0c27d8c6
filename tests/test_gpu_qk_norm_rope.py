"""sdv_qk_norm_rope on the GPU against the 64-bit oracle.

Tolerances: the result is rounded once to the 16-bit type (u of its value); before that, in
fp32, the norm's sum and root cost (dim + 6) 2^-24 of a value, the rotation three roundings
of each term and an angle that is off by up to pi 2^-24 (32 bits of a turn, rounded to a
float, and the sine's own error): 2^-21 of the pair's length covers them.
"""
import numpy as np
import pytest
import torch

from oracle import rounds

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def f64(t):
    return t.detach().cpu().double().numpy()


def frequencies(plan):
    steps = [x % 2 ** 64 for x in plan.steps.tolist()]
    return [s / 2.0 ** 64 * 2 * np.pi for s in steps]


def make(sdv, ty, dt, B, T, hq, hkv, d, page, seed, dead=True, far=0):
    gen = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((B, T, hq + 2 * hkv, d), generator=gen) * 1.5).to(ty).cuda()
    pages = -(-B * T // page) + 2
    kp, vp = (torch.full((pages, hkv, page, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen)[:B * T].reshape(B, T).to(torch.int32)
    pos = torch.randint(0, 4000, (B, T), generator=gen).to(torch.int32) + far
    if dead:
        pos[torch.rand((B, T), generator=gen) < 0.2] = -1
        slots[torch.rand((B, T), generator=gen) < 0.2] = -1
    w = [(1 + 0.3 * torch.randn(d, generator=gen)).cuda() for _ in range(2)]
    return qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], kp, vp, w[0], w[1], pos.cuda(), slots.cuda()


def check(dt, got, want, length):
    """length: per element the largest magnitude of its pair and of its own value."""
    tol = (U[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -20 * length + 2.0 ** -25
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3f} of the bound"


def run_and_check(sdv, ty, dt, B, T, hq, hkv, d, page, plan, norm_q, norm_k, seed, far=0):
    q, k, v, kp, vp, qw, kw, pos, slots = make(sdv, ty, dt, B, T, hq, hkv, d, page, seed, far=far)
    eps = 1e-5
    out = torch.full((B, T, hq, d), 7.0, dtype=dt, device="cuda")
    sdv.sdv_qk_norm_rope(q, k, v, kp, vp, qw if norm_q else None, kw if norm_k else None, eps, plan, pos, slots, out,
                         None)
    freq, amp, layout = ([], 1.0, "half") if plan is None else \
        (frequencies(plan), plan.amplitude, "pairs" if plan.layout else "half")
    p = f64(pos)
    live = p >= 0
    refs = []
    for x, w, on in ((q, qw, norm_q), (k, kw, norm_k)):
        y = rounds.norm_rope(f64(x), f64(w) if on else None, eps, p, freq, amp, layout)
        still = rounds.norm_rope(f64(x), f64(w) if on else None, eps, p, [], 1.0, layout)
        refs.append((y, np.broadcast_to(np.abs(still).max(-1, keepdims=True) * max(1.0, amp), y.shape)))
    check(dt, out.cpu()[torch.as_tensor(live)], refs[0][0][live], refs[0][1][live])
    assert torch.all(out.cpu()[torch.as_tensor(~live)] == 7.0)  # rows that are left out stay as they were
    stored = live & (slots.cpu().numpy() >= 0)
    at = torch.as_tensor(slots.cpu().numpy()[stored]).long()
    flat = lambda t: t.cpu().transpose(1, 2).reshape(-1, hkv, d)  # noqa: E731
    check(dt, flat(kp)[at], refs[1][0][stored], refs[1][1][stored])
    assert torch.equal(flat(vp)[at], v.cpu()[torch.as_tensor(stored)].to(dt))
    # every other slot is untouched
    rest = torch.ones(kp.shape[0] * page, dtype=torch.bool)
    rest[at] = False
    assert torch.isnan(flat(kp)[rest]).all() and torch.isnan(flat(vp)[rest]).all()
    return out


SHAPES = [
    # in, cache, B, T, Hq, Hkv, dim, page, rot, layout
    (F32, F16, 1, 1, 32, 8, 128, 16, 128, "half"),
    (BF16, BF16, 3, 17, 16, 2, 256, 64, 64, "pairs"),
    (F16, F16, 2, 9, 4, 4, 64, 16, 64, "half"),
    (F32, BF16, 2, 5, 6, 3, 80, 7, 80, "half"),       # 40 pairs: chunks of eight
    (F16, F16, 2, 5, 6, 3, 80, 7, 40, "half"),        # 20 pairs: not
    (BF16, BF16, 2, 3, 5, 1, 96, 5, 20, "half"),
    (F32, F16, 1, 4, 3, 1, 8, 1, 8, "half"),
    (F16, F16, 1, 4, 3, 1, 8, 4, 2, "pairs"),
    (F32, BF16, 2, 2, 2, 1, 40, 3, 14, "pairs"),
    (F16, F16, 1, 3, 2, 2, 248, 6, 240, "half"),
    (BF16, BF16, 2, 3, 2, 2, 256, 16, 256, "half"),
    (F32, F16, 1, 2, 2, 2, 24, 16, 24, "half"),
    (F16, F16, 7, 700, 8, 2, 64, 16, 32, "half"),     # more rows than warps
    (F32, BF16, 300, 1, 4, 1, 128, 16, 128, "pairs"),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_against_the_oracle(sdv, case):
    ty, dt, B, T, hq, hkv, d, page, rot, layout = SHAPES[case]
    plan = sdv.rope_plan(rot, 10000.0, layout)
    run_and_check(sdv, ty, dt, B, T, hq, hkv, d, page, plan, True, True, case)
    run_and_check(sdv, ty, dt, B, T, hq, hkv, d, page, plan, case % 2 == 0, case % 2 == 1, case + 50)


@pytest.mark.parametrize("norm", [False, True])
def test_without_rotation(sdv, norm):
    run_and_check(sdv, F32, F16, 3, 5, 4, 2, 128, 16, None, norm, norm, 3)


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 5000])
def test_far_positions(sdv, far):
    """The angle of a far position is as exact as that of a near one."""
    for layout in ("half", "pairs"):
        run_and_check(sdv, F32, F16, 2, 5, 4, 2, 128, 16, sdv.rope_plan(128, 10000.0, layout), True, True, 4, far=far)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("ramp", dict(factor=16.0, trained=4096, low=1.0, high=32.0)),
                                        ("bands", dict(factor=8.0, trained=8192, low=1.0, high=4.0))])
def test_scaled(sdv, scaling, kw):
    plan = sdv.rope_plan(64, 500000.0, "half", scaling=scaling, **kw)
    assert (plan.amplitude > 1.0) == (scaling == "ramp")
    run_and_check(sdv, F16, F16, 2, 5, 4, 2, 128, 16, plan, True, True, 5, far=60000)


def test_parts_of_the_call(sdv):
    """Queries alone, keys and values alone, in place: the same bits as the whole call's."""
    q, k, v, kp, vp, qw, kw, pos, slots = make(sdv, F16, F16, 2, 6, 8, 2, 64, 16, 9)
    plan = sdv.rope_plan(64, 10000.0, "half")
    out = torch.zeros((2, 6, 8, 64), dtype=F16, device="cuda")
    sdv.sdv_qk_norm_rope(q, k, v, kp, vp, qw, kw, 1e-6, plan, pos, slots, out, None)
    kp2, vp2, out2 = torch.full_like(kp, float("nan")), torch.full_like(vp, float("nan")), torch.zeros_like(out)
    sdv.sdv_qk_norm_rope(q, None, None, kp2, vp2, qw, None, 1e-6, plan, pos, None, out2, None)
    assert torch.equal(out2, out) and torch.isnan(kp2).all()
    sdv.sdv_qk_norm_rope(None, k, v, kp2, vp2, None, kw, 1e-6, plan, pos, slots, None, None)
    assert torch.equal(kp2.view(torch.int16), kp.view(torch.int16))
    assert torch.equal(vp2.view(torch.int16), vp.view(torch.int16))
    same = q.contiguous()
    sdv.sdv_qk_norm_rope(same, None, None, kp, vp, qw, None, 1e-6, plan, pos, None, same, None)
    live = (pos >= 0)
    assert torch.equal(same[live], out[live]) and torch.equal(same[~live], q[~live])


def test_slots_past_the_cache_are_reported(sdv):
    q, k, v, kp, vp, qw, kw, pos, slots = make(sdv, F16, F16, 1, 3, 2, 2, 64, 16, 11, dead=False)
    slots[0, 1] = kp.shape[0] * 16
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.zeros((1, 3, 2, 64), dtype=F16, device="cuda")
    sdv.sdv_qk_norm_rope(q, k, v, kp, vp, None, None, 0.0, None, pos, slots, out, ws)
    assert sdv.sdv_last_device_status(ws) == sdv.SDV_ERR_INVALID_ARG
    assert torch.equal(out, q)
    flat = kp.transpose(1, 2).reshape(-1, 2, 64)
    assert (~torch.isnan(flat).any(-1).any(-1)).sum() == 2


def test_infinities_stay_in_their_rows_and_heads(sdv):
    q, k, v, kp, vp, qw, kw, pos, slots = make(sdv, F32, F16, 1, 3, 2, 2, 64, 16, 12, dead=False)
    q[0, 1, 0, 40] = float("inf")  # behind the rotated part
    plan = sdv.rope_plan(32, 10000.0, "half")
    out = torch.zeros((1, 3, 2, 64), dtype=F16, device="cuda")
    sdv.sdv_qk_norm_rope(q, k, v, kp, vp, None, None, 0.0, plan, pos, slots, out, None)
    odd = ~torch.isfinite(out)
    assert odd.sum() == 1 and odd[0, 1, 0, 40]


def test_captured_and_on_another_stream(sdv):
    q, k, v, kp, vp, qw, kw, pos, slots = make(sdv, F32, BF16, 2, 7, 8, 2, 128, 16, 13)
    plan = sdv.rope_plan(128, 10000.0, "pairs")
    out = torch.zeros((2, 7, 8, 128), dtype=BF16, device="cuda")
    args = (q, k, v, kp, vp, qw, kw, 1e-6, plan, pos, slots)
    sdv.sdv_qk_norm_rope(*args, out, None)
    want, wk = out.clone(), kp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdv.sdv_qk_norm_rope(*args, out, None)
    out.zero_()
    kp.fill_(float("nan"))
    graph.replay()
    assert torch.equal(out, want) and torch.equal(kp.view(torch.int16), wk.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    sdv.sdv_qk_norm_rope(*args, out, None, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
