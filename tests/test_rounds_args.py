"""Refusals of the entry points around a round: the host's answers to bad arguments (CPU only: no
compute call is made), the binding's checks of tensors, and the rotation's frequencies."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


P = 1 << 20  # an aligned address that nothing follows
NAN, INF = float("nan"), float("inf")


def pages(sdv, n_pages=64, page=16, most=8, free=P, n_free=P, table=P, held=P, B=2, T=3, ctx=P, n=P, granted=P,
          positions=P, slots=P, ws=P, wsb=1 << 40):
    pool = sdv.sdv_pagepool(n_pages, page, most, free, n_free, table, held)
    return sdv.load().sdv_page_assign(ctypes.byref(pool), B, T, ctx, n, granted, positions, slots, ws, wsb, None)


def cache(sdv, **kw):
    f = dict(dtype=sdv.SDV_F16, n_pages=4, heads=2, page_size=16, dim=128, max_pages=4, k=P, v=P, table=P)
    f.update(kw)
    return sdv.sdv_kvcache(*[f[n] for n in ("dtype", "n_pages", "heads", "page_size", "dim", "max_pages", "k", "v",
                                            "table")])


def rope(sdv, c=None, ty=16, q=P, k=P, v=P, qs=512, ks=256, vs=256, B=2, T=3, hq=4, qw=P, kw=P, eps=1e-6, layout=0,
         rot=128, amplitude=1.0, steps=P, plan=True, positions=P, slots=P, out=P, ws=P):
    c = cache(sdv) if c is None else c
    r = sdv.sdv_rope(layout, rot, amplitude, steps)
    return sdv.load().sdv_qk_norm_rope(ctypes.byref(c), ty, q, k, v, qs, ks, vs, B, T, hq, qw, kw, eps,
                                       ctypes.byref(r) if plan else None, positions, slots, out, ws, None)


def prefix(sdv, c=None, ptable=P, ppages=3, plen=P, q=P, qs=512, B=2, S=3, hq=4, ctx=P, n=P, mask=P, scale=0.1, out=P,
           lse=P, ws=P, wsb=1 << 40):
    c = cache(sdv) if c is None else c
    return sdv.load().sdv_prefix_attn(ctypes.byref(c), ptable, ppages, plen, q, qs, B, S, hq, ctx, n, mask, scale, out,
                                      lse, ws, wsb, None)


def verify(sdv, ty=32, logits=P, stride=1000, B=2, S=3, V=1000, temp=P, drafts=P, n=P, probs=P, u=P, accepted=P, nxt=P,
           ws=P, wsb=1 << 40):
    return sdv.load().sdv_verify_drafts(ty, logits, stride, B, S, V, temp, drafts, n, probs, u, accepted, nxt, ws, wsb,
                                        None)


@pytest.mark.parametrize("kw", [dict(n_pages=0), dict(page=0), dict(most=0), dict(free=None), dict(n_free=None),
                                dict(table=None), dict(held=None), dict(ctx=None), dict(B=0), dict(T=0), dict(T=-3),
                                dict(free=P + 1), dict(n_free=P + 2), dict(table=P + 3), dict(held=P + 2),
                                dict(ctx=P + 1), dict(n=P + 2), dict(granted=P + 1), dict(positions=P + 2),
                                dict(slots=P + 3)])
def test_pages_refuse(sdv, kw):
    assert pages(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_pages_limits(sdv):
    for kw in (dict(B=70000), dict(n_pages=1 << 28), dict(most=1 << 28)):
        assert pages(sdv, **kw) == sdv.SDV_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=P + 4), dict(wsb=0), dict(wsb=300)):
        assert pages(sdv, **kw) == sdv.SDV_ERR_WORKSPACE
    assert sdv.sdv_page_assign_workspace_bytes(0) == 0 and sdv.sdv_page_assign_workspace_bytes(70000) == 0
    assert sdv.sdv_page_assign_workspace_bytes(7) >= 256


@pytest.mark.parametrize("kw", [dict(ty=0), dict(ty=17), dict(q=None), dict(q=None, out=None, k=None, v=None),
                                dict(k=None), dict(v=None), dict(out=None), dict(q=P + 8), dict(k=P + 8),
                                dict(v=P + 2), dict(out=P + 8), dict(qs=511), dict(qs=504), dict(ks=248), dict(vs=0),
                                dict(B=0), dict(T=0), dict(hq=0), dict(qw=P + 4), dict(kw=P + 8), dict(eps=-1.0),
                                dict(eps=NAN), dict(eps=INF), dict(layout=2), dict(rot=0), dict(rot=7), dict(rot=130),
                                dict(amplitude=NAN), dict(steps=None), dict(steps=P + 4), dict(positions=None),
                                dict(positions=P + 2), dict(slots=None), dict(slots=P + 1)])
def test_norm_and_rotation_refuse(sdv, kw):
    assert rope(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=32), dict(dim=12), dict(dim=0), dict(n_pages=0),
                                dict(heads=0), dict(page_size=0), dict(k=None), dict(v=None), dict(k=P + 8)])
def test_norm_and_rotation_refuse_caches(sdv, kw):
    assert rope(sdv, cache(sdv, **kw)) == sdv.SDV_ERR_INVALID_ARG


def test_norm_and_rotation_limits(sdv):
    assert rope(sdv, ws=P + 4) == sdv.SDV_ERR_WORKSPACE
    assert rope(sdv, cache(sdv, dim=264), qs=2048, ks=528, vs=528) == sdv.SDV_ERR_UNSUPPORTED
    assert rope(sdv, hq=5000, qs=5000 * 128) == sdv.SDV_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(ptable=None), dict(ptable=P + 2), dict(ppages=0), dict(plen=None),
                                dict(plen=P + 1), dict(q=None), dict(q=P + 2), dict(qs=511), dict(B=0), dict(S=0),
                                dict(hq=0), dict(hq=3), dict(ctx=None), dict(n=P + 3), dict(mask=P + 1),
                                dict(out=None), dict(out=P + 8), dict(lse=P + 2), dict(scale=NAN)])
def test_prefix_refuses(sdv, kw):
    assert prefix(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_prefix_limits(sdv):
    assert prefix(sdv, cache(sdv, table=None)) == sdv.SDV_ERR_INVALID_ARG
    assert prefix(sdv, S=33) == sdv.SDV_ERR_UNSUPPORTED
    assert prefix(sdv, cache(sdv, dim=264), qs=2048) == sdv.SDV_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=P + 8), dict(wsb=0), dict(wsb=256)):
        assert prefix(sdv, **kw) == sdv.SDV_ERR_WORKSPACE
    assert sdv.sdv_prefix_attn_workspace_bytes(4, 3, 8, 2, 128) >= sdv.sdv_paged_attn_workspace_bytes(4, 3, 8, 2, 128)
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 33, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 12)):
        assert sdv.sdv_prefix_attn_workspace_bytes(*bad) == 0


def test_prefix_workspaces_hold_smaller_calls(sdv):
    for heads, group, dim in ((1, 1, 64), (8, 4, 128), (2, 8, 256), (3, 5, 80), (1, 32, 128)):
        most = sdv.sdv_prefix_attn_workspace_bytes(20, 6, heads * group, heads, dim)
        for B in (1, 2, 7, 13, 19, 20):
            for S in (1, 2, 5, 6):
                assert sdv.sdv_prefix_attn_workspace_bytes(B, S, heads * group, heads, dim) <= most


@pytest.mark.parametrize("kw", [dict(ty=0), dict(ty=8), dict(logits=None), dict(logits=P + 2), dict(ty=16, logits=P + 1),
                                dict(stride=999), dict(B=0), dict(S=0), dict(V=0), dict(temp=None), dict(temp=P + 2),
                                dict(drafts=None), dict(drafts=P + 1), dict(n=P + 2), dict(probs=P + 2), dict(u=None),
                                dict(u=P + 3), dict(accepted=None), dict(accepted=P + 2), dict(nxt=None),
                                dict(nxt=P + 1)])
def test_drafts_refuse(sdv, kw):
    assert verify(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_drafts_limits(sdv):
    for kw in (dict(S=33), dict(V=(1 << 24) + 1, stride=1 << 25), dict(B=(1 << 24) + 1, S=1), dict(B=1 << 20, S=32, V=1 << 20, stride=1 << 20)):
        assert verify(sdv, **kw) == sdv.SDV_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=P + 8), dict(wsb=256)):
        assert verify(sdv, **kw) == sdv.SDV_ERR_WORKSPACE
    for bad in ((0, 1, 10), (1, 0, 10), (1, 33, 10), (1, 1, 0), (1, 1, 1 << 25)):
        assert sdv.sdv_verify_drafts_workspace_bytes(*bad) == 0
    assert sdv.sdv_verify_drafts_workspace_bytes(3, 2, 1000) <= sdv.sdv_verify_drafts_workspace_bytes(4, 2, 1000)


# ---- frequencies --------------------------------------------------------------------------

def radians(steps):
    return [s / 2.0 ** 64 * 2 * math.pi for s in steps]


def test_plain_frequencies(sdv):
    steps, amplitude = sdv.sdv_rope_steps(64, 10000.0)
    assert amplitude == 1.0 and len(steps) == 32
    # a step is rounded to 2^-64 turns: half of one against f / (2 pi)
    for i, f in enumerate(radians(steps)):
        want = 10000.0 ** (-2 * i / 64)
        assert abs(f - want) <= want * 2.0 ** -50 + 2 * math.pi * 2.0 ** -64


def test_scaled_frequencies(sdv):
    plain = radians(sdv.sdv_rope_steps(64, 500000.0)[0])
    linear, a = sdv.sdv_rope_steps(64, 500000.0, sdv.SDV_ROPE_LINEAR, 4.0)
    # both are rounded to steps: half of one, and half of one divided by the factor
    step = 2 * math.pi * 2.0 ** -64
    assert a == 1.0 and all(abs(f - p / 4) <= p * 2.0 ** -48 + step for f, p in zip(radians(linear), plain))
    base, a = sdv.sdv_rope_steps(64, 500000.0, sdv.SDV_ROPE_BASE, 4.0)
    # the fastest pair stays, the slowest is divided by the factor
    assert a == 1.0 and base[0] == sdv.sdv_rope_steps(64, 500000.0)[0][0]
    assert abs(radians(base)[-1] - plain[-1] / 4) <= plain[-1] * 2.0 ** -40
    for kind, amplitude in ((sdv.SDV_ROPE_RAMP, 0.1 * math.log(4.0) + 1.0), (sdv.SDV_ROPE_BANDS, 1.0)):
        ramp, a = sdv.sdv_rope_steps(64, 500000.0, kind, 4.0, 8192, 1.0, 32.0)
        assert abs(a - amplitude) <= 2.0 ** -24 * amplitude
        ramp = radians(ramp)
        ratio = [p / f for f, p in zip(ramp, plain)]
        for r, p in zip(ratio, plain):
            turns = 8192 * p / (2 * math.pi)
            if turns < 0.9:
                assert abs(r - 4.0) < 1e-9
            assert 1 - 1e-9 <= r <= 4 + 1e-9
        assert abs(ratio[0] - 1.0) < 1e-9 and all(b > a - 1e-9 for a, b in zip(ratio, ratio[1:]))


@pytest.mark.parametrize("args", [(0, 1e4), (7, 1e4), (64, 1.0), (64, NAN), (64, INF), (64, 1e4, 9, 2.0),
                                  (64, 1e4, -1, 2.0), (64, 1e4, 1, 0.5), (64, 1e4, 1, NAN), (2, 1e4, 2, 2.0),
                                  (64, 1e4, 3, 2.0, 0), (64, 1e4, 3, 2.0, 8192, 0.0), (64, 1e4, 4, 2.0, 8192, 2.0, 2.0),
                                  (64, 1e4, 4, 2.0, 8192, 2.0, INF)])
def test_frequencies_refuse(sdv, args):
    with pytest.raises(sdv.SdvError) as e:
        sdv.sdv_rope_steps(*args)
    assert e.value.status == sdv.SDV_ERR_INVALID_ARG


def test_the_binding_refuses(sdv):
    i = torch.zeros(1, dtype=torch.int32)
    kp = torch.zeros((2, 1, 16, 64), dtype=torch.float16)
    rows = torch.zeros((1, 1, 1, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_page_assign(i, i, i[None], i, 16, i, None, None, None, None, i)
    with pytest.raises(ValueError):
        sdv.sdv_page_assign(i, i, i, i, 16, i, None, None, None, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_qk_norm_rope(rows, rows, rows, kp, kp, None, None, 0.0, None, i[None], i[None], rows, None)
    with pytest.raises(TypeError):
        sdv.sdv_qk_norm_rope(rows.bfloat16(), None, None, kp, kp, None, None, 0.0, None, i[None], None, rows, None)
    with pytest.raises(ValueError):
        sdv.sdv_qk_norm_rope(None, None, None, kp, kp, None, None, 0.0, None, i[None], None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_prefix_attn(rows, kp, kp, i, i, i[None], i, None, None, 1.0, rows, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_verify_drafts(torch.zeros((1, 1, 5)), torch.ones(1), None, None, None, torch.ones((1, 1)), i, i, i)
    with pytest.raises(TypeError):
        sdv.sdv_verify_drafts(torch.zeros((1, 1, 5)).double(), torch.ones(1), None, None, None, torch.ones((1, 1)), i,
                              i, i)
    with pytest.raises(ValueError):
        sdv.rope_plan(64, 1e4, "middle", device="cpu")
    with pytest.raises(ValueError):
        sdv.rope_plan(64, 1e4, "half", scaling="other", device="cpu")
