"""Refusals of the token-mixing entry points: the host's answers to bad arguments
(CPU only: no compute call is made) and the binding's checks of tensors."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


P = 1 << 20  # an aligned address that nothing follows


def cache(sdv, **kw):
    f = dict(dtype=sdv.SDV_F16, n_pages=4, heads=2, page_size=16, dim=128, max_pages=4, k=P, v=P, table=P)
    f.update(kw)
    return sdv.sdv_kvcache(*[f[n] for n in ("dtype", "n_pages", "heads", "page_size", "dim", "max_pages", "k", "v",
                                            "table")])


BAD_CACHES = [dict(dtype=0), dict(dtype=8), dict(n_pages=0), dict(heads=0), dict(page_size=0), dict(dim=0),
              dict(dim=12), dict(dim=-8), dict(max_pages=0), dict(k=None), dict(v=None), dict(table=None),
              dict(k=P + 8), dict(v=P + 2), dict(table=P + 2)]


def append(sdv, c=None, k=P, v=P, ks=256, vs=256, B=2, T=3, ctx=P, n=P, ws=None):
    c = cache(sdv) if c is None else c
    return sdv.load().sdv_kv_append(ctypes.byref(c), k, v, ks, vs, B, T, ctx, n, ws, None)


def attn(sdv, c=None, q=P, qs=512, B=2, S=3, hq=4, ctx=P, n=P, mask=P, scale=0.1, out=P, lse=P, ws=P, wsb=1 << 40):
    c = cache(sdv) if c is None else c
    return sdv.load().sdv_paged_attn(ctypes.byref(c), q, qs, B, S, hq, ctx, n, mask, scale, out, lse, ws, wsb, None)


def linear(sdv, dtype=16, q=P, k=P, v=P, qs=256, ks=256, vs=512, g=P, tok=1, scale=0.1, B=2, T=5, H=4, hqk=2, dk=128,
           dv=128, n=P, s_in=P, s_out=P, o=P, ws=P, wsb=1 << 40):
    return sdv.load().sdv_linear_attn(dtype, q, k, v, qs, ks, vs, g, tok, scale, B, T, H, hqk, dk, dv, n, s_in, s_out,
                                      o, ws, wsb, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(sdv, kw):
    assert append(sdv, cache(sdv, **kw)) == sdv.SDV_ERR_INVALID_ARG
    assert attn(sdv, cache(sdv, **kw)) == sdv.SDV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 4), dict(ks=255), dict(ks=248), dict(vs=-256),
                                dict(B=0), dict(T=0), dict(T=-1), dict(ctx=None), dict(ctx=P + 1), dict(n=P + 2)])
def test_append_refuses(sdv, kw):
    assert append(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_append_limits(sdv):
    assert append(sdv, ws=P + 4) == sdv.SDV_ERR_WORKSPACE
    assert append(sdv, cache(sdv, dim=264), ks=528, vs=528) == sdv.SDV_ERR_UNSUPPORTED
    assert append(sdv, B=70000) == sdv.SDV_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=P + 2), dict(qs=511), dict(qs=504), dict(B=0), dict(S=0),
                                dict(hq=0), dict(hq=3), dict(ctx=None), dict(ctx=P + 2), dict(n=P + 3),
                                dict(mask=P + 1), dict(out=None), dict(out=P + 8), dict(lse=P + 2),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attention_refuses(sdv, kw):
    assert attn(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_attention_limits(sdv):
    assert attn(sdv, S=33) == sdv.SDV_ERR_UNSUPPORTED
    assert attn(sdv, cache(sdv, dim=264), qs=2048) == sdv.SDV_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=P + 8), dict(wsb=0), dict(wsb=256)):
        assert attn(sdv, **kw) == sdv.SDV_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(k=None), dict(v=None), dict(q=None), dict(q=P + 2), dict(k=P + 8),
                                dict(v=P + 4), dict(qs=100), dict(ks=248), dict(vs=504), dict(vs=513), dict(g=None),
                                dict(g=P + 2), dict(tok=2), dict(tok=-1), dict(scale=float("inf")), dict(B=0),
                                dict(T=0), dict(H=0), dict(hqk=0), dict(hqk=3), dict(dk=0), dict(dk=100), dict(dv=4),
                                dict(n=P + 1), dict(s_in=P + 4), dict(s_out=P + 8), dict(o=P + 2),
                                dict(o=None, s_out=None)])
def test_linear_refuses(sdv, kw):
    assert linear(sdv, **kw) == sdv.SDV_ERR_INVALID_ARG


def test_linear_limits(sdv):
    assert linear(sdv, dk=264, qs=528, ks=528) == sdv.SDV_ERR_UNSUPPORTED
    assert linear(sdv, dv=264, vs=1056) == sdv.SDV_ERR_UNSUPPORTED
    assert linear(sdv, B=70000) == sdv.SDV_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=P + 8), dict(wsb=0)):
        assert linear(sdv, **kw) == sdv.SDV_ERR_WORKSPACE


def test_workspace_sizes(sdv):
    assert sdv.sdv_paged_attn_workspace_bytes(2, 17, 16, 2, 256) >= 256
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 33, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 12),
                (1, 1, 1, 1, 264), (1, 1, 1, 0, 64)):
        assert sdv.sdv_paged_attn_workspace_bytes(*bad) == 0
    assert sdv.sdv_linear_attn_workspace_bytes(2, 17, 4, 128, 128) >= 256
    for bad in ((0, 1, 1, 64, 64), (1, 0, 1, 64, 64), (1, 1, 0, 64, 64), (1, 1, 1, 60, 64), (1, 1, 1, 64, 264)):
        assert sdv.sdv_linear_attn_workspace_bytes(*bad) == 0


def test_the_binding_refuses_cpu_tensors_and_wrong_types(sdv):
    kp = torch.zeros((2, 1, 16, 64), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    rows = torch.zeros((1, 1, 1, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_kv_append(rows, rows, kp, kp, i[None], i, None, None)
    with pytest.raises(TypeError):
        sdv.sdv_kv_append(rows, rows, kp.float(), kp.float(), i[None], i, None, None)
    with pytest.raises(TypeError):
        sdv.sdv_linear_attn(None, rows.float(), rows, i, 1.0, None, None, None, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sdv_linear_attn(rows, rows, rows, torch.zeros(1), 1.0, None, None, None, rows, i)


@pytest.mark.gpu
def test_the_binding_refuses_layouts_and_shapes(sdv):
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    kp, i, table = z(2, 2, 16, 64), torch.zeros(2, dtype=torch.int32, device="cuda"), None
    table = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    q, out = z(2, 3, 4, 64), z(2, 3, 4, 64)
    ws = sdv.paged_attn_workspace(q, kp, table)
    ok = (q, kp, kp, table, i, None, None, 0.1, out, None, ws)

    def change(**kw):
        names = ("q", "k_pages", "v_pages", "table", "ctx", "n_rows", "mask", "scale", "out", "lse", "ws")
        return [kw.get(n, x) for n, x in zip(names, ok)]

    sdv.sdv_paged_attn(*ok)
    torch.cuda.synchronize()
    for kw in (dict(q=z(2, 4, 3, 64).transpose(1, 2)), dict(q=z(3, 2, 4, 64).transpose(0, 1)),
               dict(q=z(2, 3, 4, 128)[..., ::2]), dict(out=z(2, 3, 4, 32)), dict(table=table[:1]), dict(ctx=i[:1]),
               dict(v_pages=z(2, 2, 8, 64)), dict(mask=table), dict(lse=torch.zeros((2, 3), device="cuda"))):
        with pytest.raises(ValueError):
            sdv.sdv_paged_attn(*change(**kw))
    for kw in (dict(q=q.float()), dict(out=out.bfloat16()), dict(ctx=i.long()), dict(mask=torch.zeros((2, 3), device="cuda"))):
        with pytest.raises(TypeError):
            sdv.sdv_paged_attn(*change(**kw))
    with pytest.raises(sdv.SdvError) as e:
        sdv.sdv_paged_attn(*change(ws=ws[:256]))
    assert e.value.status == sdv.SDV_ERR_WORKSPACE
