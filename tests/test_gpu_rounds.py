"""The operators around a batched verify round, together as a serving loop uses them: pages and places
for the windows, norms, positions and the rows into the cache, attention behind the shared prefix, and
the accept of drafted tokens, whose counts move the contexts on -- all on the device.

Each step of each round is held against its oracle on the inputs that it had there, with that operator's
own tolerance; a round captured into a graph and replayed gives the bits of the same round run by itself.
"""
import numpy as np
import pytest
import torch

from oracle import rounds
from tests.test_gpu_paged_attn import check as check_attention
from tests.test_gpu_qk_norm_rope import check as check_rows
from tests.test_gpu_qk_norm_rope import frequencies

pytestmark = pytest.mark.gpu
B, S, HQ, HKV, D, PAGE, V, PREFIX = 6, 5, 8, 2, 64, 16, 500, 70
DT = torch.float16


@pytest.fixture(scope="module")
def sdv():
    from speculative_decode_verify_sdv_gb300 import build, sdv as _sdv
    build.build()
    _sdv.load()
    return _sdv


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Loop:
    """One layer and a head: enough of a model for tokens to depend on everything in front of them."""

    def __init__(self, sdv, pages=120):
        self.sdv = sdv
        gen = torch.Generator().manual_seed(5)
        rand = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).cuda()  # noqa: E731
        self.embed, self.proj = rand(V, 32), rand(32, (HQ + 2 * HKV) * D, std=0.3)
        self.head = rand(HQ * D, V, std=0.2)
        self.qw, self.kw = 1 + 0.2 * rand(D), 1 + 0.2 * rand(D)
        self.rope = sdv.rope_plan(D, 10000.0, "half")
        self.k_pages, self.v_pages = (torch.full((pages, HKV, PAGE, D), float("nan"), dtype=DT, device="cuda")
                                      for _ in range(2))
        front = -(-PREFIX // PAGE)
        self.prefix_table, self.prefix_len = ints(list(range(front))), ints([PREFIX])
        self.k_pages[:front], self.v_pages[:front] = rand(front, HKV, PAGE, D).to(DT), rand(front, HKV, PAGE, D).to(DT)
        self.free, self.n_free = ints(list(range(front, pages)) + [0] * front), ints([pages - front])
        self.table, self.held = torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), ints([0] * B)
        self.ctx, self.anchor = ints([0] * B), ints([7 * b for b in range(B)])
        self.temperature = torch.tensor([1.0, 0.7, 0.0, 1.3, 1.0, 0.5], device="cuda")
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.n, self.drafts = ints([S, S, S - 1, S, 2, S]), z(B, S - 1)
        self.granted, self.positions, self.slots = z(B), z(B, S), z(B, S)
        self.q_in = z(B, S, HQ, D, dt=torch.float32)
        self.kv_in = z(B, S, 2 * HKV, D, dt=torch.float32)
        self.qkv = z(B, S, HQ + 2 * HKV, D, dt=torch.float32)
        self.q, self.out = z(B, S, HQ, D, dt=DT), z(B, S, HQ, D, dt=DT)
        self.lse = z(B, S, HQ, dt=torch.float32)
        self.logits, self.uniforms = z(B, S, V, dt=torch.float32), z(B, S, dt=torch.float32)
        self.accepted, self.next = z(B), z(B)
        need = [sdv.page_assign_workspace(self.ctx), sdv.prefix_attn_workspace(self.q, self.k_pages, self.table),
                sdv.verify_drafts_workspace(self.logits)]
        self.ws = torch.zeros(max(w.numel() for w in need), dtype=torch.uint8, device="cuda")  # one for all

    def state(self):
        return [t for t in vars(self).values() if isinstance(t, torch.Tensor)]

    def round(self):
        s = self.sdv
        s.sdv_page_assign(self.free, self.n_free, self.table, self.held, PAGE, self.ctx, self.n, self.granted,
                          self.positions, self.slots, self.ws)
        tokens = torch.cat([self.anchor[:, None], self.drafts], 1).long()
        self.qkv.copy_((self.embed[tokens] @ self.proj).view(B, S, HQ + 2 * HKV, D))
        q, k, v = self.qkv.split([HQ, HKV, HKV], 2)
        # positions go on behind the prefix; a row that is left out stays below 0
        places = torch.where(self.positions >= 0, self.positions + self.prefix_len, -1).to(torch.int32)
        s.sdv_qk_norm_rope(q, k, v, self.k_pages, self.v_pages, self.qw, self.kw, 1e-6, self.rope, places, self.slots,
                           self.q, self.ws)
        s.sdv_prefix_attn(self.q, self.k_pages, self.v_pages, self.prefix_table, self.prefix_len, self.table, self.ctx,
                          self.granted, None, D ** -0.5, self.out, self.lse, self.ws)
        self.logits.copy_(self.out.float().view(B, S, HQ * D) @ self.head)
        s.sdv_verify_drafts(self.logits, self.temperature, self.drafts, torch.clamp(self.granted - 1, min=0), None,
                            self.uniforms, self.accepted, self.next, self.ws)
        self.ctx += self.accepted + 1
        self.anchor.copy_(self.next)


def f64(t):
    return t.detach().cpu().double().numpy()


def draw(loop, gen):
    """Drafts and random numbers of the next round."""
    loop.uniforms.copy_(torch.rand((B, S), generator=gen))
    likely = loop.logits[:, :S - 1].argmax(-1)
    other = torch.randint(0, V, (B, S - 1), generator=gen).cuda()
    loop.drafts.copy_(torch.where(torch.rand((B, S - 1), generator=gen).cuda() < 0.6, likely, other))


def test_rounds_step_by_step(sdv):
    loop = Loop(sdv)
    gen = torch.Generator().manual_seed(9)
    for _ in range(4):
        draw(loop, gen)
        before = {k: v.clone() for k, v in vars(loop).items() if isinstance(v, torch.Tensor)}
        loop.round()
        assert sdv.sdv_last_device_status(loop.ws) == sdv.SDV_OK
        ctx, n = before["ctx"].tolist(), before["n"].tolist()
        want = rounds.assign(before["free"].tolist(), int(before["n_free"]), before["table"].tolist(),
                             before["held"].tolist(), PAGE, ctx, n, S)
        assert loop.table.tolist() == want["table"] and loop.slots.tolist() == want["slots"]
        assert loop.granted.tolist() == want["granted"] == n
        live = loop.positions.cpu() >= 0
        pos = f64(loop.positions) + PREFIX
        for rows, weight, got in ((loop.qkv[:, :, :HQ], loop.qw, loop.q),
                                  (loop.qkv[:, :, HQ:HQ + HKV], loop.kw, None)):
            y = rounds.norm_rope(f64(rows), f64(weight), 1e-6, pos, frequencies(loop.rope), 1.0, "half")
            size = np.broadcast_to(np.abs(y).max(-1, keepdims=True) * 1.5, y.shape)
            if got is None:
                flat = loop.k_pages.transpose(1, 2).reshape(-1, HKV, D).cpu()
                got = torch.zeros((B, S, HKV, D), dtype=DT)
                got[live] = flat[loop.slots.cpu()[live].long()]
            check_rows(DT, got.cpu()[live], y[live.numpy()], size[live.numpy()])
        ref = rounds.prefix_attention(f64(loop.q), f64(loop.k_pages), f64(loop.v_pages), loop.prefix_table.tolist(),
                                      PREFIX, loop.table.tolist(), ctx, n, None, D ** -0.5)
        check_attention(DT, ref, loop.out, loop.lse, D)
        logits, t, u, d = (x.cpu().numpy() for x in (loop.logits, loop.temperature, loop.uniforms, before["drafts"]))
        for b in range(B):
            accepted, token, margin = rounds.verify(logits[b], float(t[b]), d[b], n[b] - 1, None, u[b])
            assert margin < 2.0 ** -34 or (int(loop.accepted[b]), int(loop.next[b])) == (accepted, token)
            assert int(loop.ctx[b]) == ctx[b] + int(loop.accepted[b]) + 1
    # the requests end: every page is back
    sdv.sdv_page_assign(loop.free, loop.n_free, loop.table, loop.held, PAGE, ints([0] * B), ints([0] * B), None, None,
                        None, loop.ws)
    front = loop.prefix_table.numel()
    assert int(loop.n_free) == 120 - front and not loop.held.any()
    assert sorted(loop.free.tolist()[:120 - front]) == list(range(front, 120))


def test_a_captured_round_is_the_round(sdv):
    alone, replayed = Loop(sdv), Loop(sdv)
    draw(alone, torch.Generator().manual_seed(3))
    draw(replayed, torch.Generator().manual_seed(3))
    kept = [t.clone() for t in replayed.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.round()  # (the first calls set kernels' attributes up)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.round()
    for t, k in zip(replayed.state(), kept):
        t.copy_(k)
    for step in range(3):
        gens = [torch.Generator().manual_seed(20 + step) for _ in range(2)]
        draw(alone, gens[0])
        draw(replayed, gens[1])
        alone.round()
        graph.replay()
        for name in ("ctx", "anchor", "accepted", "next", "slots", "table", "held", "out", "lse", "logits"):
            assert torch.equal(getattr(alone, name), getattr(replayed, name)), name
    assert sdv.sdv_last_device_status(replayed.ws) == sdv.SDV_OK


def test_a_shortage_of_pages_leaves_rows_out(sdv):
    """Sequences without a page have no rows in this round: nothing of theirs is stored or attended to, the
    others go on as they were."""
    loop = Loop(sdv)
    loop.n_free.fill_(3)  # of six sequences' pages
    draw(loop, torch.Generator().manual_seed(4))
    loop.round()
    assert loop.granted.tolist() == [S, S, S - 1, 0, 0, 0]
    assert not loop.out[3:].any() and torch.isneginf(loop.lse[3:]).all()
    assert torch.isfinite(loop.out).all() and int(loop.n_free) == 0
    assert sdv.sdv_last_device_status(loop.ws) == sdv.SDV_OK
