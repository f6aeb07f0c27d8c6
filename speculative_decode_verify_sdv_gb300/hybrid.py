"""A small hybrid target -- linear-attention and attention layers under a verify
head -- decoded by speculative rounds: an example of the token mixers in use.

A round verifies [a0] + drafts in one forward over S = k + 1 rows:

* an attention layer appends the window's keys and values behind the context
  (``sdv_kv_append``) and attends to the cache (``sdv_paged_attn``).  A rejected
  row stays in the cache behind the context, where the next round writes;
* a linear-attention layer computes the window's outputs from the state before it
  (``sdv_linear_attn`` without state_out).  The state cannot take a token back,
  so it advances after the accept, by the accepted rows alone: the same call
  without o, its token count on the device;
* ``sdv_verify_head`` gives the argmaxes, the accepted drafts and the next a0.

The context and the counts stay on the device, so a round has one read-back.
The body around the mixers (embedding, norms, residuals) is plain PyTorch and the
weights are random: ``python -m speculative_decode_verify_sdv_gb300.hybrid``.
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import sdv
from .specdec import PAD, NgramDrafter

WINDOW = 32  # rows of one attention call, and of one projection


class _Linear:
    """A quantised projection of up to WINDOW rows at once."""

    def __init__(self, n: int, k: int, gen: torch.Generator, device):
        self.w = sdv.quantize(torch.randn((n, k), generator=gen).to(device) * k ** -0.5, sdv.SDV_Q8)
        self.ws = sdv.workspace(sdv.SDV_OP_QLINEAR, n, k, WINDOW, device=device)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        y = torch.empty((x.shape[0], self.w.n), dtype=torch.float32, device=x.device)
        for t in range(0, x.shape[0], WINDOW):
            rows = x[t:t + WINDOW]
            sdv.sdv_qlinear(self.w, rows, rows.shape[0], y[t:t + WINDOW], self.ws)
        return y


class _AttentionLayer:
    """Grouped-query attention over a paged cache of one sequence."""

    def __init__(self, d: int, pages: int, gen, device, heads=8, kv_heads=2, dim=64, page=16):
        self.hq, self.hkv, self.dim = heads, kv_heads, dim
        self.qkv = _Linear((heads + 2 * kv_heads) * dim, d, gen, device)
        self.out = _Linear(d, heads * dim, gen, device)
        shape = (pages, kv_heads, page, dim)
        self.k = torch.zeros(shape, dtype=torch.float16, device=device)
        self.v = torch.zeros(shape, dtype=torch.float16, device=device)
        self.table = torch.randperm(pages, generator=gen).to(torch.int32).to(device)[None]
        probe = torch.empty((1, WINDOW, heads, dim), dtype=torch.float16, device=device)
        self.ws = sdv.paged_attn_workspace(probe, self.k, self.table)

    def __call__(self, x: torch.Tensor, ctx: torch.Tensor) -> torch.Tensor:
        T, hq, hkv, dim = x.shape[0], self.hq, self.hkv, self.dim
        rows = self.qkv(x).half().view(1, T, hq + 2 * hkv, dim)  # q, k and v are slices of one tensor
        q, k, v = rows[:, :, :hq], rows[:, :, hq:hq + hkv], rows[:, :, hq + hkv:]
        sdv.sdv_kv_append(k, v, self.k, self.v, self.table, ctx, None, self.ws)
        o = torch.empty((1, T, hq, dim), dtype=torch.float16, device=x.device)
        for t in range(0, T, WINDOW):
            sdv.sdv_paged_attn(q[:, t:t + WINDOW], self.k, self.v, self.table, ctx + t, None, None, dim ** -0.5,
                               o[:, t:t + WINDOW], None, self.ws)
        return self.out(o.view(T, hq * dim))

    def commit(self, n: torch.Tensor) -> None:
        """Nothing to do: the context moves on."""


class _LinearLayer:
    """Linear attention with one fixed decay per head and one state."""

    def __init__(self, d: int, gen, device, heads=8, qk_heads=4, dim=64):
        self.h, self.hqk, self.dim = heads, qk_heads, dim
        self.qkv = _Linear((heads + 2 * qk_heads) * dim, d, gen, device)
        self.out = _Linear(d, heads * dim, gen, device)
        self.decay = -torch.logspace(-3, -0.5, heads).to(device)
        self.state = torch.zeros((1, heads, dim, dim), dtype=torch.float32, device=device)
        self.kv = None
        self.wss: dict[int, torch.Tensor] = {}  # per length

    def __call__(self, x: torch.Tensor, ctx: torch.Tensor) -> torch.Tensor:
        T, h, hqk, dim = x.shape[0], self.h, self.hqk, self.dim
        rows = self.qkv(x).half().view(1, T, h + 2 * hqk, dim)
        q, k, v = rows[:, :, :hqk], rows[:, :, hqk:2 * hqk], rows[:, :, 2 * hqk:]
        if T not in self.wss:
            self.wss[T] = sdv.linear_attn_workspace(k, v)
        self.kv = k, v
        o = torch.empty((1, T, h, dim), dtype=torch.float16, device=x.device)
        sdv.sdv_linear_attn(q, k, v, self.decay, 1.0 / dim, None, self.state, None, o, self.wss[T])
        return self.out(o.view(T, h * dim))

    def commit(self, n: torch.Tensor) -> None:
        """The state takes the first n rows of the last window, in place."""
        k, v = self.kv
        sdv.sdv_linear_attn(None, k, v, self.decay, 0.0, n, self.state, self.state, None, self.wss[k.shape[1]])


class HybridTarget:
    """One sequence through a hybrid body and a verify head."""

    def __init__(self, vocab: int = 4096, d: int = 256, layers: Sequence[str] = ("linear", "linear", "attention"),
                 max_tokens: int = 4096, seed: int = 0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.device = device
        self.embed = torch.randn((vocab, d), generator=gen).to(device)
        self.layers = [_AttentionLayer(d, -(-max_tokens // 16), gen, device) if kind == "attention" else
                       _LinearLayer(d, gen, device) for kind in layers]
        self.head = sdv.quantize(torch.randn((vocab, d), generator=gen).to(device) * 4 * d ** -0.5, sdv.SDV_Q8)
        self.head_ws = sdv.workspace(sdv.SDV_OP_VERIFY_HEAD, vocab, d, WINDOW, device=device)
        self.ctx = torch.zeros(1, dtype=torch.int32, device=device)
        self.result = torch.empty(2, dtype=torch.int32, device=device)  # accepted, next a0
        self.argmax = torch.empty(WINDOW, dtype=torch.int32, device=device)

    def _body(self, tokens: torch.Tensor) -> torch.Tensor:
        x = self.embed[tokens]
        for layer in self.layers:
            x = x + layer(torch.nn.functional.rms_norm(x, x.shape[1:]).half(), self.ctx)
        return torch.nn.functional.rms_norm(x, x.shape[1:]).half()

    def _commit(self, n: torch.Tensor) -> None:
        for layer in self.layers:
            layer.commit(n)
        self.ctx += n

    def prefill(self, prompt: Sequence[int], logits: torch.Tensor | None = None) -> int:
        """The whole prompt enters caches and states; returns the first a0."""
        x = self._body(torch.tensor(list(prompt), device=self.device))
        self._commit(torch.full((1,), len(prompt), dtype=torch.int32, device=self.device))
        self._verify(x[-1:], torch.empty(0, dtype=torch.int32, device=self.device), 0, logits)
        return int(self.result[1])

    def _verify(self, x: torch.Tensor, drafts: torch.Tensor, n_valid: int, logits) -> None:
        S = x.shape[0]
        sdv.sdv_verify_head(self.head, x, S, drafts, n_valid, logits, self.argmax[:S], self.result[:1],
                            self.result[1:], self.head_ws)

    def round(self, a0: int, drafts: Sequence[int], k: int, logits: torch.Tensor | None = None) -> tuple[int, int]:
        """Verifies [a0] + drafts (at most k, padded to k) and commits a0 and the accepted
        ones; returns how many drafts those were and the next a0."""
        n_valid = len(drafts)
        if not 0 <= n_valid <= k < WINDOW:
            raise ValueError(f"{n_valid} drafts in a window for {k}, at most {WINDOW - 1}")
        window = torch.tensor([a0, *drafts] + [PAD] * (k - n_valid), dtype=torch.int32).to(self.device)
        x = self._body(window.long())
        self._verify(x, window[1:].clone(), n_valid, logits)
        self._commit(self.result[:1] + 1)
        accepted, a0 = self.result.tolist()
        return accepted, a0

    def status(self) -> int:
        """The first device status of the operators' workspaces that is not SDV_OK, or SDV_OK."""
        spaces = [self.head_ws]
        for layer in self.layers:
            spaces += [layer.ws] if isinstance(layer, _AttentionLayer) else list(layer.wss.values())
        return next((s for s in map(sdv.sdv_last_device_status, spaces) if s != sdv.SDV_OK), sdv.SDV_OK)


def generate(target: HybridTarget, prompt: Sequence[int], count: int, k: int = 8, m: int = 2) -> tuple[list[int], int]:
    """``count`` greedy tokens by n-gram speculative rounds; also how many rounds they took."""
    stream = [int(t) for t in prompt]
    drafter = NgramDrafter(m)
    drafter.append(stream)
    a0, rounds = target.prefill(stream), 0
    end = len(stream) + count
    while True:
        stream.append(a0)
        drafter.append([a0])
        if len(stream) >= end:
            return stream[len(prompt):end], rounds
        drafts = drafter.propose(k)
        accepted, a0 = target.round(a0, drafts, k)
        stream += drafts[:accepted]
        drafter.append(drafts[:accepted])
        rounds += 1


def main() -> None:
    target = HybridTarget()
    prompt = torch.randint(0, 4096, (700,), generator=torch.Generator().manual_seed(1)).tolist()
    tokens, rounds = generate(target, prompt, 256)
    print(f"{len(prompt)} prompt tokens, {len(tokens)} generated in {rounds} rounds, "
          f"status {target.status()}: {tokens[:12]} ...")


if __name__ == "__main__":
    main()
