"""What surrounds a batched verify round, in 64 bits (oracle): pages, norms and
positions, attention behind a shared prefix, drafted tokens.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path; it
shares no code with it.  Plain Python and NumPy from the definitions:

* pages: a stack of free pages; what sequences hold too much goes back first, then
  those that need more take theirs, in order, until one cannot have all;
* norm and rotation of a head: x / sqrt(mean x^2 + eps) w, then pairs as complex
  numbers times amplitude e^(i p f);
* a prefix is a sequence's first positions: the attention of ``oracle.mixing`` over a
  table and cache of both;
* drafted tokens: test after test, then a draw by the running sum of the weights.
"""
from __future__ import annotations

import numpy as np

from . import mixing


def assign(free, n_free, table, held, page, ctx, n, T):
    """Lists in, a dict of lists out (free: the whole array, of which n_free count)."""
    free, table, held = list(free), [list(r) for r in table], list(held)
    width, top = len(table[0]), n_free
    want = [min(-(-(c + r) // page), width) for c, r in zip(ctx, n)]
    back = [(b, j) for b in range(len(held)) for j in range(want[b], held[b])]
    top += len(back)
    for k, (b, j) in enumerate(back):
        free[top - 1 - k] = table[b][j]
        table[b][j] = -1
    for b in range(len(held)):
        held[b] = min(held[b], want[b])
    for b in range(len(held)):
        short = want[b] - held[b]
        if short > top:
            break
        for _ in range(short):
            top -= 1
            table[b][held[b]] = free[top]
            held[b] += 1
    out = {"granted": [], "positions": [], "slots": []}
    for b in range(len(held)):
        rows = max(0, min(n[b], held[b] * page - ctx[b]))
        at = [ctx[b] + t for t in range(rows)]
        out["granted"].append(rows)
        out["positions"].append(at + [-1] * (T - rows))
        out["slots"].append([table[b][p // page] * page + p % page for p in at] + [-1] * (T - rows))
    return {**out, "free": free, "n_free": top, "table": table, "held": held}


def norm_rope(x, weight, eps, positions, frequencies, amplitude, layout):
    """x [..., heads, dim] with positions [...]; frequencies: radians per position of each pair
    (none: no rotation)."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    half = len(frequencies)
    if half:
        turn = amplitude * np.exp(1j * positions[..., None, None] * np.asarray(frequencies))
        first, second = (slice(0, half), slice(half, 2 * half)) if layout == "half" else \
            (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        z = (y[..., first] + 1j * y[..., second]) * turn
        y = y.copy()
        y[..., first], y[..., second] = z.real, z.imag
    return y


def prefix_attention(q, k_pages, v_pages, prefix_table, prefix, table, ctx, n, mask, scale):
    """As ``oracle.mixing.attention``, behind the prefix: on a cache of pages of one position."""
    page, hkv, d = k_pages.shape[2], k_pages.shape[1], k_pages.shape[3]
    singles = lambda x: x.transpose(0, 2, 1, 3).reshape(-1, hkv, 1, d)  # noqa: E731
    rows = []
    front = [prefix_table[p // page] * page + p % page for p in range(prefix)]
    for b in range(q.shape[0]):
        rows.append(front + [table[b][p // page] * page + p % page for p in range(ctx[b] + n[b])])
    return mixing.attention(q, singles(k_pages), singles(v_pages), rows, [prefix + c for c in ctx], n, mask, scale)


def target_probs(logits, temperature):
    """One row's probabilities."""
    x = logits.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    p = np.zeros_like(x)
    if not x.max() > -np.inf:
        return p
    if not temperature > 0:
        p[int(x.argmax())] = 1.0
        return p
    p = np.exp((x - x.max()) / temperature)
    return p / p.sum()


def verify(logits, temperature, drafts, n, probs, uniforms):
    """One sequence: logits [S, V], drafts and probs (or None) of S - 1 rows, uniforms [S] ->
    (accepted, token, margin): the least distance of a test or of the draw from its border,
    relative to the probability or to all weights."""
    V = logits.shape[1]
    margin = np.inf
    weights = None
    i = 0
    while i < n:
        p, d = target_probs(logits[i], temperature), int(drafts[i])
        q = np.zeros(V)
        if probs is not None:
            q = np.where(probs[i] > 0, probs[i], 0.0).astype(np.float64)
        elif 0 <= d < V:
            q[d] = 1.0
        pd, qd = (p[d], q[d]) if 0 <= d < V else (0.0, 0.0)
        if pd > 0:
            margin = min(margin, abs(float(uniforms[i]) * qd - pd) / pd)
        if not (0 <= d < V and float(uniforms[i]) * qd < pd):
            weights = np.maximum(p - q, 0.0)
            if not weights.sum() > 0:
                weights = p
            break
        i += 1
    if weights is None:
        weights = target_probs(logits[i], temperature)
    total = weights.sum()
    if not total > 0:
        return i, -1, margin
    running = np.cumsum(weights)
    want = float(uniforms[-1]) * running[-1]
    token = int(np.searchsorted(running, want, side="right"))
    margin = min(margin, np.abs(running - want).min() / running[-1])
    return i, token, margin
