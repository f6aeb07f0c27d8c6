"""Token mixing in 64 bits (oracle): paged cache, its attention, linear attention.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path; it
shares no code with it.  Plain NumPy from the definitions:

* append: row t of sequence b goes to position ctx[b] + t, which lives in slot
  p % page of page table[b][p // page];
* attention of a window row over the positions it sees: softmax(scale q.k) v,
  and the logarithm of the softmax's denominator; nothing seen: 0 and -inf;
* linear attention: M_t = exp(g_t) M_{t-1} + k_t v_t^T, o_t = scale M_t^T q_t.

Beside each result come the magnitudes its rounding errors scale with (sums of
absolute values), from which the tests take their tolerances.
"""
from __future__ import annotations

import numpy as np


def rows_of_cache(pages: np.ndarray, table: np.ndarray, head: int, count: int) -> np.ndarray:
    """The first ``count`` positions of one sequence's head: [count, dim]."""
    page = pages.shape[2]
    out = np.zeros((count, pages.shape[3]))
    for p in range(count):
        out[p] = pages[table[p // page], head, p % page]
    return out


def append(pages: np.ndarray, rows: np.ndarray, table: np.ndarray, ctx, n) -> np.ndarray:
    """A copy of ``pages`` with ``rows`` [B, T, heads, dim] written behind ctx."""
    out = pages.copy()
    page = pages.shape[2]
    for b in range(rows.shape[0]):
        for t in range(n[b]):
            p = ctx[b] + t
            out[table[b][p // page], :, p % page] = rows[b, t]
    return out


def seen(i: int, n: int, word) -> list[int]:
    """Window positions that row i of n sees (word: its visibility bits, None: causal)."""
    if word is None:
        return list(range(i + 1))
    return [j for j in range(n) if int(word) >> j & 1]


def attention(q, k_pages, v_pages, table, ctx, n, mask, scale):
    """q [B, S, Hq, dim] -> dict of out, lse and, per output, ``weight`` (sum of
    p |v|), ``total`` (sum of |v| over the seen positions); per row ``dot`` (the
    largest sum |q k| scale) and ``count`` (positions seen)."""
    B, S, hq, d = q.shape
    hkv = k_pages.shape[1]
    g = hq // hkv
    out = {"out": np.zeros((B, S, hq, d)), "lse": np.full((B, S, hq), -np.inf), "weight": np.zeros((B, S, hq, d)),
           "total": np.zeros((B, S, hq, d)), "dot": np.zeros((B, S, hq)), "count": np.zeros((B, S, hq))}
    for b in range(B):
        for h in range(hkv):
            k = rows_of_cache(k_pages, table[b], h, ctx[b] + n[b])
            v = rows_of_cache(v_pages, table[b], h, ctx[b] + n[b])
            for i in range(n[b]):
                at = list(range(ctx[b])) + [ctx[b] + j for j in seen(i, n[b], None if mask is None else mask[b][i])]
                if not at:
                    continue
                kk, vv = k[at], v[at]
                for e in range(g):
                    x = q[b, i, h * g + e]
                    s = kk @ x * scale
                    m = s.max()
                    w = np.exp(s - m)
                    z = w.sum()
                    w = w / z
                    o = (b, i, h * g + e)
                    out["out"][o] = w @ vv
                    out["lse"][o] = m + np.log(z)
                    out["weight"][o] = w @ np.abs(vv)
                    out["total"][o] = np.abs(vv).sum(0)
                    out["dot"][o] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
                    out["count"][o] = len(at)
    return out


def linear(q, k, v, g, scale, n, state):
    """q, k [B, T, Hqk, Dk], v [B, T, H, Dv], g [B, T, H], state [B, H, Dk, Dv] ->
    dict of o, state and the same with every term's absolute value (``o_abs``,
    ``state_abs``)."""
    B, T, H, dv = v.shape
    r = H // k.shape[2]
    m, ma = state.astype(np.float64).copy(), np.abs(state.astype(np.float64))
    o, oa = np.zeros((B, T, H, dv)), np.zeros((B, T, H, dv))
    for b in range(B):
        for h in range(H):
            for t in range(n[b]):
                f = np.exp(min(g[b, t, h], 0.0))
                kk, vv = k[b, t, h // r], v[b, t, h]
                m[b, h] = (f * m[b, h] if f else 0.0) + np.outer(kk, vv)
                ma[b, h] = (f * ma[b, h] if f else 0.0) + np.outer(np.abs(kk), np.abs(vv))
                if q is not None:
                    o[b, t, h] = scale * (q[b, t, h // r] @ m[b, h])
                    oa[b, t, h] = abs(scale) * (np.abs(q[b, t, h // r]) @ ma[b, h])
    return {"o": o, "state": m, "o_abs": oa, "state_abs": ma}


def linear_squares(q, k, v, g, scale, n, state, chunk):
    """Per output the sum of squares of what may be rounded to 16 bits on its way: the
    decayed scores' terms inside the token's chunk, the terms of the state at the chunk's
    start, and the output.  Arguments as for ``linear`` (g above -inf); also returns o."""
    B, T, H, dv = v.shape
    r = H // k.shape[2]
    out, squares = np.zeros((B, T, H, dv)), np.zeros((B, T, H, dv))
    for b in range(B):
        for h in range(H):
            m = state[b, h].astype(np.float64)
            for t in range(0, n[b], chunk):
                at = slice(t, min(t + chunk, n[b]))
                qc, kc, vc = q[b, at, h // r], k[b, at, h // r], v[b, at, h]
                run = np.cumsum(np.minimum(g[b, at, h], 0.0))
                p = np.tril(qc @ kc.T * np.exp(np.minimum(run[:, None] - run[None, :], 0.0)))
                dec = np.exp(run)[:, None]
                o = scale * (p @ vc + dec * (qc @ m))
                out[b, at, h] = o
                squares[b, at, h] = scale ** 2 * ((p * p) @ (vc * vc) + dec ** 2 * ((qc * qc) @ (m * m))) + o * o
                m = np.exp(run[-1]) * m + (kc * np.exp(run[-1] - run)[:, None]).T @ vc
    return out, squares


def attention_squares(q, k_pages, v_pages, table, ctx, n, mask, scale):
    """Per output of ``attention`` the sum of squares of its weights' terms and of itself."""
    B, S, hq, d = q.shape
    hkv = k_pages.shape[1]
    g = hq // hkv
    squares = np.zeros((B, S, hq, d))
    for b in range(B):
        for h in range(hkv):
            k = rows_of_cache(k_pages, table[b], h, ctx[b] + n[b])
            v = rows_of_cache(v_pages, table[b], h, ctx[b] + n[b])
            for i in range(n[b]):
                at = list(range(ctx[b])) + [ctx[b] + j for j in seen(i, n[b], None if mask is None else mask[b][i])]
                if not at:
                    continue
                for e in range(g):
                    s = k[at] @ q[b, i, h * g + e] * scale
                    w = np.exp(s - s.max())
                    w = w / w.sum()
                    squares[b, i, h * g + e] = (w * w) @ (v[at] * v[at]) + (w @ v[at]) ** 2
    return squares
