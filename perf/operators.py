"""The token-mixing operators of a verify round, as cases that can be measured.

* ``append``: a window's (or a prompt's) keys and values into a paged cache;
* ``attn``: attention of the 1..32 rows of a verify window over a paged cache,
  grouped heads, causal or with a 32-bit visibility word per row (trees);
* ``linear``: linear attention with a decay per head: prompts, single tokens, and
  a speculative round (outputs of the window, then the state advanced by the
  accepted tokens only).

``run`` computes a case in elementary torch operations in 32 bits, or, where
``own`` is true, through the framework's entry points on the same state.
Lengths are a function of the case alone (so is ``work``); the seed draws the
values, the order of the lengths, the page order and the trees.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------------------

def listed():
    return [
        # one sequence's newest token into its cache: the smallest call there is
        {"name": "append_one", "op": "append", "type": "f16", "B": 1, "T": 1, "Hkv": 8, "D": 128, "page": 16,
         "lo": 1000, "hi": 1000},
        # eight prompts of unequal length enter the cache at once
        {"name": "append_prompts", "op": "append", "type": "bf16", "B": 8, "T": 4096, "Hkv": 8, "D": 128, "page": 16,
         "lo": 0, "hi": 0},
        # single-user decoding early in a conversation: latency
        {"name": "attn_one_short", "op": "attn", "type": "f16", "B": 1, "S": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "lo": 613, "hi": 613, "mask": "causal"},
        # batched decoding, one token for each of 48 users whose contexts differ widely
        {"name": "attn_batch", "op": "attn", "type": "bf16", "B": 48, "S": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "lo": 40, "hi": 16001, "mask": "causal"},
        # the 17-row verify window of one user over a long document, few wide kv heads
        {"name": "attn_window", "op": "attn", "type": "f16", "B": 1, "S": 17, "Hq": 16, "Hkv": 2, "D": 256,
         "page": 64, "lo": 32768, "hi": 32768, "mask": "causal"},
        # tree windows of six users: pad nodes, short windows, users without a context
        {"name": "attn_tree", "op": "attn", "type": "bf16", "B": 6, "S": 32, "Hq": 24, "Hkv": 4, "D": 128,
         "page": 32, "lo": 0, "hi": 6001, "mask": "tree"},
        # one token over a book-length cache: the read of the cache is everything
        {"name": "attn_long", "op": "attn", "type": "f16", "B": 1, "S": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 64, "lo": 500001, "hi": 500001, "mask": "causal"},
        # single-user decoding: one token through a layer's states
        {"name": "linear_one", "op": "linear", "form": "step", "type": "f16", "B": 1, "T": 1, "H": 32, "Hqk": 16,
         "Dk": 128, "Dv": 128, "decay": "token"},
        # batched decoding: the states' read and write are everything
        {"name": "linear_batch", "op": "linear", "form": "step", "type": "bf16", "B": 128, "T": 1, "H": 32, "Hqk": 16,
         "Dk": 128, "Dv": 128, "decay": "token"},
        # a speculative round of 16 users: 17-row windows, then the accepted tokens enter the state
        {"name": "linear_round", "op": "linear", "form": "round", "type": "f16", "B": 16, "T": 17, "H": 32, "Hqk": 16,
         "Dk": 128, "Dv": 128, "decay": "token"},
        # one long prompt
        {"name": "linear_prompt", "op": "linear", "form": "prompt", "type": "f16", "B": 1, "T": 8192, "H": 32,
         "Hqk": 16, "Dk": 128, "Dv": 128, "decay": "token"},
        # prompts of unequal length through heads with narrow keys and one fixed decay each
        {"name": "linear_prompts", "op": "linear", "form": "prompt", "type": "bf16", "B": 6, "T": 3001, "H": 24,
         "Hqk": 24, "Dk": 64, "Dv": 128, "decay": "head"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the listed ones' ranges, sizes spread over their logarithm."""
    typ = rng.choice(["f16", "bf16"])
    op = rng.choice(["append", "attn", "attn", "linear", "linear"])
    if op == "append":
        B, hkv, d = _log_int(rng, 1, 64), rng.choice([2, 4, 8]), rng.choice([64, 128, 256])
        T = _log_int(rng, 1, max(1, min(4096, 8 * 4096 * 8 * 128 // (B * hkv * d))))
        lo = _log_int(rng, 1, 3000) - 1
        return {"op": op, "type": typ, "B": B, "T": T, "Hkv": hkv, "D": d, "page": rng.choice([16, 32, 64, 128]),
                "lo": lo, "hi": lo + _log_int(rng, 1, 500) - 1}
    if op == "attn":
        B, S = _log_int(rng, 1, 64), rng.choice([1, 1, rng.randint(2, 32)])
        hkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8]), rng.choice([64, 128, 128, 256])
        # the mean context stays where the cache and the plain form's scores are no larger than the listed cases'
        most = min(500000, 480000 * 8 * 128 // (B * hkv * d), 1 << 28 if S == 1 else (1 << 28) // (B * hkv * group * S))
        hi = _log_int(rng, 1, max(1, most))
        lo = 0 if rng.random() < 0.2 else _log_int(rng, 1, hi)
        return {"op": op, "type": typ, "B": B, "S": S, "Hq": hkv * group, "Hkv": hkv, "D": d,
                "page": rng.choice([16, 32, 64, 128]), "lo": lo, "hi": hi,
                "mask": rng.choice(["causal", "tree"]) if S > 1 else "causal"}
    form = rng.choice(["step", "round", "prompt", "prompt"])
    hqk = rng.choice([4, 8, 16])
    H = hqk * rng.choice([1, 2])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    if form == "prompt":
        T = _log_int(rng, 40, 8192)
        B = _log_int(rng, 1, max(1, min(32, 24 * 8192 * 8192 // (H * T * T), 16 * 8192 // T)))
    else:
        T = 1 if form == "step" else rng.randint(2, 32)
        B = _log_int(rng, 1, 128)
    return {"op": op, "form": form, "type": typ, "B": B, "T": T, "H": H, "Hqk": hqk, "Dk": dk, "Dv": dv,
            "decay": rng.choice(["token", "head"])}


def _spread(lo, hi, n):
    """n lengths from hi down to lo, even in their logarithm (lo may be 0)."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [int(round(math.exp(b + (a - b) * i / (n - 1)) - 1.0)) for i in range(n)]


def _counts(case):
    """Rows of each sequence: full windows in the causal cases, shorter ones among the others."""
    B = case["B"]
    if case["op"] == "append":
        return _spread(max(1, case["T"] // 4), case["T"], B)
    if case["op"] == "attn":
        S = case["S"]
        return [S if case["mask"] == "causal" else max(1, S - 3 * (i % 4)) for i in range(B)]
    T = case["T"]
    if case["form"] == "round":  # accepted tokens + 1, from a first-draft miss to a full window
        return [1 + (7 * i + T - 1) % T for i in range(B)]
    if case["form"] == "prompt":
        return _spread(max(1, T // 5), T, B)
    return [T] * B


def _contexts(case):
    return _spread(case["lo"], case["hi"], case["B"])


def work(case):
    n, B = _counts(case), case["B"]
    if case["op"] == "append":
        rows = sum(n) * case["Hkv"] * case["D"]
        return {"bytes": 2 * 2 * 2 * rows + 8 * B, "flops": 0}
    if case["op"] == "attn":
        ctx = _contexts(case)
        kv = sum(c + r for c, r in zip(ctx, n)) * case["Hkv"] * case["D"] * 2 * 2
        rows = B * case["S"] * case["Hq"]
        pairs = sum(r * c + r * (r + 1) // 2 for c, r in zip(ctx, n)) * case["Hq"]
        return {"bytes": kv + rows * case["D"] * 2 * 2 + rows * 4 + 8 * B, "flops": 4 * case["D"] * pairs}
    H, hqk, dk, dv, T = case["H"], case["Hqk"], case["Dk"], case["Dv"], case["T"]
    state = B * H * dk * dv * 4
    toks = B * T if case["form"] == "round" else sum(n)
    qkv = toks * (2 * hqk * dk + H * dv) * 2 + B * T * H * dv * 2
    decay = (toks * H if case["decay"] == "token" else H) * 4
    flops = toks * H * 4 * dk * dv + (sum(n) * H * 2 * dk * dv if case["form"] == "round" else 0)
    return {"bytes": 2 * state + qkv + decay, "flops": flops}


# ---- inputs -----------------------------------------------------------------------------

def _perm(rng, n):
    return torch.randperm(n, generator=rng).tolist()


def _tree_masks(rng, B, S, n):
    """Visibility words of random draft trees: a node sees its ancestors and itself; a
    node without a parent (a pad) sees nothing of the window."""
    r = torch.rand((B, S, 2), generator=rng).tolist()
    words = []
    for b in range(B):
        seen = [1]
        for i in range(1, S):
            if i >= n[b] or r[b][i][0] < 0.1:
                seen.append(0)
                continue
            parent = int(r[b][i][1] * i)
            seen.append(seen[parent] | 1 << i if seen[parent] else 0)
        # a user whose whole window is pads
        if b == B - 1 and B > 1:
            seen = [0] * S
        words.append([w - (1 << 32) if w >= 1 << 31 else w for w in seen])
    return torch.tensor(words, dtype=torch.int32)


def prepare(case, seed):
    dt = TYPES[case["type"]]
    gpu = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    B = case["B"]
    n = _counts(case)
    order = _perm(cpu, B)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, device=DEV, generator=gpu) * std).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    st = {"case": case}
    if case["op"] == "linear":
        T, H, hqk, dk, dv = (case[k] for k in ("T", "H", "Hqk", "Dk", "Dv"))
        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1)  # noqa: E731
        st["q"] = (unit(normal(B, T, hqk, dk)) * math.sqrt(dk)).to(dt)
        st["k"] = unit(normal(B, T, hqk, dk)).to(dt)
        st["v"] = normal(B, T, H, dv)
        # decay rates from a token or two to a thousand tokens, over the heads
        rate = torch.exp(torch.linspace(math.log(1e-3), math.log(0.7), H, device=DEV))
        if case["decay"] == "token":
            st["g"] = -rate * torch.nn.functional.softplus(
                torch.randn((B, T, H), device=DEV, generator=gpu) * 1.5)
        else:
            st["g"] = -rate * (1 + 0.2 * torch.rand((H,), device=DEV, generator=gpu))
        st["state"] = torch.randn((B, H, dk, dv), device=DEV, generator=gpu) * 0.3
        st["n"] = ints([n[i] for i in order])
        st["scale"] = dk ** -0.5
        st["o"] = torch.empty((B, T, H, dv), dtype=dt, device=DEV)
        st["state_out"] = torch.empty_like(st["state"])
        return st
    ctx = [_contexts(case)[i] for i in order]
    n = [n[i] for i in order]
    hkv, d, page = case["Hkv"], case["D"], case["page"]
    need = [-(-(c + r) // page) for c, r in zip(ctx, n)]
    total, width = sum(need), max(need)
    pages = total + total // 8 + 1  # a cache that is nearly full
    ids = _perm(cpu, pages)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = torch.tensor(ids[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    st["table"] = table.to(DEV)
    st["ctx"], st["n"] = ints(ctx), ints(n)
    st["k_pages"], st["v_pages"] = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
    if case["op"] == "append":
        # keys and values as the two halves of one projection's output
        kv = normal(B, case["T"], 2, hkv, d)
        st["k"], st["v"] = kv[:, :, 0], kv[:, :, 1]
        return st
    # what lies behind a sequence's end in its last page is left over from other requests
    for b in range(B):
        used = (ctx[b] + n[b]) % page
        if used:
            last = int(table[b, need[b] - 1])
            st["k_pages"][last, :, used:] = float("nan")
            st["v_pages"][last, :, used:] = float("nan")
    S, hq = case["S"], case["Hq"]
    st["q"] = normal(B, S, hq, d, std=1.7)
    st["mask"] = _tree_masks(cpu, B, S, n).to(DEV) if case["mask"] == "tree" else None
    st["scale"] = d ** -0.5
    st["o"] = torch.empty((B, S, hq, d), dtype=dt, device=DEV)
    st["lse"] = torch.empty((B, S, hq), dtype=torch.float32, device=DEV)
    return st


# ---- one pass ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "linear": _own_linear}[op](st)
    return {"append": _plain_append, "attn": _plain_attn, "linear": _plain_linear}[op](st)


def _own_append(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    sdv.sdv_kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["ctx"], st["n"], None)
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _own_attn(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = sdv.paged_attn_workspace(st["q"], st["k_pages"], st["table"])
    sdv.sdv_paged_attn(st["q"], st["k_pages"], st["v_pages"], st["table"], st["ctx"], st["n"], st["mask"],
                       st["scale"], st["o"], st["lse"], ws)
    return {"o": st["o"], "lse": st["lse"]}


def _own_linear(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = sdv.linear_attn_workspace(st["k"], st["v"])
    if st["case"]["form"] == "round":
        # the whole window's outputs from the state as it stands, then the accepted tokens into it
        sdv.sdv_linear_attn(st["q"], st["k"], st["v"], st["g"], st["scale"], None, st["state"], None, st["o"], ws)
        sdv.sdv_linear_attn(None, st["k"], st["v"], st["g"], st["scale"], st["n"], st["state"], st["state_out"],
                            None, ws)
    else:
        sdv.sdv_linear_attn(st["q"], st["k"], st["v"], st["g"], st["scale"], st["n"], st["state"], st["state_out"],
                            st["o"], ws)
    return {"o": st["o"], "state": st["state_out"]}


def _plain_append(st):
    B, T = st["k"].shape[:2]
    page = st["k_pages"].shape[2]
    t = torch.arange(T, device=DEV)
    live = t[None, :] < st["n"][:, None]
    pos = (st["ctx"][:, None] + t[None, :]).long()
    b = torch.arange(B, device=DEV)[:, None].expand(B, T)[live]
    pos = pos[live]
    ids = st["table"][b, pos // page].long()
    st["k_pages"][ids, :, pos % page] = st["k"][live]
    st["v_pages"][ids, :, pos % page] = st["v"][live]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_attn(st):
    q, table = st["q"], st["table"].long().clamp(min=0)
    B, S, hq, d = q.shape
    hkv, page = st["k_pages"].shape[1:3]
    L, G = table.shape[1] * page, hq // hkv
    gather = lambda x: x[table].permute(0, 2, 1, 3, 4).reshape(B, hkv, L, d).float()  # noqa: E731
    k, v = gather(st["k_pages"]), gather(st["v_pages"])
    p = torch.arange(L, device=DEV)
    ctx, n, i = st["ctx"].long(), st["n"].long(), torch.arange(S, device=DEV)
    v = torch.where((p[None, :] < (ctx + n)[:, None])[:, None, :, None], v, 0.0)
    j = p[None, :] - ctx[:, None]  # the window position of a cache position
    if st["mask"] is None:
        inside = j[:, None, :] <= i[None, :, None]
    else:
        bit = (st["mask"].long()[:, :, None] >> j.clamp(0, 31)[:, None, :]) & 1
        inside = (j[:, None, :] < 0) | (bit == 1)
    see = inside & (j[:, None, :] < n[:, None, None]) & (i[None, :, None] < n[:, None, None])
    rows = q.reshape(B, S, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * S, d).float()
    s = (rows @ k.transpose(2, 3)) * st["scale"]
    s = s.reshape(B, hkv, G, S, L).masked_fill(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(B, hkv, G * S, L) @ v).reshape(B, hkv, G, S, d) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(B, S, hq, d).to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, S, hq)}


def _plain_linear(st):
    r = st["case"]["H"] // st["case"]["Hqk"]
    B, T = st["k"].shape[:2]
    heads = lambda x: x.float().permute(0, 2, 1, 3)  # noqa: E731
    q, k, v = heads(st["q"]).repeat_interleave(r, 1), heads(st["k"]).repeat_interleave(r, 1), heads(st["v"])
    g = st["g"] if st["g"].dim() == 3 else st["g"].expand(B, T, -1)
    g = g.permute(0, 2, 1)
    t = torch.arange(T, device=DEV)
    live = (t[None, :] < st["n"][:, None].long())[:, None, :]  # the tokens that enter the state
    rows = torch.ones_like(live) if st["case"]["form"] == "round" else live
    total = torch.cumsum(g, -1)
    diff = (total[..., :, None] - total[..., None, :]).masked_fill_(t[:, None] < t[None, :], float("-inf"))
    a = (q @ k.transpose(2, 3)).mul_(diff.exp_())
    o = (a @ v + torch.exp(total)[..., None] * (q @ st["state"])) * st["scale"]
    o = torch.where(rows[..., None], o, 0.0).permute(0, 2, 1, 3).to(st["v"].dtype)
    # the decay from behind each token to the end, summed from the end: the weights that count are exact
    after = torch.where(live, g, 0.0).flip(-1).cumsum(-1).flip(-1)
    whole = after[..., :1]
    behind = torch.cat([after[..., 1:], torch.zeros_like(whole)], -1)
    w = torch.where(live, torch.exp(behind), 0.0)[..., None]
    state = torch.exp(whole)[..., None] * st["state"] + (k * w).transpose(2, 3) @ v
    return {"o": o, "state": state}


# ---- the same in 64 bits, from the definitions -------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "attn":
        return _exact_attn(case, st)
    return _exact_linear(case, st)


def _exact_append(st):
    """The cache row by row: no arithmetic, the rows as they are."""
    out = {}
    page = st["k_pages"].shape[2]
    for rows, pages in (("k", "k_pages"), ("v", "v_pages")):
        kept = st[pages].double()
        for b, (c, m) in enumerate(zip(st["ctx"].tolist(), st["n"].tolist())):
            for p0 in range(c // page * page, c + m, page):
                lo, hi = max(p0, c), min(p0 + page, c + m)
                kept[int(st["table"][b, p0 // page]), :, lo - p0:hi - p0] = \
                    st[rows][b, lo - c:hi - c].double().transpose(0, 1)
        out[pages] = kept
    return out


def _exact_attn(case, st):
    S, hq, hkv, d, page = case["S"], case["Hq"], case["Hkv"], case["D"], case["page"]
    G = hq // hkv
    o = torch.zeros((case["B"], S, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"], S, hq), float("-inf"), dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        c, n = int(st["ctx"][b]), int(st["n"][b])
        where = torch.arange(c + n, device=DEV)
        ids = st["table"][b].long()[where // page]
        words = [(1 << i + 1) - 1 for i in range(S)] if st["mask"] is None else st["mask"][b].tolist()
        seen = [[bool(words[i] >> j & 1) for j in range(n)] for i in range(n)]
        see = torch.ones((n, c + n), dtype=torch.bool, device=DEV)
        see[:, c:] = torch.tensor(seen, device=DEV)
        for h in range(hkv):
            k = st["k_pages"][ids, h, where % page].double()
            v = st["v_pages"][ids, h, where % page].double()
            for g in range(G):
                s = st["q"][b, :n, h * G + g].double() @ k.T * st["scale"]
                s[~see] = float("-inf")
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - z[:, None]).nan_to_num(0.0)
                o[b, :n, h * G + g] = w @ v
                lse[b, :n, h * G + g] = z
    return {"o": o, "lse": lse}


def _exact_linear(case, st):
    B, T, H = case["B"], case["T"], case["H"]
    r = H // case["Hqk"]
    q, k = (st[x].double().repeat_interleave(r, 2) for x in ("q", "k"))
    v = st["v"].double()
    g = st["g"].double().expand(B, T, H) if st["g"].dim() == 1 else st["g"].double()
    n = st["n"].long()
    state = st["state"].double()
    kept = state.clone()
    o = torch.zeros((B, T, H, case["Dv"]), dtype=torch.float64, device=DEV)
    step = 32
    for t0 in range(0, T, step):
        at = slice(t0, min(t0 + step, T))
        C = at.stop - t0
        qc, kc, vc, gc = (x[:, at].transpose(1, 2) for x in (q, k, v, g[..., None]))
        run_g = torch.cumsum(gc[..., 0], -1)
        low = torch.ones((C, C), dtype=torch.bool, device=DEV).tril()
        w = torch.where(low, torch.exp(torch.where(low, run_g[..., :, None] - run_g[..., None, :], 0.0)), 0.0)
        y = ((qc @ kc.mT) * w) @ vc
        y = y + torch.exp(run_g)[..., None] * (qc @ state)
        o[:, at] = (y * st["scale"]).transpose(1, 2)
        # the state at each sequence's own end, if it ends in this stretch
        m = (n - t0).clamp(0, C)
        inside = torch.arange(C, device=DEV)[None, :] < m[:, None]
        end = torch.where(m > 0, m - 1, 0)
        end_g = run_g.gather(2, end[:, None, None].expand(B, H, 1))
        wk = torch.where(inside[:, None, :], torch.exp(torch.where(inside[:, None, :], end_g - run_g, 0.0)), 0.0)
        ended = torch.exp(end_g)[..., None] * state + (kc * wk[..., None]).mT @ vc
        kept = torch.where(((m > 0) & (n > t0))[:, None, None, None], ended, kept)
        full = torch.exp(run_g[..., -1:] - run_g)
        state = torch.exp(run_g[..., -1])[..., None, None] * state + (kc * full[..., None]).mT @ vc
    if case["form"] != "round":
        o[~(torch.arange(T, device=DEV)[None, :] < n[:, None])] = 0.0
    return {"o": o, "state": kept}
