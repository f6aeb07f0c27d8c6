"""The operators around a batched verify round, as cases that can be measured.

* ``pages``: page tables and slot maps of a paged cache, from the requests' lengths;
* ``rope``: norms of query and key heads and the position rotation, the queries out,
  keys and values into the cache;
* ``prefix``: attention of a batch whose requests share a long prefix, over that
  prefix and each request's own cache;
* ``verify``: drafted tokens against the target's probabilities, and the next token,
  from given random numbers.

``run`` computes a case in elementary torch operations, or, where ``own`` is true,
through the framework's entry points on the same state.  Lengths are a function of
the case alone (so is ``work``); the seed draws the values, the order of the lengths,
the page order, the trees, drafts and random numbers.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------

def listed():
    return [
        # 48 users' verify windows get their pages and slots, and give back what an
        # abandoned round does not keep: pure latency
        {"name": "pages_round", "op": "pages", "B": 48, "T": 17, "page": 16, "lo": 40, "hi": 16001},
        # 512 prompts are admitted and later retired
        {"name": "pages_admit", "op": "pages", "B": 512, "T": 2001, "page": 16, "lo": 0, "hi": 0},
        # single-user decoding: one token of an fp32 projection
        {"name": "rope_one", "op": "rope", "in": "f32", "type": "f16", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "layout": "half", "norm": True, "page": 16, "at": 1000, "scaling": "none"},
        # 17-row windows of 16 users far into long documents, wide heads rotated in part, scaled positions
        {"name": "rope_window", "op": "rope", "in": "bf16", "type": "bf16", "B": 16, "T": 17, "Hq": 16, "Hkv": 2,
         "D": 256, "rot": 64, "layout": "pairs", "norm": True, "page": 64, "at": 500001, "scaling": "ramp"},
        # prompts of unequal length
        {"name": "rope_prompt", "op": "rope", "in": "f16", "type": "f16", "B": 6, "T": 8001, "Hq": 32, "Hkv": 8,
         "D": 128, "rot": 128, "layout": "half", "norm": True, "page": 16, "at": 0, "scaling": "bands"},
        # four users behind a system prompt, early in their conversations: latency
        {"name": "prefix_few", "op": "prefix", "type": "f16", "B": 4, "S": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "prefix": 1201, "lo": 1, "hi": 100, "mask": "causal"},
        # batched decoding of 64 users about one long document
        {"name": "prefix_batch", "op": "prefix", "type": "bf16", "B": 64, "S": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "prefix": 32768, "lo": 40, "hi": 2001, "mask": "causal"},
        # tree windows of 24 users, wide heads, a prefix that ends inside a page
        {"name": "prefix_tree", "op": "prefix", "type": "f16", "B": 24, "S": 9, "Hq": 16, "Hkv": 2, "D": 256,
         "page": 64, "prefix": 8011, "lo": 0, "hi": 900, "mask": "tree"},
        # windows of 256 users over a long instruction: products, not the cache's read
        {"name": "prefix_many", "op": "prefix", "type": "bf16", "B": 256, "S": 5, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 32, "prefix": 16384, "lo": 100, "hi": 1001, "mask": "causal"},
        # one user's window, drafts from a deterministic drafter
        {"name": "verify_one", "op": "verify", "type": "f32", "B": 1, "S": 5, "V": 151936, "probs": False,
         "greedy": 0},
        # the windows of 32 users whose drafts a small model has drawn
        {"name": "verify_batch", "op": "verify", "type": "f32", "B": 32, "S": 9, "V": 151936, "probs": True,
         "greedy": 3},
        # plain sampling of one token for each of 200 users, 16-bit logits of an odd vocabulary
        {"name": "verify_sample", "op": "verify", "type": "bf16", "B": 200, "S": 1, "V": 50257, "probs": False,
         "greedy": 40},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the listed ones' ranges, sizes spread over their logarithm."""
    op = rng.choice(["pages", "rope", "rope", "prefix", "prefix", "verify", "verify"])
    if op == "pages":
        B = _log_int(rng, 1, 512)
        T = _log_int(rng, 1, 2001)
        lo = 0 if T > 64 else _log_int(rng, 1, 1000)
        return {"op": op, "B": B, "T": T, "page": rng.choice([8, 16, 16, 32, 48, 64]), "lo": lo,
                "hi": lo + (0 if T > 64 else _log_int(rng, 1, 15000))}
    if op == "rope":
        typ = rng.choice(["f16", "bf16"])
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 128, 256])
        hq = hkv * rng.choice([1, 2, 4, 8])
        most = 6 * 6000 * 48 * 128 // ((hq + 2 * hkv) * d * 2)
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(8192, most // B)))
        return {"op": op, "in": rng.choice(["f32", typ, typ]), "type": typ, "B": B, "T": T, "Hq": hq, "Hkv": hkv,
                "D": d, "rot": rng.choice([d, d, d // 2, 20]), "layout": rng.choice(["half", "pairs"]),
                "norm": rng.random() < 0.7, "page": rng.choice([8, 16, 32, 48, 64]),
                "at": _log_int(rng, 1, 1000001) - 1, "scaling": rng.choice(["none", "linear", "base", "ramp", "bands"])}
    if op == "prefix":
        B, S = _log_int(rng, 2, 256), rng.choice([1, 1, rng.randint(2, 32)])
        hkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8]), rng.choice([64, 128, 128, 256])
        # rows x prefix and the batch's own positions stay below the largest listed case's
        rows = B * S * hkv * group
        most = min(65536, 16384 * 256 * 5 * 32 * 128 // (rows * d))
        hi = _log_int(rng, 1, max(2, min(2001, 1001 * 256 * 8 * 128 // (B * hkv * d), (1 << 29) // rows)))
        return {"op": op, "type": rng.choice(["f16", "bf16"]), "B": B, "S": S, "Hq": hkv * group, "Hkv": hkv, "D": d,
                "page": rng.choice([16, 32, 64, 128]), "prefix": _log_int(rng, 1, max(2, most)),
                "lo": rng.randint(0, min(hi, 100)), "hi": hi,
                "mask": rng.choice(["causal", "tree"]) if S > 1 else "causal"}
    V = rng.choice([32000, 50257, 151936, 248320])
    S = rng.choice([1, rng.randint(2, 17)])
    B = _log_int(rng, 1, max(1, min(256, 32 * 9 * 151936 // (2 * V * S))))
    return {"op": op, "type": rng.choice(["f32", "f16", "bf16"]), "B": B, "S": S, "V": V,
            "probs": S > 1 and rng.random() < 0.6, "greedy": rng.choice([0, B // 4])}


def _spread(lo, hi, n):
    """n lengths from hi down to lo, even in their logarithm (lo may be 0)."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [int(round(math.exp(b + (a - b) * i / (n - 1)) - 1.0)) for i in range(n)]


def _counts(case):
    """Rows of each sequence."""
    B = case["B"]
    if case["op"] == "prefix":
        S = case["S"]
        return [S if case["mask"] == "causal" else max(1, S - 3 * (i % 4)) for i in range(B)]
    T = case["T"]
    # windows are full or a draft or two short, prompts of any length
    return [max(1, T - i % 3) for i in range(B)] if T <= 64 else _spread(max(1, T // 5), T, B)


def _contexts(case):
    if case["op"] == "rope":
        return [max(0, case["at"] - 37 * i) for i in range(case["B"])]
    return _spread(case["lo"], case["hi"], case["B"])


def work(case):
    B = case["B"]
    if case["op"] == "pages":
        page = case["page"]
        moved = sum(-(-(c + r) // page) - -(-c // page) for c, r in zip(_contexts(case), _counts(case)))
        # lengths and counts in and out twice, the pages' ids there and back, positions and slots
        return {"bytes": 2 * 16 * B + 2 * 8 * moved + 8 * B * case["T"], "flops": 0}
    if case["op"] == "rope":
        size = 4 if case["in"] == "f32" else 2
        n = sum(_counts(case))
        elements = n * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        return {"bytes": elements * (size + 2) + 8 * B * case["T"], "flops": 6 * elements}
    if case["op"] == "prefix":
        ctx, n = _contexts(case), _counts(case)
        kv = (case["prefix"] + sum(ctx) + sum(n)) * case["Hkv"] * case["D"] * 2 * 2
        rows = B * case["S"] * case["Hq"]
        pairs = sum(r * (case["prefix"] + c) + r * (r + 1) // 2 for c, r in zip(ctx, n)) * case["Hq"]
        return {"bytes": kv + rows * case["D"] * 2 * 2 + rows * 4 + 8 * B, "flops": 4 * case["D"] * pairs}
    size = 4 if case["type"] == "f32" else 2
    V = case["V"]
    # every row's logits; of the drafter's probabilities the rejected row
    return {"bytes": B * case["S"] * V * size + (B * V * 4 if case["probs"] else 0), "flops": 4 * B * case["S"] * V}


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
        words.append([w - (1 << 32) if w >= 1 << 31 else w for w in seen])
    return torch.tensor(words, dtype=torch.int32)


def _frequencies(case):
    """Angle per position of each rotated pair (64 bits) and the factor on the rotation."""
    rot, theta, kind = case["rot"], 10000.0 if case["scaling"] == "none" else 500000.0, case["scaling"]
    half = rot // 2
    if kind == "base":
        theta *= 8.0 ** (rot / (rot - 2))
    f = [theta ** (-2.0 * i / rot) for i in range(half)]
    if kind == "linear":
        return [x / 8.0 for x in f], 1.0
    if kind == "ramp":
        # pairs that turn more than 32 times in 8192 positions stay, those below one turn are
        # interpolated, a ramp over the pair's index between
        at = [rot * math.log(8192 / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        share = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(half)]
        return [x / 8.0 * s + x * (1 - s) for x, s in zip(f, share)], 0.1 * math.log(8.0) + 1.0
    if kind == "bands":
        # the same by turns in 8192 positions: 4 and more stay, 1 and fewer are interpolated
        share = [min(1.0, max(0.0, (8192 * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [x / 8.0 * (1 - s) + x * s for x, s in zip(f, share)], 1.0
    return f, 1.0


def prepare(case, seed):
    gpu = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    return {"pages": _prepare_pages, "rope": _prepare_rope, "prefix": _prepare_prefix,
            "verify": _prepare_verify}[case["op"]](case, gpu, cpu)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(gpu, dt, *shape, std=1.0):
    return (torch.randn(shape, device=DEV, generator=gpu) * std).to(dt)


def _prepare_pages(case, gpu, cpu):
    B, T, page = case["B"], case["T"], case["page"]
    order = _perm(cpu, B)
    ctx, n = [_contexts(case)[i] for i in order], [_counts(case)[i] for i in order]
    held = [-(-c // page) for c in ctx]
    need = [-(-(c + r) // page) for c, r in zip(ctx, n)]
    width = max(need) + 1
    total = sum(need)
    pages = total + total // 8 + 1
    ids = _perm(cpu, pages)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = torch.tensor(ids[at:at + held[b]], dtype=torch.int32)
        at += held[b]
    free = torch.zeros(pages, dtype=torch.int32)
    free[:pages - at] = torch.tensor(ids[at:], dtype=torch.int32)
    return {"case": case, "table": table.to(DEV), "held": _ints(held), "free": free.to(DEV),
            "n_free": _ints([pages - at]), "ctx": _ints(ctx), "n": _ints(n), "none": _ints([0] * B),
            "granted": _ints([0] * B), "positions": torch.zeros((B, T), dtype=torch.int32, device=DEV),
            "slots": torch.zeros((B, T), dtype=torch.int32, device=DEV)}


def _prepare_rope(case, gpu, cpu):
    B, T, hq, hkv, d, page = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    dt = TYPES[case["type"]]
    order = _perm(cpu, B)
    ctx, n = [_contexts(case)[i] for i in order], [_counts(case)[i] for i in order]
    total = sum(n)
    pages = -(-total // page) + 2
    st = {"case": case}
    # one projection's output: the queries' heads, the keys', the values'
    qkv = _normal(gpu, TYPES[case["in"]], B, T, hq + 2 * hkv, d, std=1.5)
    st["q"], st["k"], st["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    st["k_pages"], st["v_pages"] = _normal(gpu, dt, pages, hkv, page, d), _normal(gpu, dt, pages, hkv, page, d)
    # places of the rows: pages in any order, a sequence's rows one after another
    t = torch.arange(T)
    live = t[None, :] < torch.tensor(n)[:, None]
    where = torch.full((B, T), -1, dtype=torch.long)
    where[live] = torch.arange(total) + page // 2
    ids = torch.randperm(pages, generator=cpu)
    slots = torch.where(live, ids[where.clamp(min=0) // page] * page + where % page, -1)
    st["slots"] = slots.to(torch.int32).to(DEV)
    st["positions"] = torch.where(live, torch.tensor(ctx)[:, None] + t[None, :], -1).to(torch.int32).to(DEV)
    if case["norm"]:
        st["q_weight"] = 1.0 + 0.2 * torch.randn(d, device=DEV, generator=gpu)
        st["k_weight"] = 1.0 + 0.2 * torch.randn(d, device=DEV, generator=gpu)
    else:
        st["q_weight"] = st["k_weight"] = None
    st["eps"] = 1e-6
    st["q_out"] = torch.zeros((B, T, hq, d), dtype=dt, device=DEV)
    f, st["amplitude"] = _frequencies(case)
    st["frequencies"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if own:
        from speculative_decode_verify_sdv_gb300 import sdv
        st["rope"] = sdv.rope_plan(case["rot"], 10000.0 if case["scaling"] == "none" else 500000.0, case["layout"],
                                   **{"none": {}, "linear": {"scaling": "linear", "factor": 8.0},
                                      "base": {"scaling": "base", "factor": 8.0},
                                      "ramp": {"scaling": "ramp", "factor": 8.0, "trained": 8192, "low": 1.0,
                                               "high": 32.0},
                                      "bands": {"scaling": "bands", "factor": 8.0, "trained": 8192, "low": 1.0,
                                                "high": 4.0}}[case["scaling"]], device=DEV)
    return st


def _prepare_prefix(case, gpu, cpu):
    B, S, hq, hkv, d, page = (case[k] for k in ("B", "S", "Hq", "Hkv", "D", "page"))
    dt = TYPES[case["type"]]
    order = _perm(cpu, B)
    ctx, n = [_contexts(case)[i] for i in order], [_counts(case)[i] for i in order]
    need = [-(-(c + r) // page) for c, r in zip(ctx, n)]
    shared = -(-case["prefix"] // page)
    total, width = sum(need) + shared, max(need)
    pages = total + total // 8 + 1  # a cache that is nearly full
    ids = _perm(cpu, pages)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = shared
    for b in range(B):
        table[b, :need[b]] = torch.tensor(ids[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    st = {"case": case, "table": table.to(DEV), "prefix_table": _ints(ids[:shared]),
          "prefix_len": _ints([case["prefix"]]), "ctx": _ints(ctx), "n": _ints(n)}
    st["k_pages"], st["v_pages"] = _normal(gpu, dt, pages, hkv, page, d), _normal(gpu, dt, pages, hkv, page, d)
    # what lies behind an end in its last page is left over from other requests
    ends = [(ids[shared - 1], case["prefix"] % page)]
    ends += [(int(table[b, need[b] - 1]), (ctx[b] + n[b]) % page) for b in range(B)]
    for last, used in ends:
        if used:
            st["k_pages"][last, :, used:] = float("nan")
            st["v_pages"][last, :, used:] = float("nan")
    st["q"] = _normal(gpu, dt, B, S, hq, d, std=1.7)
    st["mask"] = _tree_masks(cpu, B, S, n).to(DEV) if case["mask"] == "tree" else None
    st["scale"] = d ** -0.5
    st["o"] = torch.empty((B, S, hq, d), dtype=dt, device=DEV)
    st["lse"] = torch.empty((B, S, hq), dtype=torch.float32, device=DEV)
    return st


def _prepare_verify(case, gpu, cpu):
    B, S, V = case["B"], case["S"], case["V"]
    dt = TYPES[case["type"]]
    order = _perm(cpu, B)
    st = {"case": case}
    # a few hundred likely tokens over a long tail, as trained models' logits are
    logits = torch.randn((B, S, V), device=DEV, generator=gpu).mul_(2.2)
    near = logits[:, :S - 1] + 0.7 * torch.randn((B, S - 1, V), device=DEV, generator=gpu) if case["probs"] else None
    st["logits"] = logits.to(dt)
    warm = [0.6 + 0.1 * (i % 7) for i in range(B)]
    for i in range(case["greedy"]):
        warm[i] = 0.0
    t = [warm[i] for i in order]
    st["temperature"] = torch.tensor(t, dtype=torch.float32, device=DEV)
    st["uniforms"] = torch.rand((B, S), device=DEV, generator=gpu)
    st["n_drafts"] = _ints([max(0, S - 1 - 2 * (i % 3)) for i in order])
    soft = torch.tensor([max(x, 0.6) for x in t], device=DEV)[:, None, None]
    if case["probs"]:
        st["draft_probs"] = torch.softmax(near.div_(soft), -1)
        race = torch.empty_like(near).exponential_(generator=gpu)
        st["drafts"] = (st["draft_probs"] / race).argmax(-1).to(torch.int32)
    else:
        st["draft_probs"] = None
        # mostly what the target would say, else any token
        likely = st["logits"][:, :S - 1].argmax(-1)
        other = torch.randint(0, V, (B, S - 1), device=DEV, generator=gpu)
        hit = torch.rand((B, S - 1), device=DEV, generator=gpu) < 0.8
        st["drafts"] = torch.where(hit, likely, other).to(torch.int32)
    st["accepted"], st["next"] = _ints([0] * B), _ints([0] * B)
    return st


# ---- one pass ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"pages": _own_pages, "rope": _own_rope, "prefix": _own_prefix, "verify": _own_verify}[op](st)
    return {"pages": _plain_pages, "rope": _plain_rope, "prefix": _plain_prefix, "verify": _plain_verify}[op](st)


def _own_pages(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = sdv.page_assign_workspace(st["ctx"])
    page = st["case"]["page"]
    # the rows' pages and places, then the pages back: the state is as it was
    sdv.sdv_page_assign(st["free"], st["n_free"], st["table"], st["held"], page, st["ctx"], st["n"], st["granted"],
                        st["positions"], st["slots"], ws)
    sdv.sdv_page_assign(st["free"], st["n_free"], st["table"], st["held"], page, st["ctx"], st["none"], None, None,
                        None, ws)
    return {k: st[k] for k in ("granted", "positions", "slots", "table", "held", "free", "n_free")}


def _own_rope(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    sdv.sdv_qk_norm_rope(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["q_weight"], st["k_weight"],
                         st["eps"], st["rope"], st["positions"], st["slots"], st["q_out"], None)
    return {k: st[k] for k in ("q_out", "k_pages", "v_pages")}


def _own_prefix(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = sdv.prefix_attn_workspace(st["q"], st["k_pages"], st["table"])
    sdv.sdv_prefix_attn(st["q"], st["k_pages"], st["v_pages"], st["prefix_table"], st["prefix_len"], st["table"],
                        st["ctx"], st["n"], st["mask"], st["scale"], st["o"], st["lse"], ws)
    return {"o": st["o"], "lse": st["lse"]}


def _own_verify(st):
    from speculative_decode_verify_sdv_gb300 import sdv
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = sdv.verify_drafts_workspace(st["logits"])
    sdv.sdv_verify_drafts(st["logits"], st["temperature"], st["drafts"], st["n_drafts"], st["draft_probs"],
                          st["uniforms"], st["accepted"], st["next"], ws)
    return {"accepted": st["accepted"], "next": st["next"]}


def _plain_assign(st, n, places):
    page, ctx, held, table = st["case"]["page"], st["ctx"], st["held"], st["table"]
    B, width = table.shape
    want = ((ctx + n + page - 1) // page).clamp(max=width)
    col = torch.arange(width, device=DEV)
    # back on the list: the k-th page given back lies k places below the new top
    gone = (col >= want[:, None]) & (col < held[:, None])
    back = torch.cumsum(gone.flatten(), 0).reshape(B, width)
    top = st["n_free"].long() + back[-1, -1]
    place = torch.where(gone, top - back, st["free"].numel())
    grown = torch.cat([st["free"], st["free"].new_zeros(1)])
    grown[place.flatten()] = table.flatten()
    st["free"].copy_(grown[:-1])
    # the k-th page taken is the k-th from the top; who cannot have all its pages has none
    need = (want - held).clamp(min=0)
    through = torch.cumsum(need, 0)
    served = through <= top
    k = (through - need)[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < want[:, None]) & served[:, None]
    taken = st["free"][(top - 1 - k).clamp(0, st["free"].numel() - 1)]
    table.copy_(torch.where(fresh, taken, torch.where(gone, -1, table)))
    st["n_free"].copy_(top - torch.where(served, need, 0).sum())
    held.copy_(torch.where(served, want, torch.minimum(held, want)))
    if not places:
        return
    rows = torch.minimum(n, held * page - ctx).clamp(min=0)
    t = torch.arange(st["slots"].shape[1], device=DEV)
    live = t < rows[:, None]
    pos = ctx[:, None] + t
    slot = table.gather(1, (pos // page).clamp(max=width - 1)) * page + pos % page
    st["granted"].copy_(rows)
    st["positions"].copy_(torch.where(live, pos, -1))
    st["slots"].copy_(torch.where(live, slot, -1))


def _plain_pages(st):
    _plain_assign(st, st["n"], True)
    _plain_assign(st, st["none"], False)
    return {k: st[k] for k in ("granted", "positions", "slots", "table", "held", "free", "n_free")}


def _plain_rope(st):
    case = st["case"]
    rot, page = case["rot"], case["page"]
    pos, slots = st["positions"].long(), st["slots"].long()
    live = pos >= 0
    angle = pos[live][:, None].double() * st["frequencies"]
    cos, sin = (torch.cos(angle) * st["amplitude"]).float(), (torch.sin(angle) * st["amplitude"]).float()
    cos, sin = cos[:, None], sin[:, None]

    def turn(x, weight):
        x = x[live].float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * weight
        y = x.clone()
        if case["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return y

    st["q_out"][live] = turn(st["q"], st["q_weight"]).to(st["q_out"].dtype)
    at = slots[live]
    st["k_pages"][at // page, :, at % page] = turn(st["k"], st["k_weight"]).to(st["k_pages"].dtype)
    st["v_pages"][at // page, :, at % page] = st["v"][live].to(st["v_pages"].dtype)
    return {k: st[k] for k in ("q_out", "k_pages", "v_pages")}


def _plain_prefix(st):
    q = st["q"]
    B, S, hq, d = q.shape
    hkv, page = st["k_pages"].shape[1:3]
    G = hq // hkv
    # the shared positions: one product for all rows
    P = st["case"]["prefix"]
    shared = lambda x: x[st["prefix_table"].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :P].float()  # noqa: E731
    rows = q.reshape(B, S, hkv, G, d).permute(2, 0, 3, 1, 4).float() * st["scale"]
    far = rows.reshape(hkv, B * G * S, d) @ shared(st["k_pages"]).transpose(1, 2)
    m1 = far.amax(-1, keepdim=True)
    far = far.sub_(m1).exp_()
    l1 = far.sum(-1, keepdim=True)
    o1 = far @ shared(st["v_pages"])
    by_seq = lambda x: x.reshape(hkv, B, G, S, -1)  # noqa: E731
    m1, l1, o1 = by_seq(m1), by_seq(l1), by_seq(o1)
    # each request's own
    table = st["table"].long().clamp(min=0)
    L = table.shape[1] * page
    own_rows = lambda x: x[table].permute(2, 0, 1, 3, 4).reshape(hkv, B, L, d).float()  # noqa: E731
    p = torch.arange(L, device=DEV)
    ctx, n, i = st["ctx"].long(), st["n"].long(), torch.arange(S, device=DEV)
    v = torch.where((p[None, :] < (ctx + n)[:, None])[None, :, :, None], own_rows(st["v_pages"]), 0.0)
    j = p[None, :] - ctx[:, None]  # the window position of a cache position
    if st["mask"] is None:
        inside = j[:, None, :] <= i[None, :, None]
    else:
        bit = (st["mask"].long()[:, :, None] >> j.clamp(0, 31)[:, None, :]) & 1
        inside = (j[:, None, :] < 0) | (bit == 1)
    see = inside & (j[:, None, :] < n[:, None, None])
    s = rows.reshape(hkv, B, G * S, d) @ own_rows(st["k_pages"]).transpose(2, 3)
    s = s.reshape(hkv, B, G, S, L).masked_fill(~see[None, :, None], float("-inf"))
    m = torch.maximum(m1, s.amax(-1, keepdim=True))
    e = torch.exp(s - m)
    f = torch.exp(m1 - m)
    total = f * l1 + e.sum(-1, keepdim=True)
    o = (f * o1 + (e.reshape(hkv, B, G * S, L) @ v).reshape(hkv, B, G, S, d)) / total
    lse = (m + torch.log(total))[..., 0]
    live = i[None, :] < n[:, None]
    o = torch.where(live[:, :, None, None], o.permute(1, 3, 0, 2, 4).reshape(B, S, hq, d), 0.0)
    lse = torch.where(live[:, :, None], lse.permute(1, 3, 0, 2).reshape(B, S, hq), float("-inf"))
    return {"o": o.to(q.dtype), "lse": lse}


def _plain_verify(st):
    """In 64 bits where a token's weight is set against a random number."""
    case = st["case"]
    B, S, V = case["B"], case["S"], case["V"]
    x = st["logits"].double()
    t = st["temperature"].double()
    warm = t > 0
    e = torch.exp((x - x.amax(-1, keepdim=True)) / torch.where(warm, t, 1.0)[:, None, None])
    p = e / e.sum(-1, keepdim=True)
    v = torch.arange(V, device=DEV)
    best = torch.where(x == x.amax(-1, keepdim=True), v, V).amin(-1)  # the lowest of equals
    p = torch.where(warm[:, None, None], p, (v == best[..., None]).double())
    d, n = st["drafts"].long(), st["n_drafts"].long()
    pd = p[:, :S - 1].gather(2, d[..., None])[..., 0]
    qd = 1.0 if st["draft_probs"] is None else st["draft_probs"].gather(2, d[..., None])[..., 0].double()
    i = torch.arange(S - 1, device=DEV)
    ok = (st["uniforms"][:, :S - 1].double() * qd < pd) & (i < n[:, None])
    accepted = torch.cumprod(ok.long(), 1).sum(1)
    b = torch.arange(B, device=DEV)
    row = p[b, accepted]
    if S > 1:
        at = accepted.clamp(max=S - 2)
        miss = (accepted < n)[:, None]
        less = (v == d[b, at][:, None]).double() if st["draft_probs"] is None else st["draft_probs"][b, at].double()
        rest = (row - less).clamp(min=0.0) if st["draft_probs"] is not None else row * (1.0 - less)
        row = torch.where(miss & (rest.sum(-1, keepdim=True) > 0), rest, row)
    cum = torch.cumsum(row, -1)
    token = torch.where(cum > st["uniforms"][:, S - 1:].double() * cum[:, -1:], v, V).amin(-1)
    st["accepted"].copy_(accepted)
    st["next"].copy_(token)
    return {"accepted": st["accepted"], "next": st["next"]}


# ---- the same in 64 bits, from the definitions -------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"pages": _exact_pages, "rope": _exact_rope, "prefix": _exact_prefix,
            "verify": _exact_verify}[case["op"]](case, st)


def _exact_pages(case, st):
    """Request by request on a stack; giving the same pages back restores it."""
    page, T = case["page"], case["T"]
    stack = st["free"].tolist()
    top = int(st["n_free"])
    table = st["table"].tolist()
    granted, positions, slots = [], [], []
    for b, (c, r, h) in enumerate(zip(st["ctx"].tolist(), st["n"].tolist(), st["held"].tolist())):
        row = table[b][:h]
        while len(row) < -(-(c + r) // page):
            top -= 1
            row.append(stack[top])
        granted.append(r)
        positions.append([c + t if t < r else -1 for t in range(T)])
        slots.append([row[(c + t) // page] * page + (c + t) % page if t < r else -1 for t in range(T)])
    return {"granted": _ints(granted), "positions": _ints(positions), "slots": _ints(slots), "table": st["table"],
            "held": st["held"], "free": st["free"], "n_free": st["n_free"]}


def _exact_rope(case, st):
    """A rotated pair is a complex number times a unit one."""
    rot, page = case["rot"], case["page"]
    pos = st["positions"].long()
    out = {k: st[k].double() for k in ("q_out", "k_pages", "v_pages")}
    for b in range(case["B"]):
        at = (pos[b] >= 0).nonzero()[:, 0]
        angle = torch.outer(pos[b, at].double(), st["frequencies"])
        unit = torch.polar(torch.full_like(angle, st["amplitude"]), angle)[:, None]

        def turned(x, weight):
            x = x[b, at].double()
            if weight is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + st["eps"]) * weight.double()
            head, tail = x[..., :rot], x[..., rot:]
            pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" \
                else head.unflatten(-1, (rot // 2, 2))
            z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * unit)
            z = z.transpose(-1, -2) if case["layout"] == "half" else z
            return torch.cat([z.flatten(-2), tail], -1)

        out["q_out"][b, at] = turned(st["q"], st["q_weight"])
        where = st["slots"][b, at].long()
        out["k_pages"][where // page, :, where % page] = turned(st["k"], st["k_weight"])
        out["v_pages"][where // page, :, where % page] = st["v"][b, at].double()
    return out


def _exact_prefix(case, st):
    B, S, hq, hkv, page, P = (case[k] for k in ("B", "S", "Hq", "Hkv", "page", "prefix"))
    G = hq // hkv
    o = torch.zeros((B, S, hq, case["D"]), dtype=torch.float64, device=DEV)
    lse = torch.full((B, S, hq), float("-inf"), dtype=torch.float64, device=DEV)
    front = torch.arange(P, device=DEV)
    front_ids = st["prefix_table"].long()[front // page]
    for h in range(hkv):
        k0 = st["k_pages"][front_ids, h, front % page].double()
        v0 = st["v_pages"][front_ids, h, front % page].double()
        for b in range(B):
            c, n = int(st["ctx"][b]), int(st["n"][b])
            where = torch.arange(c + n, device=DEV)
            ids = st["table"][b].long()[where // page]
            k = torch.cat([k0, st["k_pages"][ids, h, where % page].double()])
            v = torch.cat([v0, st["v_pages"][ids, h, where % page].double()])
            see = torch.ones((n, P + c + n), dtype=torch.bool, device=DEV)
            words = [(1 << i + 1) - 1 for i in range(S)] if st["mask"] is None else st["mask"][b].tolist()
            see[:, P + c:] = torch.tensor([[bool(words[i] >> j & 1) for j in range(n)] for i in range(n)], device=DEV)
            rows = st["q"][b, :n, h * G:h * G + G].double().reshape(n * G, -1)
            s = (rows @ k.T * st["scale"]).reshape(n, G, -1)
            s = torch.where(see[:, None], s, float("-inf"))
            z = torch.logsumexp(s, -1)
            o[b, :n, h * G:h * G + G] = (torch.exp(s - z[..., None]).reshape(n * G, -1) @ v).reshape(n, G, -1)
            lse[b, :n, h * G:h * G + G] = z
    return {"o": o, "lse": lse}


def _exact_verify(case, st):
    """Request by request: test after test, then the draw by a search in the running sum."""
    S = case["S"]
    accepted, tokens = [], []
    for b in range(case["B"]):
        temp, u = float(st["temperature"][b]), st["uniforms"][b].tolist()

        def target(i):
            x = st["logits"][b, i].double()
            if temp > 0:
                return torch.softmax(x / temp, 0)
            one = torch.zeros_like(x)
            one[int((x == x.max()).nonzero()[0])] = 1.0
            return one

        weights = None
        for i in range(int(st["n_drafts"][b])):
            p, token = target(i), int(st["drafts"][b, i])
            if st["draft_probs"] is None:
                q = torch.zeros_like(p)
                q[token] = 1.0
            else:
                q = st["draft_probs"][b, i].double()
            if not u[i] * float(q[token]) < float(p[token]):
                weights = torch.relu(p - q)
                weights = weights if float(weights.sum()) > 0 else p
                break
        else:
            i = int(st["n_drafts"][b])
        running = torch.cumsum(target(i) if weights is None else weights, 0)
        accepted.append(i)
        tokens.append(int(torch.searchsorted(running, u[S - 1] * running[-1], right=True)))
    return {"accepted": _ints(accepted), "next": _ints(tokens)}
