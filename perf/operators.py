"""Measured cases of the prompt path: page tables and slot maps built on the
GPU (`deft_page_table`), K and V rows written into the pages (`deft_kv_write`)
and causal attention of whole prompts over the paged cache
(`deft_prompt_attn`).

A prompt is the last `prompt_len` tokens of a node of a token tree: each of
them attends to every token of the nodes above and to its own node up to
itself.  A forest of roots without children is a packed batch of ordinary
prompts.  `run` computes every operator in plain torch operations; with `own`
true it makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _prompt(name, **kw):
    c = {"op": "prompt", "name": name, "roots": 1, "root_lo": 1, "root_hi": 1, "levels": 1, "branches": 0, "len_lo": 1,
         "len_hi": 1, "new": 0, "kv_heads": 8, "group": 4, "head_dim": 128, "shuffle": False, "lens_seed": 4}
    c.update(kw)
    return c


def listed():
    return [
        # The smallest tree of the benchmark (a 128-token root, two levels of
        # short nodes, 4 heads of 64): one prefill of all seven nodes, where
        # the launch and the latency of one unit are all there is.
        _prompt("prompt tiny tree", root_lo=128, root_hi=128, levels=3, branches=2, len_lo=8, len_hi=16, kv_heads=4,
                group=1, head_dim=64),
        # The few-shot workload's prefill: the shared 4096-token prefix and
        # its 32 examples of 256 tokens in one batch, 32 heads without
        # grouping.
        _prompt("prompt few-shot", root_lo=4096, root_hi=4096, levels=2, branches=32, len_lo=256, len_hi=256,
                kv_heads=32, group=1),
        # The reasoning workload's prefill: four levels of 100-600 token
        # steps under one another, grouped heads, pages in random order.
        _prompt("prompt reasoning tree", root_lo=100, root_hi=600, levels=4, branches=4, len_lo=100, len_hi=600,
                shuffle=True),
        # One long document, the prefix of the imbalance workload.
        _prompt("prompt long", root_lo=32768, root_hi=32768),
        # Chunked prefill: the next 512 tokens of eight requests that have up
        # to 16k tokens in the cache.
        _prompt("prompt chunk", roots=8, root_lo=5000, root_hi=16384, new=512, shuffle=True),
        # A decode step through the same call: one token of each of 64
        # requests of very different lengths.
        _prompt("prompt single token", roots=64, root_lo=64, root_hi=8192, new=1, shuffle=True),
        # A packed batch of ragged prompts of one token to some thousand,
        # heads of 64, an odd group.
        _prompt("prompt packed d64", roots=24, root_lo=1, root_hi=3000, kv_heads=4, group=3, head_dim=64),
        # A decode step's bookkeeping: 256 requests grow by one token each.
        {"op": "table", "name": "table step", "nodes": 256, "len_lo": 64, "len_hi": 8192, "prev": 1, "grow": 1, "pad": 0, "lens_seed": 5},
        # The bookkeeping of a large prefill with a padded token batch.
        {"op": "table", "name": "table prompts", "nodes": 20000, "len_lo": 1, "len_hi": 400, "prev": 0, "grow": 0, "pad": 4099,
         "lens_seed": 6},
        # The K and V of one decode step of 256 requests.
        {"op": "write", "name": "write step", "tokens": 256, "kv_heads": 8, "group": 4, "head_dim": 128, "f32": False, "skip": 0, "lens_seed": 7},
        # A 32768-token prefill's K and V, views of the fused projection's output.
        {"op": "write", "name": "write prompts", "tokens": 32768, "kv_heads": 8, "group": 4, "head_dim": 128, "f32": False, "skip": 0,
         "lens_seed": 8},
        # An odd number of fp32 rows with heads of 64, some of them padding.
        {"op": "write", "name": "write f32 d64", "tokens": 10007, "kv_heads": 4, "group": 3, "head_dim": 64, "f32": True, "skip": 500,
         "lens_seed": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "table", "write"])
    seed = rng.randrange(1 << 30)
    if op == "table":
        nodes = _log(rng, 1, 20000)
        hi = _log(rng, 1, max(1, min(8192, 4000000 // nodes)))
        return {"op": op, "nodes": nodes, "len_lo": _log(rng, 1, hi), "len_hi": hi, "prev": rng.randrange(2), "grow": _log(rng, 1, 64),
                "pad": rng.choice([0, 1, 37, 4099]), "lens_seed": seed}
    kv, group, d = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128])
    if op == "write":
        tokens = _log(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "kv_heads": min(kv, 8), "group": min(group, 4), "head_dim": d, "f32": rng.random() < 0.3,
                "skip": rng.choice([0, 0, tokens // 7]), "lens_seed": seed}
    c = _prompt("", kv_heads=kv, group=group, head_dim=d, shuffle=rng.random() < 0.5, lens_seed=seed)
    del c["name"]
    form = rng.choice(["packed", "tree", "tree", "chunk", "token"])
    if form == "packed":
        hi = _log(rng, 1, 16384)
        c.update(roots=_log(rng, 1, 64), root_lo=_log(rng, 1, hi), root_hi=hi)
    elif form == "tree":
        hi, top = _log(rng, 1, 1024), _log(rng, 1, 8192)
        c.update(root_lo=_log(rng, 1, top), root_hi=top, levels=rng.choice([2, 2, 3, 4]), branches=rng.choice([1, 2, 3, 4]), len_lo=_log(rng, 1, hi),
                 len_hi=hi)
    else:
        hi = _log(rng, 16, 16384)
        c.update(roots=_log(rng, 1, 64), root_lo=_log(rng, 1, hi), root_hi=hi, new=1 if form == "token" else _log(rng, 2, 1024))
    # No dearer than the long prompt, and a cache of at most 4 GB: the
    # lengths are halved until the case fits.
    most = work(listed()[3])["flops"]
    while work(c)["flops"] > most or _cache_bytes(c) > 4 << 30:
        c["root_hi"] = max(1, c["root_hi"] // 2)
        c["root_lo"] = min(c["root_lo"], c["root_hi"])
        c["roots"] = max(1, c["roots"] * 3 // 4)
    return c


def _tree(c):
    """parent, length of every node and the prompt length of every node (all
    nodes are prompts), from the case alone."""
    rng = random.Random(c["lens_seed"])
    parent, length, level = [], [], []
    for _ in range(c["roots"]):
        parent.append(-1)
        length.append(_log(rng, c["root_lo"], c["root_hi"]))
        level.append(len(parent) - 1)
    for _ in range(c["levels"] - 1):
        below = []
        for n in level:
            for _ in range(c["branches"]):
                parent.append(n)
                length.append(_log(rng, c["len_lo"], c["len_hi"]))
                below.append(len(parent) - 1)
        level = below
    new = [min(c["new"], x) if c["new"] else x for x in length]
    return parent, length, new


def _context(parent, length):
    """Tokens above each node (parents come before their children)."""
    above = []
    for p in parent:
        above.append(0 if p < 0 else above[p] + length[p])
    return above


def _cache_bytes(c):
    return sum(-(-x // PAGE) * PAGE for x in _tree(c)[1]) * c["kv_heads"] * c["head_dim"] * 4


def _table_lens(c):
    rng = random.Random(c["lens_seed"])
    length = [_log(rng, c["len_lo"], c["len_hi"]) for _ in range(c["nodes"])]
    prev = [max(0, x - c["grow"]) for x in length] if c["prev"] else [0] * len(length)
    return length, prev


def work(case):
    c = case
    if c["op"] == "table":
        length, prev = _table_lens(c)
        pages = sum(-(-x // PAGE) for x in length)
        new = sum(x - p for x, p in zip(length, prev))
        nodes = len(length)
        # lengths (and the earlier lengths and offsets) read, every page id
        # read once and written once, both offset arrays and the slots written
        return {"bytes": 4 * (nodes * (3 if c["prev"] else 1) + 2 * pages + 2 * (nodes + 1) + new + c["pad"] + 4), "flops": 0}
    if c["op"] == "write":
        kept = c["tokens"] - c["skip"]
        row = c["kv_heads"] * c["head_dim"]
        return {"bytes": 4 * c["tokens"] + kept * 2 * row * ((4 if c["f32"] else 2) + 2), "flops": 0}
    parent, length, new = _tree(c)
    above = _context(parent, length)
    heads, d = c["kv_heads"] * c["group"], c["head_dim"]
    rows = sum(new)
    pairs = sum(m * (a + x - m) + m * (m + 1) // 2 for a, x, m in zip(above, length, new))
    tokens = sum(length)
    return {"bytes": rows * heads * (4 * d + 4) + tokens * c["kv_heads"] * d * 4 + 4 * sum(-(-x // PAGE) for x in length),
            "flops": 4 * pairs * heads * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pages(counts, shuffle, seed, spare):
    """node_page_off and page_id for nodes of these page counts."""
    off = np.zeros(len(counts) + 1, dtype=np.int64)
    off[1:] = np.cumsum(counts)
    total = int(off[-1])
    ids = np.random.default_rng(seed).permutation(total + spare)[:total] if shuffle else np.arange(total)
    return off, ids, total + spare


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "table":
        length, prev = _table_lens(c)
        pages = [-(-x // PAGE) for x in length]
        kept = [-(-x // PAGE) for x in prev]
        total, need, new = sum(pages), sum(pages) - sum(kept), sum(length) - sum(prev)
        # the pool hands out pages in any order; a few are left over
        ids = np.random.default_rng(seed).permutation(total + 7)
        s = {"op": "table", "prev": bool(c["prev"]), "total": total, "new": new, "node_len": _i32(length),
             "prev_len": _i32(prev), "prev_off": _i32(np.concatenate([[0], np.cumsum(kept)])), "prev_id": _i32(ids[:max(1, sum(kept))]),
             "free": _i32(ids[sum(kept):sum(kept) + need + 7]),
             "page_off": torch.empty(len(length) + 1, dtype=torch.int32, device="cuda"),
             "page_id": torch.empty(total, dtype=torch.int32, device="cuda"),
             "tok_off": torch.empty(len(length) + 1, dtype=torch.int32, device="cuda"),
             "slot": torch.empty(new + c["pad"], dtype=torch.int32, device="cuda"),
             "counts": torch.empty(4, dtype=torch.int32, device="cuda")}
        if own:
            import shared_prefix_kv_deft_gb300 as deft
            s["table"] = deft.PageTable(s["page_off"], s["page_id"], s["tok_off"], s["slot"], s["counts"], deft.page_table_workspace(len(length)))
        return s
    if c["op"] == "write":
        kv, d, tokens = c["kv_heads"], c["head_dim"], c["tokens"]
        dt = torch.float32 if c["f32"] else torch.bfloat16
        # one row of the fused projection: the query heads, then K, then V
        qkv = torch.randn((tokens, (c["group"] + 2) * kv, d), generator=g, device="cuda", dtype=torch.float32).to(dt)
        pages = -(-tokens // PAGE) + 64
        rng = np.random.default_rng(seed)
        if tokens <= 4096:      # a decode step: single slots of many pages
            pages += tokens // 2
            slot = rng.permutation(pages * PAGE)[:tokens]
        else:                   # prompts: whole pages in any order
            slot = (rng.permutation(pages)[:-(-tokens // PAGE), None] * PAGE + np.arange(PAGE)).reshape(-1)[:tokens]
        slot[tokens - c["skip"]:] = -1
        return {"op": "write", "k": qkv[:, c["group"] * kv:(c["group"] + 1) * kv], "v": qkv[:, (c["group"] + 1) * kv:], "slot": _i32(slot),
                "k_pages": torch.zeros((pages, kv, PAGE, d), dtype=torch.bfloat16, device="cuda"),
                "v_pages": torch.zeros((pages, kv, PAGE, d), dtype=torch.bfloat16, device="cuda")}
    parent, length, new = _tree(c)
    kv, group, d = c["kv_heads"], c["group"], c["head_dim"]
    off, ids, pool = _pages([-(-x // PAGE) for x in length], c["shuffle"], seed, 3)
    shape = (pool, kv, PAGE, d)
    # activations as a model's normalised projections have them: unit
    # variance, logits of order one
    s = {"op": "prompt", "parent": parent, "length": length, "new": new, "kv_heads": kv, "group": group, "head_dim": d,
         "q": torch.randn((sum(new), kv * group, d), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16),
         "k_pages": torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16),
         "v_pages": torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16),
         "node_page_off": _i32(off), "page_id": _i32(ids)}
    if own:
        # made once a step and kept for all layers of the model
        import shared_prefix_kv_deft_gb300 as deft
        s["plan"] = deft.PromptPlan(parent, length, list(range(len(parent))), kv, group, prompt_len=new)
        s["plan"].upload()
        s["bufs"] = deft.alloc_buffers(s["plan"], sum(new), kv * group, d)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import shared_prefix_kv_deft_gb300 as deft
        if s["op"] == "table":
            t = deft.deft_page_table(s["node_len"], s["free"], prev=(s["prev_len"], s["prev_off"], s["prev_id"]) if s["prev"] else None,
                                     table=s["table"])
            return {"page_off": t.page_off, "page_id": t.page_id, "tok_off": t.tok_off, "slot": t.slot, "counts": t.counts}
        if s["op"] == "write":
            deft.deft_kv_write(s["k"], s["v"], s["slot"], s["k_pages"], s["v_pages"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        out, lse = deft.deft_prompt_attn(s["q"], s["k_pages"], s["v_pages"], s["node_page_off"], s["page_id"], s["plan"], s["bufs"])
        return {"out": out, "lse": lse}
    return {"table": _plain_table, "write": _plain_write, "prompt": _plain_prompt}[s["op"]](s)


def _offsets(n):
    return torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])


def _plain_table(s):
    length = s["node_len"].long()
    prev = s["prev_len"].long() if s["prev"] else torch.zeros_like(length)
    pages = (length + PAGE - 1) // PAGE
    kept = torch.minimum((prev + PAGE - 1) // PAGE, pages)
    new = (length - prev).clamp(min=0)
    page_off, tok_off, take_off = _offsets(pages), _offsets(new), _offsets(pages - kept)
    nodes = torch.arange(length.numel(), device=length.device)
    n = torch.repeat_interleave(nodes, pages, output_size=s["total"])
    j = torch.arange(s["total"], device=length.device) - page_off[n]
    page_id = s["free"].long()[(take_off[n] + (j - kept[n]).clamp(min=0)).clamp(max=s["free"].numel() - 1)]
    if s["prev"]:
        old = s["prev_id"].long()
        page_id = torch.where(j < kept[n], old[(s["prev_off"].long()[n] + j).clamp(max=old.numel() - 1)], page_id)
    n = torch.repeat_interleave(nodes, new, output_size=s["new"])
    t = prev[n] + torch.arange(s["new"], device=length.device) - tok_off[n]
    slot = torch.full_like(s["slot"], -1)
    slot[:s["new"]] = (page_id[page_off[n] + t // PAGE] * PAGE + t % PAGE).int()
    counts = torch.stack([page_off[-1], take_off[-1], tok_off[-1], torch.zeros_like(tok_off[-1])])
    return {"page_off": page_off.int(), "page_id": page_id.int(), "tok_off": tok_off.int(), "slot": slot, "counts": counts.int()}


def _plain_write(s):
    held = s["slot"] >= 0
    at = s["slot"][held].long()
    s["k_pages"][at // PAGE, :, at % PAGE] = s["k"][held].to(torch.bfloat16)
    s["v_pages"][at // PAGE, :, at % PAGE] = s["v"][held].to(torch.bfloat16)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _path(parent, n):
    return ([] if parent[n] < 0 else _path(parent, parent[n])) + [n]


def _rows(s, n, begin, end, q):
    """Rows begin..end-1 (positions in node n) against the path's tokens."""
    path = _path(s["parent"], n)
    seen = [s["length"][x] for x in path[:-1]] + [end]
    at = torch.cat([s["node_page_off"][x] * PAGE + torch.arange(m, device=q.device) for x, m in zip(path, seen)])
    page = s["page_id"].long()[at // PAGE]
    k = s["k_pages"][page, :, at % PAGE].float().permute(1, 2, 0)     # [heads, d, tokens]
    v = s["v_pages"][page, :, at % PAGE].float().permute(1, 0, 2)     # [heads, tokens, d]
    m, d = end - begin, s["head_dim"]
    x = q.float().view(m, s["kv_heads"], s["group"], d).permute(1, 2, 0, 3).reshape(s["kv_heads"], s["group"] * m, d)
    p = torch.matmul(x * (1.0 / math.sqrt(d)), k).view(s["kv_heads"], s["group"], m, -1)
    own_at = torch.arange(end, device=q.device)
    p[..., -end:].masked_fill_(own_at[None, :] > own_at[begin:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(s["kv_heads"], s["group"] * m, -1), v).view(s["kv_heads"], s["group"], m, d) / total
    lse = (top + total.log())[..., 0]
    return out.permute(2, 0, 1, 3).reshape(m, -1, d).to(torch.bfloat16), lse.permute(2, 0, 1).reshape(m, -1)


def _plain_prompt(s):
    first = [sum(s["new"][:n]) for n in range(len(s["new"]))]
    done = [_rows(s, n, b, min(b + 4096, x), s["q"][f + b - (x - m):f + min(b + 4096, x) - (x - m)])
            for n, (x, m, f) in enumerate(zip(s["length"], s["new"], first)) for b in range(x - m, x, 4096)]
    return {"out": torch.cat([o for o, _ in done]), "lse": torch.cat([z for _, z in done])}


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] == "table":
        return None     # whole numbers: compared as they are
    s = prepare(case, seed)
    if c["op"] == "write":
        out = {}
        slot = s["slot"].cpu().numpy()
        for name in ("k", "v"):
            rows = s[name].double().cpu().numpy()
            pages = np.zeros(s[name + "_pages"].shape)
            for t in range(len(slot)):
                if slot[t] >= 0:
                    pages[slot[t] >> 4, :, slot[t] & 15] = rows[t]
            out[name + "_pages"] = torch.from_numpy(pages)
        return out
    parent, length, new = _tree(c)
    d, group = c["head_dim"], c["group"]
    heads = c["kv_heads"] * group
    off, ids = s["node_page_off"].cpu().tolist(), s["page_id"].long()
    # tokens of every node in order, [heads, tokens, d]
    def tokens(pool, n):
        x = pool[ids[off[n]:off[n + 1]]].transpose(1, 2).reshape(-1, c["kv_heads"], d)
        return x[:length[n]].double().transpose(0, 1)
    out = torch.empty((sum(new), heads, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((sum(new), heads), dtype=torch.float64, device="cuda")
    row = 0
    for n in range(len(parent)):
        chain, a = [], n
        while a >= 0:
            chain.insert(0, a)
            a = parent[a]
        keys = torch.cat([tokens(s["k_pages"], a) for a in chain], 1)
        values = torch.cat([tokens(s["v_pages"], a) for a in chain], 1)
        before = keys.shape[1] - length[n]
        step = max(1, min(1024, (1 << 28) // keys.shape[1]))
        for b in range(length[n] - new[n], length[n], step):
            e = min(b + step, length[n])
            seen = before + e
            hidden = torch.arange(seen, device="cuda")[None, :] > before + torch.arange(b, e, device="cuda")[:, None]
            for h in range(heads):
                x = torch.einsum("id,jd->ij", s["q"][row:row + e - b, h].double(), keys[h // group, :seen]) / math.sqrt(d)
                x[hidden] = -math.inf
                z = torch.logsumexp(x, 1)
                out[row:row + e - b, h] = torch.exp(x - z[:, None]) @ values[h // group, :seen]
                lse[row:row + e - b, h] = z
            row += e - b
    return {"out": out, "lse": lse}
