"""Measured cases of the attention block between its projections: norms of
queries and keys for each head and their rotation, with keys and values
appended to the paged cache in the same pass (`deft_qkv_write`), the same into
a cache held in 4 bits (`deft_qkv_write4`), pages of that cache as bf16 pages
(`deft_kv_unpack4`) and a tree-attention step that reads it
(`deft_tree_attn4`).

The 4-bit cache: 16 consecutive elements of a token's head share a scale s,
held in e4m3; an element is a 4-bit float (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and stands for element * s * g, with
one fp32 g for K and one for V.  A page of one head is 8 * head_dim bytes of
elements, [16 tokens][head_dim / 2], the even element in the low half of a
byte, and then head_dim bytes of scales, [16 tokens][head_dim / 16].

`run` computes every operator in plain torch operations; with `own` true it
makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
BLOCK = 16      # elements that share a scale
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attn(name, **kw):
    c = {"op": "attn4", "name": name, "roots": 1, "root_lo": 1, "root_hi": 1, "levels": 1, "branches": 0, "len_lo": 1, "len_hi": 1,
         "queries": 0, "every_node": False, "kv_heads": 8, "group": 4, "head_dim": 128, "chunk": 256, "k_scale": 1.0, "v_scale": 1.0,
         "shuffle": False, "lens_seed": 4}
    c.update(kw)
    return c


def _write(op, name, **kw):
    c = {"op": op, "name": name, "tokens": 1, "kv_heads": 8, "group": 4, "head_dim": 128, "rot_dim": 128, "interleaved": False, "norm": True,
         "f32": False, "skip": 0, "k_scale": 1.0, "v_scale": 1.0}
    c.update(kw)
    return c


def listed():
    return [
        # The smallest tree of the benchmark (a 128-token root, two levels of
        # short nodes, 4 heads of 64): a step is its launches and latency.
        _attn("attn4 tiny tree", root_lo=128, root_hi=128, levels=3, branches=2, len_lo=8, len_hi=16, kv_heads=4, group=1, head_dim=64),
        # The few-shot workload's step: one 4096-token prefix read for 32
        # queries, 32 branches of 256 tokens read for one each, no grouping.
        _attn("attn4 few-shot", root_lo=4096, root_hi=4096, levels=2, branches=32, len_lo=256, len_hi=256, kv_heads=32, group=1),
        # The reasoning workload's step: four levels of 100-600 token nodes,
        # 128 queries at the leaves, grouped heads, pages in random order.
        _attn("attn4 reasoning", root_lo=100, root_hi=600, levels=4, branches=4, len_lo=100, len_hi=600, queries=128, shuffle=True),
        # One long document with 64 ragged branches (the imbalance workload's
        # shape with a quarter of its branches).
        _attn("attn4 long", root_lo=32768, root_hi=32768, levels=2, branches=64, len_lo=64, len_hi=8192, shuffle=True, k_scale=0.5, v_scale=0.7),
        # A decode step of 64 requests of very different lengths, one token
        # each and nothing shared but the grouped heads.
        _attn("attn4 single tokens", roots=64, root_lo=64, root_hi=8192, shuffle=True),
        # The new tokens of a decode step of 256 requests, bf16 cache.
        _write("write", "qkv step", tokens=256),
        # A 32768-token prefill, views of the fused projection's output.
        _write("write", "qkv prompts", tokens=32768),
        # An odd number of fp32 rows with heads of 64, a quarter of each
        # rotated in neighbouring pairs, no norms, some of them padding.
        _write("write", "qkv f32 d64", tokens=10007, kv_heads=4, group=3, head_dim=64, rot_dim=16, interleaved=True, norm=False, f32=True, skip=500),
        # A prefill into the 4-bit cache, whose pages are then read back as
        # the bf16 pages that the prompts' attention takes.
        _write("write4", "qkv4 prompts", tokens=16384),
        # An odd batch with heads of 64, half of each rotated, scaled caches.
        _write("write4", "qkv4 d64", tokens=3001, kv_heads=4, group=3, head_dim=64, rot_dim=32, k_scale=0.37, v_scale=0.125, skip=100),
        # The cached pages of a batch of requests before their next chunk.
        {"op": "unpack4", "name": "unpack4 requests", "pages": 6007, "pool": 9000, "kv_heads": 8, "head_dim": 128, "k_scale": 1.0, "v_scale": 1.0},
        # One short request of a small model.
        {"op": "unpack4", "name": "unpack4 small", "pages": 9, "pool": 64, "kv_heads": 4, "head_dim": 64, "k_scale": 0.3, "v_scale": 2.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn4", "attn4", "attn4", "write", "write4", "unpack4"])
    kv, group, d = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128])
    scales = {"k_scale": rng.choice([1.0, 1.0, 0.25, round(rng.uniform(0.05, 4), 4)]), "v_scale": rng.choice([1.0, 1.0, 0.25, round(rng.uniform(0.05, 4), 4)])}
    seed = rng.randrange(1 << 30)
    if op == "unpack4":
        pages = _log(rng, 1, 6007)
        return {"op": op, "pages": pages, "pool": pages + _log(rng, 1, 3000), "kv_heads": min(kv, 8), "head_dim": d, **scales}
    if op in ("write", "write4"):
        tokens = _log(rng, 1, 16384)
        c = _write(op, "", tokens=tokens, kv_heads=min(kv, 8), group=min(group, 4), head_dim=d, rot_dim=rng.choice([0, 16, d // 2, d, d]),
                   interleaved=rng.random() < 0.4, norm=rng.random() < 0.6, f32=rng.random() < 0.3, skip=rng.choice([0, 0, tokens // 7]))
        if op == "write4":
            c.update(scales)
        del c["name"]
        return c
    c = _attn("", kv_heads=kv, group=group, head_dim=d, chunk=rng.choice([64, 256, 256, 500, 1024]), shuffle=rng.random() < 0.5, lens_seed=seed,
              **scales)
    del c["name"]
    form = rng.choice(["tree", "tree", "requests", "speculative"])
    if form == "requests":
        hi = _log(rng, 1, 16384)
        c.update(roots=_log(rng, 1, 128), root_lo=_log(rng, 1, hi), root_hi=hi)
    elif form == "tree":
        hi, top = _log(rng, 1, 2048), _log(rng, 1, 16384)
        c.update(root_lo=_log(rng, 1, top), root_hi=top, levels=rng.choice([2, 2, 3, 4]), branches=rng.choice([1, 2, 3, 4]), len_lo=_log(rng, 1, hi),
                 len_hi=hi, queries=_log(rng, 1, 128))
    else:
        # one-token nodes under each request's context, every node a query
        hi = _log(rng, 16, 8192)
        c.update(roots=_log(rng, 1, 8), root_lo=_log(rng, 1, hi), root_hi=hi, levels=rng.choice([2, 3, 4]), branches=rng.choice([1, 2, 3]), every_node=True)
    # No dearer than the long document, dense products of at most 300 million
    # logits: the lengths are halved until the case fits.
    most = work(listed()[3])
    while any(work(c)[m] > most[m] for m in most) or _dense(c) > 300e6:
        c["root_hi"] = max(1, c["root_hi"] // 2)
        c["root_lo"] = min(c["root_lo"], c["root_hi"])
        c["roots"] = max(1, c["roots"] * 3 // 4)
        if c["root_hi"] < 16:
            c["len_hi"] = max(1, c["len_hi"] // 2)
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
            c["kv_heads"] = max(1, c["kv_heads"] // 2)
    return c


def _tree(c):
    """parent and length of every node, and the node of every query, from the case alone."""
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
    if c["every_node"]:
        level = [n for n in range(len(parent)) if c["levels"] == 1 or parent[n] >= 0]
    return parent, length, [level[i % len(level)] for i in range(c["queries"] or len(level))]


def _above(parent, length):
    """Tokens on each node's path, its own included (parents come first)."""
    total = []
    for p, n in zip(parent, length):
        total.append(n + (0 if p < 0 else total[p]))
    return total


def _dense(c):
    parent, length, query = _tree(c)
    return len(query) * sum(length) * c["kv_heads"] * c["group"]


def work(case):
    c = case
    d, kv = c["head_dim"], c["kv_heads"]
    if c["op"] == "unpack4":
        return {"bytes": c["pages"] * (kv * 2 * (9 * d + 32 * d) + 4), "flops": 0}
    heads = kv * c["group"]
    row = 2 * kv * d
    if c["op"] in ("write", "write4"):
        es, kept = (4 if c["f32"] else 2), c["tokens"] - c["skip"]
        # q read and written, K and V read and written, slot and position, the
        # rows of the rotation's table that are used
        b = c["tokens"] * heads * d * (es + 2) + kept * row * es + c["tokens"] * (8 + 4 * c["rot_dim"])
        b += kept * row * 9 // 16 if c["op"] == "write4" else kept * row * 2
        if c["op"] == "write4":     # the pages read again and written as bf16
            b += -(-c["tokens"] // PAGE) * (kv * 2 * (9 * d + 32 * d) + 4)
        return {"bytes": b, "flops": 0}
    parent, length, query = _tree(c)
    path = _above(parent, length)
    rows, tokens = len(query), sum(length)
    used, pages = tokens * row * 9 // 16, sum(-(-x // PAGE) for x in length)
    b = used + rows * heads * (4 * d + 4) + 4 * pages
    return {"bytes": b, "flops": 4 * sum(path[n] for n in query) * heads * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _angles(rot, positions, base=10000.0):
    """cos and sin of every position's angles, [positions, rot]."""
    if not rot:
        return None
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _cache4(g, pages, kv, d, scale):
    """A 4-bit pool filled with quantised activations of unit variance."""
    x = _randn(g, pages * kv * PAGE, d).to(torch.bfloat16).float()
    codes, s = _quantise(x, scale)
    return torch.cat([codes.view(pages, kv, 8 * d), s.view(pages, kv, d)], 2)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kv, d = c["kv_heads"], c["head_dim"]
    if c["op"] == "unpack4":
        shape = (c["pages"], kv, PAGE, d)
        return {"op": "unpack4", "k4": _cache4(g, c["pool"], kv, d, c["k_scale"]), "v4": _cache4(g, c["pool"], kv, d, c["v_scale"]),
                "page_id": _i32(np.random.default_rng(seed).permutation(c["pool"])[:c["pages"]]), "scales": (c["k_scale"], c["v_scale"]),
                "k_pages": torch.empty(shape, dtype=torch.bfloat16, device="cuda"), "v_pages": torch.empty(shape, dtype=torch.bfloat16, device="cuda")}
    if c["op"] in ("write", "write4"):
        tokens = c["tokens"]
        s = _new_rows(c, g, tokens)
        pages = -(-tokens // PAGE)
        rng = np.random.default_rng(seed)
        if c["op"] == "write" and tokens <= 4096:       # a decode step: single slots of many pages
            pool = pages + tokens // 2 + 64
            slot = rng.permutation(pool * PAGE)[:tokens]
            at = np.full(tokens, 5000) - rng.integers(0, 5000, tokens)
        else:                                           # prompts: whole pages in any order
            pool = pages + 64
            ids = rng.permutation(pool)[:pages]
            slot = (ids[:, None] * PAGE + np.arange(PAGE)).reshape(-1)[:tokens]
            at = np.arange(tokens)
            s["page_id"] = _i32(ids)
        slot[tokens - c["skip"]:] = -1
        s.update(slot=_i32(slot), position=_i32(at), cos_sin=_angles(c["rot_dim"], max(int(at.max()) + 1, 2)), scales=(c["k_scale"], c["v_scale"]))
        if c["op"] == "write":
            s["k_pages"], s["v_pages"] = (torch.zeros((pool, kv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        else:
            s["k4"], s["v4"] = (torch.zeros((pool, kv, 9 * d), dtype=torch.uint8, device="cuda") for _ in "kv")
            s["k_pages"], s["v_pages"] = (torch.empty((pages, kv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        return s
    parent, length, query = _tree(c)
    counts = [-(-x // PAGE) for x in length]
    off = np.concatenate([[0], np.cumsum(counts)])
    pool = int(off[-1]) + 3
    ids = np.random.default_rng(seed).permutation(pool)[:pool - 3] if c["shuffle"] else np.arange(pool - 3)
    rows = len(query)
    s = {"op": "attn4", "q": _randn(g, rows, kv * c["group"], d).to(torch.bfloat16), "group": c["group"], "page_off": _i32(off), "page_id": _i32(ids),
         "scales": (c["k_scale"], c["v_scale"]), "k4": _cache4(g, pool, kv, d, c["k_scale"]), "v4": _cache4(g, pool, kv, d, c["v_scale"])}
    # The plain form's index of every token and of who attends it.
    tok_page = np.concatenate([ids[o:o + n] for o, n in zip(off, counts)]).repeat(PAGE)
    place = np.concatenate([np.arange(n * PAGE) < x for n, x in zip(counts, length)])
    s["tok"] = torch.from_numpy((tok_page * PAGE + np.tile(np.arange(PAGE), len(tok_page) // PAGE))[place]).cuda()
    on = np.zeros((rows, len(length)), dtype=bool)
    for i, n in enumerate(query):
        while n >= 0:
            on[i, n] = True
            n = parent[n]
    s["seen"] = torch.from_numpy(on).cuda()
    s["tok_node"] = torch.from_numpy(np.arange(len(length)).repeat(length)).cuda()
    if own:
        # made once a step and kept for all layers of the model
        import shared_prefix_kv_deft_gb300 as deft
        s["plan"] = deft.Plan(parent, length, query, c["chunk"], c["group"], naive=False)
        s["plan"].upload()
        s["bufs"] = deft.alloc_buffers(s["plan"], rows, kv * c["group"], d)
    return s


def _new_rows(c, g, tokens):
    """One row of the fused projection a token: the query heads, then K, then V."""
    kv, d, group = c["kv_heads"], c["head_dim"], c["group"]
    dt = torch.float32 if c["f32"] else torch.bfloat16
    qkv = _randn(g, tokens, (group + 2) * kv, d).to(dt)
    s = {"op": c["op"], "q": qkv[:, :group * kv], "k": qkv[:, group * kv:(group + 1) * kv], "v": qkv[:, (group + 1) * kv:], "q_norm": None, "k_norm": None,
         "interleaved": c["interleaved"], "q_out": torch.empty((tokens, group * kv, d), dtype=torch.bfloat16, device="cuda")}
    if c["norm"]:
        s["q_norm"], s["k_norm"] = ((1 + 0.1 * _randn(g, d)).to(dt) for _ in "qk")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _own_run(s)
    if s["op"] == "unpack4":
        return _plain_unpack4(s)
    if s["op"] == "attn4":
        return _plain_attn4(s)
    q = _plain_rows(s, s["q"], s["q_norm"])
    k = _plain_rows(s, s["k"], s["k_norm"])
    v = s["v"].to(torch.bfloat16)
    held = s["slot"] >= 0
    at = s["slot"][held].long()
    if s["op"] == "write":
        s["k_pages"][at // PAGE, :, at % PAGE] = k[held]
        s["v_pages"][at // PAGE, :, at % PAGE] = v[held]
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    _plain_append4(s["k4"], at, k[held], s["scales"][0])
    _plain_append4(s["v4"], at, v[held], s["scales"][1])
    return {"q": q, **_plain_unpack4(s)}


def _own_run(s):
    import shared_prefix_kv_deft_gb300 as deft
    if s["op"] in ("write", "write4"):
        rows = {"position": s["position"], "cos_sin": s["cos_sin"], "interleaved": s["interleaved"], "q_norm": s["q_norm"], "k_norm": s["k_norm"], "eps": EPS,
                "q_out": s["q_out"]}
        if s["op"] == "write":
            q = deft.deft_qkv_write(s["q"], s["k"], s["v"], s["slot"], s["k_pages"], s["v_pages"], **rows)
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        q = deft.deft_qkv_write4(s["q"], s["k"], s["v"], s["slot"], s["k4"], s["v4"], k_scale=s["scales"][0], v_scale=s["scales"][1], **rows)
    if s["op"] in ("unpack4", "write4"):
        deft.deft_kv_unpack4(s["k4"], s["v4"], s["page_id"], s["k_pages"], s["v_pages"], k_scale=s["scales"][0], v_scale=s["scales"][1])
        pages = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return {"q": q, **pages} if s["op"] == "write4" else pages
    out, lse = deft.deft_tree_attn4(s["q"], s["k4"], s["v4"], s["page_off"], s["page_id"], s["plan"], s["bufs"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    return {"out": out, "lse": lse}


def _plain_rows(s, x, weight):
    """Heads normed by their root mean square, then rotated, as bf16."""
    x = x.float()
    d = x.shape[-1]
    if weight is not None:
        # a fixed order of the sum's additions, neighbours onto one another,
        # so that a value next to a border of the 4-bit format does not turn
        # on it
        sq = x * x
        while sq.shape[-1] > 1:
            sq = sq[..., 0::2] + sq[..., 1::2]
        x = x * (1.0 / torch.sqrt(sq / d + EPS)) * weight.float()
    if s["cos_sin"] is not None:
        half = s["cos_sin"].shape[1] // 2
        row = s["cos_sin"][s["position"].long()][:, None]
        cos, sin = row[..., :half], row[..., half:]
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        x = torch.cat([turned, x[..., 2 * half:]], -1)
    return x.to(torch.bfloat16)


def _quantise(x, g):
    """Rows [n, d] as bytes of two elements and bytes of scales."""
    n, d = x.shape
    x = x.view(n, d // BLOCK, BLOCK)
    s = (x.abs().amax(-1) / (6.0 * torch.tensor(g, device=x.device))).clamp(max=448.0).to(torch.float8_e4m3fn)
    sg = s.float() * g
    y = x / torch.where(sg > 0, sg, torch.full_like(sg, math.inf))[..., None]
    a = y.abs()
    # to the nearest element, halfway to the one with an even last bit
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    code += torch.signbit(y).byte() * 8
    code = code.view(n, d // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s.view(torch.uint8)


def _parts(pool):
    """The elements' and the scales' bytes of a 4-bit pool, [pages, heads, 16, ...]."""
    pages, heads, size = pool.shape
    d = size // 9
    return pool[..., :8 * d].view(pages, heads, PAGE, d // 2), pool[..., 8 * d:].view(pages, heads, PAGE, d // BLOCK)


def _plain_append4(pool, at, x, g):
    n, heads, d = x.shape
    codes, scales = _quantise(x.float().reshape(n * heads, d), g)
    to_codes, to_scales = _parts(pool)
    to_codes[at // PAGE, :, at % PAGE] = codes.view(n, heads, d // 2)
    to_scales[at // PAGE, :, at % PAGE] = scales.view(n, heads, d // BLOCK)


def _values(codes, scales, g):
    """What bytes of elements and of their scales stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    x = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.view(*s.shape, BLOCK) * s[..., None]).flatten(-2) * g


def _plain_unpack4(s):
    for pool, pages, g in zip((s["k4"], s["v4"]), (s["k_pages"], s["v_pages"]), s["scales"]):
        codes, scales = _parts(pool)
        at = s["page_id"].long()
        pages.copy_(_values(codes[at], scales[at].contiguous(), g).to(torch.bfloat16))
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn4(s):
    """Every query against every token, those off its path left out."""
    q = s["q"]
    rows, heads, d = q.shape
    at, group = s["tok"], s["group"]

    def tokens(pool, g):    # [heads, tokens, d]
        codes, scales = _parts(pool)
        return _values(codes[at // PAGE, :, at % PAGE].transpose(0, 1), scales[at // PAGE, :, at % PAGE].transpose(0, 1).contiguous(), g)
    k = tokens(s["k4"], s["scales"][0])
    x = q.float().view(rows, heads // group, group, d).permute(1, 2, 0, 3).reshape(heads // group, group * rows, d)
    p = torch.matmul(x * (1.0 / math.sqrt(d)), k.transpose(1, 2)).view(heads // group, group, rows, -1)
    p.masked_fill_(~s["seen"][:, s["tok_node"]], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = tokens(s["v4"], s["scales"][1])
    out = torch.matmul(p.view(heads // group, group * rows, -1), v).view(heads // group, group, rows, d) / total
    lse = (top + total.log())[..., 0]
    return {"out": out.permute(2, 0, 1, 3).reshape(rows, heads, d).to(torch.bfloat16), "lse": lse.permute(2, 0, 1).reshape(rows, heads)}


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(c, x, weight, position):
    """Norm and rotation of [tokens, heads, d] in 64 bits."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS)
    rot = c["rot_dim"]
    if rot:
        # the table's own values: angles as complex numbers of modulus one
        i = torch.arange(rot // 2, device=x.device)
        a = position.double()[:, None] * 10000.0 ** (-2.0 * i.double() / rot)
        turn = torch.complex(torch.cos(a).float().double(), torch.sin(a).float().double())[:, None]
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
    return x


def _nearest(x, grid):
    """The nearest of the grid's ascending values, halfway to one at an even place."""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])


def _exact4(x, g):
    """What the 4-bit cache holds of rows of bf16 values."""
    x = x.to(torch.bfloat16).double()
    b = x.unflatten(-1, (-1, BLOCK))
    e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)],
                        dtype=torch.float64, device=x.device)
    s = _nearest(b.abs().amax(-1, keepdim=True) / 6 / g, e4m3)
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    y = torch.where(s > 0, b.abs() / (s * g), torch.zeros_like(b))
    return (_nearest(y, e2m1) * torch.sign(b) * s * g).flatten(-2)


def _exact_pool(pool, g):
    """A 4-bit pool's values, [pages, heads, 16, d], bit by bit."""
    pages, heads, size = pool.shape
    d = size // 9
    byte = pool[..., :8 * d].long()
    code = torch.empty((pages, heads, 16 * d), dtype=torch.long, device=pool.device)
    code[..., 0::2], code[..., 1::2] = byte % 16, byte // 16
    e, m = (code // 2) % 4, code % 2
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).double()) * (1 - 2 * (code // 8))
    s = pool[..., 8 * d:].long()
    e, m = (s // 8) % 16, s % 8
    s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7).double()) * (1 - 2 * (s // 128))
    return (x.view(pages, heads, -1, BLOCK) * s[..., None] * g).view(pages, heads, PAGE, d)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    gk, gv = float(np.float32(c.get("k_scale", 1))), float(np.float32(c.get("v_scale", 1)))
    if c["op"] == "unpack4":
        at = s["page_id"].long()
        return {"k_pages": _exact_pool(s["k4"][at], gk), "v_pages": _exact_pool(s["v4"][at], gv)}
    if c["op"] in ("write", "write4"):
        q = _exact_rows(c, s["q"], s["q_norm"], s["position"])
        k = _exact_rows(c, s["k"], s["k_norm"], s["position"])
        v = s["v"].double()
        if c["op"] == "write4":
            k, v = _exact4(k, gk), _exact4(v, gv)
        out = {"q": q}
        slot = s["slot"].tolist()
        where = {int(p): i for i, p in enumerate(s["page_id"].tolist())} if c["op"] == "write4" else None
        rows = [t for t in range(len(slot)) if slot[t] >= 0]
        page = torch.tensor([where[slot[t] // PAGE] if where else slot[t] // PAGE for t in rows], device="cuda")
        place = torch.tensor([slot[t] % PAGE for t in rows], device="cuda")
        for name, x in (("k_pages", k), ("v_pages", v)):
            out[name] = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
            for h in range(x.shape[1]):
                out[name][page, h, place] = x[rows, h]
        return out
    K, V = _exact_pool(s["k4"], gk), _exact_pool(s["v4"], gv)
    parent, length, query = _tree(c)
    off, ids = s["page_off"].tolist(), s["page_id"].long()
    d, group = c["head_dim"], c["group"]
    out, lse = [], []
    for i, n in enumerate(query):
        x, keys, values = s["q"][i].double().view(-1, group, d), [], []
        while n >= 0:
            for pool, into in ((K, keys), (V, values)):
                into.append(pool[ids[off[n]:off[n + 1]]].transpose(0, 1).reshape(c["kv_heads"], -1, d)[:, :length[n]])
            n = parent[n]
        z = torch.einsum("hgd,htd->hgt", x, torch.cat(keys, 1)) / math.sqrt(d)
        norm = torch.logsumexp(z, -1)
        out.append(torch.einsum("hgt,htd->hgd", torch.exp(z - norm[..., None]), torch.cat(values, 1)).reshape(-1, d))
        lse.append(norm.reshape(-1))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
