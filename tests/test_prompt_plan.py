"""The prompt plan (deft_prompt_plan) on the CPU: what its items cover, how
units are dealt, what it refuses, and the argument checks of the calls around
it that need no GPU."""
from __future__ import annotations

import ctypes
import random
import time

import numpy as np
import pytest

import shared_prefix_kv_deft_gb300 as deft

PAGE = 16
EINVAL, ECYCLE, ERANGE, EUNSUPPORTED, EWORKSPACE, ESTATE = -1, -2, -3, -5, -7, -8


def path_pages(parent, node_len, n):
    """Pages of n's path in the plan's order: ancestors from the parent up,
    then n's own, as (node, page) pairs."""
    out, a = [], parent[n]
    while a >= 0:
        out += [(a, j) for j in range(-(-node_len[a] // PAGE))]
        a = parent[a]
    return out + [(n, j) for j in range(-(-node_len[n] // PAGE))]


def check_plan(parent, node_len, prompt_node, prompt_len, hkv, group):
    plan = deft.PromptPlan(parent, node_len, prompt_node, hkv, group, prompt_len=prompt_len)
    st, items = plan.stats, plan.get("items")
    tile = 128 // group
    m_of = [node_len[n] if prompt_len is None or m < 0 else m
            for n, m in zip(prompt_node, prompt_len if prompt_len is not None else [-1] * len(prompt_node))]
    assert st["num_rows"] == sum(m_of)
    first = np.concatenate([[0], np.cumsum(m_of)]).astype(int)
    # every (row, page it sees) pair lies in exactly one item
    seen = {}
    for it in items:
        row0, ta, tb, pos0, node, pages, na, nb, sn, sp, part0, _ = (int(x) for x in it)
        assert 1 <= ta <= tile and 0 <= tb <= tile and (tb == 0 or ta == tile) and pages >= 1
        p = int(np.searchsorted(first, row0, side="right")) - 1
        assert prompt_node[p] == node and pos0 == node_len[node] - m_of[p] + row0 - first[p]
        way = path_pages(parent, node_len, node)
        at = way.index((sn, sp))
        assert max(na, nb) == -(-pages // 8)
        assert na <= nb or nb == 0
        for tiles, t0, t in ((na, 0, ta), (nb, ta, tb)):
            for i in range(t):
                row = row0 + t0 + i
                # what the kernel attends: pages of the first `tiles` KV tiles,
                # own tokens past the row's position masked
                rng = way[at:at + min(pages, tiles * 8)]
                got = [x for x in rng if x[0] != node or x[1] * PAGE <= pos0 + t0 + i]
                seen.setdefault(row, []).extend(got)
    for p, n in enumerate(prompt_node):
        way = path_pages(parent, node_len, n)
        for i in range(m_of[p]):
            pos = node_len[n] - m_of[p] + i
            want = [x for x in way if x[0] != n or x[1] * PAGE <= pos]
            assert sorted(seen.get(first[p] + i, [])) == sorted(want)
    # every unit is run once, by one CTA
    units = plan.get("cta_unit")
    off = plan.get("cta_off")
    assert off[0] == 0 and off[-1] == len(units) == st["num_units"] == len(items) * hkv
    assert (np.diff(off) >= 0).all() and sorted(units) == list(range(len(units)))
    assert st["ctas"] == min(152, len(units)) and (np.diff(off)[st["ctas"]:] == 0).all()
    # partial slots: pieces of an item side by side, none shared
    used = set()
    pieces = {}
    for it in items:
        if it[10] >= 0:
            rows = (int(it[1]) + int(it[2])) * group
            span = range(int(it[10]), int(it[10]) + rows * hkv)
            assert not used & set(span)
            used |= set(span)
            pieces.setdefault(int(it[0]), []).append(int(it[10]))
    assert len(used) == st["partial_slots"]
    for row0, tokens, part0, count in plan.get("merges"):
        rows = int(tokens) * group * hkv
        assert sorted(pieces.pop(int(row0))) == [int(part0) + j * rows for j in range(count)] and count > 1
    assert not pieces
    pairs = 0
    for p, n in enumerate(prompt_node):
        up, a = 0, parent[n]
        while a >= 0:
            up, a = up + node_len[a], parent[a]
        m = m_of[p]
        pairs += m * (up + node_len[n] - m) + m * (m + 1) // 2
    assert st["pair_tokens"] == pairs
    assert plan.workspace_bytes(hkv * group, 64) >= st["partial_slots"] * 65 * 4
    return plan


@pytest.mark.parametrize("seed", range(24))
def test_items_cover_every_row_and_page_once(seed):
    rng = random.Random(seed)
    n = rng.randint(1, 14)
    parent = [-1 if i == 0 or rng.random() < 0.2 else rng.randrange(i) for i in range(n)]
    if seed % 3 == 2:      # parents after their children too
        perm = list(range(n))
        rng.shuffle(perm)
        parent2 = [0] * n
        for i, p in enumerate(parent):
            parent2[perm[i]] = -1 if p < 0 else perm[p]
        parent = parent2
    node_len = [0 if rng.random() < 0.15 else rng.choice([1, 15, 16, 17, rng.randint(1, 300), rng.randint(1, 900)]) for _ in range(n)]
    prompt_node = [rng.randrange(n) for _ in range(rng.randint(0, 8))]
    lens = None if seed % 2 else [rng.choice([-1, 0, min(1, node_len[x]), rng.randint(0, node_len[x])]) for x in prompt_node]
    check_plan(parent, node_len, prompt_node, lens, rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 64]))


@pytest.mark.parametrize("lens,new,hkv,group", [([1], None, 1, 1), ([4096], [1], 1, 8), ([4096], [1], 8, 4), ([2047, 1], [64, 1], 2, 64),
                                                ([129], None, 1, 1), ([5000, 31], [40, 31], 2, 3)])
def test_few_rows_over_long_ranges(lens, new, hkv, group):
    plan = check_plan([-1] * len(lens), lens, list(range(len(lens))), new, hkv, group)
    if max(lens) >= 4096:
        assert plan.stats["num_split_items"] > 0      # one tile a head would leave the other SMs idle


def test_many_units_are_not_split():
    plan = deft.PromptPlan(None, [4096] * 8, list(range(8)), 8, 4)
    assert plan.stats["num_split_items"] == 0 and plan.stats["ctas"] == 152
    # the dealt lists are near one another in estimated work
    items, off, unit = plan.get("items"), plan.get("cta_off"), plan.get("cta_unit")
    load = [sum(2 + max(items[u // 8][6], items[u // 8][7]) for u in unit[off[c]:off[c + 1]]) for c in range(152)]
    assert max(load) < 1.1 * (sum(load) / 152)


def test_equal_units_are_levelled_by_the_shortest():
    """160 nearly equal units on 152 CTAs, and 512 units of eight lengths: the
    shortest ranges alone are cut, into small pieces, and level the CTAs."""
    plan = check_plan([-1] * 4, [2227, 1960, 2297, 2209], [0, 1, 2, 3], [20] * 4, 8, 64)
    items = plan.get("items")
    tiles = items[:, 6:8].max(axis=1)
    whole, cut = tiles[items[:, 10] < 0], tiles[items[:, 10] >= 0]
    assert plan.stats["num_split_items"] == 5 and len(whole) == 15 and cut.max() < whole.min()
    plan = deft.PromptPlan(None, [5120 + 1408 * i for i in range(8)], list(range(8)), 8, 4, prompt_len=[512] * 8)
    items, off, unit = plan.get("items"), plan.get("cta_off"), plan.get("cta_unit")
    load = [sum(max(items[u // 8][6], items[u // 8][7]) for u in unit[off[c]:off[c + 1]]) for c in range(152)]
    assert 0 < plan.stats["num_split_items"] <= 8 and max(load) < 1.05 * (sum(load) / 152)


def test_rebuild_equals_a_fresh_plan_and_survives_errors():
    plan = deft.PromptPlan(None, [4000], [0], 4, 2)
    plan.rebuild([-1, 0], [100, 20], [1, 0], 2, 3, prompt_len=[5, -1])
    fresh = deft.PromptPlan([-1, 0], [100, 20], [1, 0], 2, 3, prompt_len=[5, -1])
    for name in deft.PROMPT_ARRAYS:
        assert np.array_equal(plan.get(name), fresh.get(name)), name
    with pytest.raises(deft.DeftError):
        plan.rebuild([-1, 5], [100, 20], [1, 0], 2, 3)
    assert plan.stats == fresh.stats and np.array_equal(plan.get("items"), fresh.get("items"))


@pytest.mark.parametrize("kw,status", [
    (dict(parent=[-1, 2], node_len=[1, 1], prompt_node=[0]), ERANGE),
    (dict(parent=[-1, -2], node_len=[1, 1], prompt_node=[0]), ERANGE),
    (dict(parent=[1, 0], node_len=[1, 1], prompt_node=[0]), ECYCLE),
    (dict(parent=[0], node_len=[1], prompt_node=[0]), ECYCLE),
    (dict(parent=None, node_len=[-1], prompt_node=[0]), EINVAL),
    (dict(parent=None, node_len=[5], prompt_node=[1]), ERANGE),
    (dict(parent=None, node_len=[5], prompt_node=[-1]), ERANGE),
    (dict(parent=None, node_len=[5], prompt_node=[0], prompt_len=[6]), ERANGE),
    (dict(parent=None, node_len=[5], prompt_node=[0], prompt_len=[-2]), ERANGE),
    (dict(parent=None, node_len=[5], prompt_node=[0], num_kv_heads=0), EINVAL),
    (dict(parent=None, node_len=[5], prompt_node=[0], gqa_group=0), EINVAL),
    (dict(parent=None, node_len=[5], prompt_node=[0], gqa_group=65), EINVAL),
    (dict(parent=None, node_len=[2 ** 31 - 1], prompt_node=[0], prompt_len=[1]), EUNSUPPORTED),
    (dict(parent=None, node_len=[2 ** 28], prompt_node=[0], num_kv_heads=8, gqa_group=64), EUNSUPPORTED),
    (dict(parent=None, node_len=[], prompt_node=[]), EINVAL),
])
def test_refusals(kw, status):
    args = dict(num_kv_heads=2, gqa_group=2)
    args.update(kw)
    with pytest.raises(deft.DeftError) as e:
        deft.PromptPlan(**args)
    assert e.value.status == status


def test_array_lengths_that_differ():
    with pytest.raises(ValueError):
        deft.PromptPlan([-1], [1, 2], [0], 1)
    with pytest.raises(ValueError):
        deft.PromptPlan(None, [1, 2], [0], 1, prompt_len=[1, 1])


def test_null_arguments():
    lib = deft.load()
    h = ctypes.c_void_p()
    assert lib.deft_prompt_plan(None, None, 1, None, None, 0, 1, 1, ctypes.byref(h)) == EINVAL
    assert lib.deft_prompt_plan_rebuild(None, None, None, 1, None, None, 0, 1, 1) == EINVAL
    assert lib.deft_prompt_plan_upload(None, None) == EINVAL
    assert lib.deft_prompt_plan_stats_get(None, None) == EINVAL
    assert lib.deft_prompt_workspace_bytes(None, 1, 64) == 0
    plan = deft.PromptPlan(None, [5], [0], 1)
    buf = np.zeros(4, dtype=np.int32)
    assert lib.deft_prompt_plan_get(plan.handle, 9, buf.ctypes.data, buf.nbytes) == EINVAL
    assert lib.deft_prompt_plan_get(plan.handle, 1, buf.ctypes.data, 4) == EINVAL
    lib.deft_prompt_plan_free(None)


# ---- argument checks made before any CUDA call (made-up addresses: every
# call below is refused before it could use one) ----

A = 1 << 20


def attn_args(owner, **kw):
    d = dict(q=A, q_stride=8 * 64, num_rows=5, k=A, v=A, npo=A, pid=A, num_pages=4, hq=8, hkv=2, head_dim=64, page_size=16, scale=0.125,
             plan=owner.handle, out=A, out_dtype=0, lse=A, ws=A, ws_bytes=1 << 20, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(out=None), EINVAL), (dict(lse=None), EINVAL), (dict(npo=None), EINVAL),
    (dict(plan=None), EINVAL), (dict(q=A + 8), EINVAL), (dict(k=A + 2), EINVAL), (dict(out=A + 4), EINVAL), (dict(out_dtype=2), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(num_pages=0), EINVAL),
    (dict(q_stride=8 * 64 - 8), EINVAL), (dict(q_stride=8 * 64 + 4), EINVAL), (dict(num_rows=-1), EINVAL), (dict(hq=7), EINVAL),
    (dict(head_dim=96, q_stride=8 * 96), EUNSUPPORTED), (dict(page_size=32), EUNSUPPORTED), (dict(hkv=4), ESTATE), (dict(hq=4), ESTATE),
    (dict(), ESTATE),      # never uploaded
])
def test_attn_argument_checks(kw, status):
    plan = deft.PromptPlan(None, [5], [0], 2, 4)
    assert deft.load().deft_prompt_attn(*attn_args(plan, **kw)) == status


def table_args(**kw):
    d = dict(node_len=A, num_nodes=3, prev_len=None, prev_off=None, prev_id=None, num_prev=0, num_ids=0, free=A, num_free=4, page_size=16,
             npo=2 * A, pid=3 * A, max_pages=4, tok_off=4 * A, slot=5 * A, max_tokens=64, counts=6 * A, ws=None, ws_bytes=0, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(node_len=None), EINVAL), (dict(num_nodes=0), EINVAL), (dict(npo=None), EINVAL), (dict(tok_off=None), EINVAL),
    (dict(counts=None), EINVAL), (dict(pid=None), EINVAL), (dict(slot=None), EINVAL), (dict(free=None), EINVAL), (dict(num_free=-1), EINVAL),
    (dict(max_pages=-1), EINVAL), (dict(max_tokens=-1), EINVAL), (dict(num_prev=2), EINVAL), (dict(num_prev=4, prev_len=A, prev_off=A), EINVAL),
    (dict(num_prev=2, prev_len=A, prev_off=A, num_ids=2), EINVAL),
    (dict(num_prev=2, prev_len=A, prev_off=2 * A, num_ids=2, prev_id=7 * A), EINVAL),      # written while it is read
    (dict(num_prev=2, prev_len=A, prev_off=7 * A, num_ids=2, prev_id=3 * A), EINVAL),
    (dict(page_size=8), EUNSUPPORTED), (dict(num_nodes=(1 << 20) + 1), EUNSUPPORTED), (dict(num_nodes=2049), EWORKSPACE),
    (dict(num_nodes=2049, ws=A + 128, ws_bytes=1 << 20), EWORKSPACE), (dict(num_nodes=2049, ws=A, ws_bytes=64), EWORKSPACE),
])
def test_table_argument_checks(kw, status):
    assert deft.load().deft_page_table(*table_args(**kw)) == status


def test_table_workspace():
    f = deft.load().deft_page_table_workspace_bytes
    assert f(0) == 0 and f(1) == 0 and f(2048) == 0 and f(2049) > 0 and f(1 << 20) > 0


def write_args(**kw):
    d = dict(k=A, v=A, in_dtype=0, ks=128, vs=128, slot=A, num_tokens=3, kp=2 * A, vp=3 * A, num_pages=4, hkv=2, head_dim=64, page_size=16,
             stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(slot=None), EINVAL), (dict(kp=None), EINVAL), (dict(vp=2 * A), EINVAL),
    (dict(num_tokens=-1), EINVAL), (dict(num_pages=0), EINVAL), (dict(hkv=0), EINVAL), (dict(in_dtype=2), EINVAL), (dict(k=A + 8), EINVAL),
    (dict(kp=A + 8), EINVAL), (dict(ks=120), EINVAL), (dict(vs=132), EINVAL), (dict(in_dtype=1, ks=130), EINVAL),
    (dict(head_dim=32), EUNSUPPORTED), (dict(page_size=64), EUNSUPPORTED), (dict(num_pages=1 << 27), EUNSUPPORTED), (dict(num_tokens=0), 0),
])
def test_write_argument_checks(kw, status):
    assert deft.load().deft_kv_write(*write_args(**kw)) == status


def test_deep_chain():
    """A chain of nodes, each a prompt: the tokens above a node are counted
    once a node, not by a walk to the root for every prompt (60000 nodes took
    3.8 s), and pair_tokens is their closed form."""
    n = 60000
    parent, lens = np.arange(-1, n - 1), np.arange(n) % 3      # empty nodes among them
    t0 = time.process_time()
    plan = deft.PromptPlan(parent, lens, np.arange(n), 1, 1)
    spent = time.process_time() - t0
    above = np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(np.int64)
    assert plan.stats["pair_tokens"] == int((lens * above + lens * (lens + 1) // 2).sum())
    plan = deft.PromptPlan(parent, lens, [n - 1, n // 2, 0], 2, 4, prompt_len=[1, 0, -1])
    assert plan.stats["pair_tokens"] == int(above[n - 1] + lens[n - 1])
    assert spent < 1
