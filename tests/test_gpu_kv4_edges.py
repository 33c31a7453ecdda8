"""The calls around the 4-bit cache at their edges, on the GPU: empty batches,
launch shapes that only many units reach, plans that are updated and rebuilt,
rows that are not finite."""
import numpy as np
import pytest
import torch

import shared_prefix_kv_deft_gb300 as deft
from test_gpu_attn4 import Tree, check, cu, f64
from test_gpu_qkv import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from shared_prefix_kv_deft_gb300 import build as deft_build
    deft_build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_no_tokens_with_a_rotation(interleaved):
    r = Rows(T=1, hq=2, hkv=1, d=64, rot=32, interleaved=interleaved)
    kw = dict(r.kw, position=r.kw["position"][:0])
    for pools, call in ((r.pools(), deft.deft_qkv_write), (r.pools4(), deft.deft_qkv_write4)):
        before = [p.clone() for p in pools]
        assert call(r.q[:0], r.k[:0], r.v[:0], cu([]), *pools, **kw).shape == (0, 2, 64)
        assert all(torch.equal(a, b) for a, b in zip(pools, before))


@pytest.mark.parametrize("first", [(1 << 32) // (8 * 18) - 7, 1 << 27])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_far_from_the_pools_start(d, first):
    """Pages whose rows, counted from the pool's start, pass 2^32 (and 256 GB):
    a pool that begins so far before the pages which the step names, all of
    which are there.  Units of 2, 12, 20 and 40 rows."""
    import ctypes
    for queries in (2, 12, 20, 40):
        t = Tree([-1] + [0] * queries, [300] + [1 + i % 33 for i in range(queries)], list(range(1, queries + 1)), 8, 1, d, seed=queries)
        plan = t.plan()
        q, k4, v4, off, ids = t.tensors()
        want = t.run(plan)
        ids = ids + first
        bufs = deft.alloc_buffers(plan, queries, 8, d, out_dtype=deft.DEFT_OUT_F32)
        start = first * 8 * 9 * d
        rc = deft.load().deft_tree_attn4(q.data_ptr(), k4.data_ptr() - start, v4.data_ptr() - start, 1.0, 1.0, off.data_ptr(), ids.data_ptr(),
                                         first + k4.shape[0], 8, 8, d, 16, 1 / d ** 0.5, plan.handle, bufs.out.data_ptr(), deft.DEFT_OUT_F32,
                                         bufs.lse.data_ptr(), bufs.workspace.data_ptr(), ctypes.c_size_t(bufs.workspace.numel()),
                                         torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and plan.step_status() == 0
        assert torch.equal(bufs.out, want[0]) and torch.equal(bufs.lse, want[1])


@pytest.mark.parametrize("d,hq,rot", [(64, 3, 64), (64, 5, 16), (128, 32, 128), (128, 1, 48)])
def test_queries_in_place(d, hq, rot):
    """q_out on q itself, from a start in the middle of a sector on (so that
    neighbouring rows share sectors), is q_out elsewhere, bit for bit."""
    r = Rows(T=3000, hq=hq, hkv=1, d=d, rot=rot)
    want = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), *r.pools(), **r.kw)
    for call, pools in ((deft.deft_qkv_write, r.pools()), (deft.deft_qkv_write4, r.pools4())):
        q = torch.empty(r.q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(r.q.shape)
        q.copy_(r.q)
        assert q.data_ptr() % 32 == 16
        assert call(q, r.k, r.v, cu(r.slot), *pools, q_out=q, **r.kw) is q and torch.equal(q, want)


@pytest.mark.parametrize("place", [0, 20, -1])
def test_the_smoke_check_sees_one_wrong_page_of_v(monkeypatch, place):
    """Expected outputs with a page of V an eighth too small: of the prefix (16
    of more than 740 tokens), or of a branch."""
    import __graft_entry__ as entry
    entry.smoke_kv4(deft, torch)
    unpack = deft.deft_kv_unpack4

    def other(*a, **kw):
        kp, vp = unpack(*a, **kw)
        vp[place] *= 0.875
        return kp, vp

    monkeypatch.setattr(deft, "deft_kv_unpack4", other)
    with pytest.raises(RuntimeError):
        entry.smoke_kv4(deft, torch)


def traced(call):
    """What the call returns, and (kernel, bucket, items) of its launches."""
    deft.trace_enable(True)
    try:
        got = call()
        return got, [(r["kernel"], r["bucket"], r["items"]) for r in deft.trace_read()]
    finally:
        deft.trace_enable(False)


# KV heads, group, head_dim; units' rows, CTAs an SM of that width, KV heads a
# CTA takes at most.
WIDTHS = [(8, 4, 128, 8, 4, 4), (8, 4, 64, 8, 4, 4), (32, 1, 128, 8, 4, 4), (6, 3, 64, 8, 4, 2), (8, 12, 128, 16, 3, 4), (4, 15, 64, 16, 3, 4),
          (6, 9, 128, 16, 3, 2), (8, 16, 64, 64, 2, 2), (8, 40, 64, 64, 2, 2), (5, 33, 64, 64, 2, 1)]


@pytest.mark.parametrize("beside,pieces", [("one less", 1), ("whole", 1), ("one more", 1), ("a quarter more", 1), ("a quarter more", 2), ("half more", 2),
                                           ("twice", 1)])
@pytest.mark.parametrize("width", WIDTHS)
def test_rounds_of_ctas(width, beside, pieces):
    """So many requests that CTAs which take several KV heads of an item fill
    the device (a unit a warp, no joining of warps), exactly, with one CTA
    less, with some more in a second launch, whose CTAs take fewer heads, and
    twice over; each request one unit a head, or two and a merge
    (as after all units of the tensor-core list)."""
    hkv, group, d, rows, per_sm, most = width
    slots = per_sm * torch.cuda.get_device_properties(0).multi_processor_count
    groups = hkv // most
    one, two = (-(-x * slots // groups) for x in (1, 2))    # items that fill one round, and two
    items = {"one less": one - 1, "whole": one, "one more": one + 1, "a quarter more": one + one // 4, "half more": one + one // 2, "twice": two}[beside]
    n = round(items / pieces)
    unit = max(64, 16 * group)      # (a chunk is at least 16 tokens a row long)
    length = [unit * (pieces - 1) + unit // 2 + 1 + (7 * i) % (unit // 2) for i in range(n)]
    t = Tree([-1] * n, length, list(range(n)), hkv, group, d, seed=n)
    plan = t.plan(unit)
    total = n * pieces
    assert plan.stats["num_fma_items"] + plan.stats["num_mma_items"] == total
    got, launches = traced(lambda: t.run(plan))
    bulk = total * groups // slots * slots // groups
    want = [("phase1_kv4", rows, x) for x in (bulk, total - bulk) if x] + ([("phase2_merge", 0, n)] if pieces > 1 or rows == 64 else [])
    assert launches == want
    if pieces == 1:
        assert (bulk > 0) == (beside != "one less") and (total > bulk or beside in ("whole", "twice"))
    check(t, got)


@pytest.mark.parametrize("hkv,group,d", [(8, 1, 128), (8, 3, 64), (4, 2, 128)])
def test_many_widths_at_once(hkv, group, d):
    """Prefixes under 3 to 40 branches each: one, two and more rows a unit in
    one list, wide units beside them, every launch of a width and its rest."""
    parent, length, query = [], [], []
    for i in range(60):
        root = len(parent)
        parent.append(-1)
        length.append(300 + 37 * (i % 11))
        for j in range([3, 6, 8, 5, 20, 40][i % 6]):
            query.append(len(parent))
            parent.append(root)
            length.append(1 + (13 * i + 29 * j) % 100)
    t = Tree(parent, length, query, hkv, group, d, seed=hkv)
    plan = t.plan(128)
    got, launches = traced(lambda: t.run(plan))
    kinds = [b for k, b, _ in launches if k == "phase1_kv4"]
    assert kinds.count(8) == 2 and max(kinds) == 64 and launches[-1][0] == "phase2_merge"
    check(t, got)


@pytest.mark.parametrize("chunk", [2048, 64])
@pytest.mark.parametrize("shape", [(1, 4, 64), (1, 4, 128), (1, 12, 64), (1, 12, 128), (9, 2, 64), (20, 2, 128)])
def test_rows_that_are_not_finite_have_a_lse_of_nan(shape, chunk):
    """Never an infinity, which would say that a row attended nothing: rows
    of one partial, written by their unit, and of several, by the merge; at
    every width.  Queries with a NaN or an infinity of their own, then a NaN
    key.  The other rows are as near to 64 bits as ever (check's bounds), not
    the same bits: a unit's rows raise their maxima together, and a row that is
    not finite calls for none.  A weight is 2^11 times a power of two times
    itself when it is rounded, 2^15 at most, whichever time that was: the bounds
    hold for each."""
    queries, group, d = shape
    if queries == 1:
        t = Tree([-1], [200], [0], 2, group, d)
    else:
        t = Tree([-1] + [0] * queries, [200] + [9] * queries, list(range(1, queries + 1)), 2, group, d)
    plan = t.plan(chunk)
    base = t.run(plan)
    q = t.q.copy()

    def others(out, lse):
        t.q = q
        check(t, (torch.where(lse.isnan()[..., None], base[0], out), torch.where(lse.isnan(), base[1], lse)))

    hit = np.zeros(base[1].shape, bool)
    for i, (value, row) in enumerate([(np.nan, 0), (np.inf, 2), (-np.inf, group), (np.nan, 2 * group - 1)]):
        t.q[i % queries, row, 5 * i] = value
        hit[i % queries, row] = True
    got = t.run(plan)
    assert (np.isnan(f64(got[1])) == hit).all() and np.isnan(f64(got[0])[hit]).all()
    others(*got)
    s = t.slots(0)[77]          # a key of KV head 1 that all queries attend
    scale = t.k4[..., 8 * d:].reshape(-1, 2, 16, d // 16)[s // 16, 1, s % 16, 1:2]
    was = scale.copy()
    scale[:] = 0x7F
    got = t.run(plan)
    hit[:], hit[:, group:] = False, True
    assert (np.isnan(f64(got[1])) == hit).all() and np.isnan(f64(got[0])[hit]).all()
    scale[:] = was
    others(*got)


@pytest.mark.parametrize("hkv,group,d", [(2, 2, 128), (2, 3, 64), (8, 1, 128)])
def test_plans_that_are_updated_and_rebuilt(hkv, group, d):
    """One plan through Plan.update (tokens appended, a branch pruned) and
    Plan.rebuild (other trees, larger and smaller), uploaded and used again
    each time."""
    rng = np.random.default_rng(d + group)
    parent, length = [-1] + [0] * 20, [500] + [int(x) for x in rng.integers(1, 60, 20)]
    t = Tree(parent, length, list(range(1, 21)), hkv, group, d, seed=1)
    plan = t.plan(128)
    steps = [(t, t.run(plan))]
    for step in range(4):
        length = [length[0]] + [n + int(rng.integers(0, 20)) for n in length[1:]]
        if step == 2:
            length[5] = 0
        t = Tree(parent, length, list(range(1, 21)), hkv, group, d, seed=step + 2)
        plan.update(length)
        plan.upload()
        steps.append((t, t.run(plan)))
    for n, m in ((3, 1200), (40, 90), (1, 5), (17, 400)):
        parent, length = [-1] + [0] * n, [m] + [1 + 7 * i % 50 for i in range(n)]
        t = Tree(parent, length, list(range(1, n + 1)), hkv, group, d, seed=m)
        plan.rebuild(parent, length, list(range(1, n + 1)), 128, group, naive=False)
        plan.upload()
        steps.append((t, t.run(plan)))
    for t, got in steps:
        check(t, got)
