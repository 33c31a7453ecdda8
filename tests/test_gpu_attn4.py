"""deft_tree_attn4 against softmax attention in 64 bits over what the 4-bit
cache's bytes stand for."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref
import shared_prefix_kv_deft_gb300 as deft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from shared_prefix_kv_deft_gb300 import build as deft_build
    deft_build.build()
    torch.cuda.set_device(0)


def cu(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dt))).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


class Tree:
    """A tree, its pages in random order, and a cache of random bytes: those
    of tokens have scales of 0.25 to 2, all others (places past a node's last
    token, pages no node has) hold anything, NaN scales among them."""

    def __init__(self, parent, length, query, hkv, group, d, pos=None, seed=0, kg=1.0, vg=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.parent, self.length, self.query, self.pos = parent, length, query, pos
        self.hkv, self.group, self.d, self.g = hkv, group, d, (kg, vg)
        counts = [-(-n // 16) for n in length]
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        pool = int(self.off[-1]) + spare
        self.ids = rng.permutation(pool)[:int(self.off[-1])].astype(np.int32)
        self.k4, self.v4 = (rng.integers(0, 256, (pool, hkv, 9 * d), dtype=np.uint8) for _ in "kv")
        slots = np.concatenate([self.slots(n) for n in range(len(length))]) if len(length) else np.zeros(0, int)
        for p in (self.k4, self.v4):
            s = p[..., 8 * d:].reshape(pool, hkv, 16, d // 16)
            s[slots // 16, :, slots % 16] = rng.integers(0x28, 0x41, (len(slots), hkv, d // 16))
        self.q = (rng.standard_normal((len(query), hkv * group, d)) / 4).astype(np.float32)
        self.q = f64(torch.from_numpy(self.q).bfloat16())

    def slots(self, n):
        j = np.arange(self.length[n])
        return self.ids[self.off[n] + j // 16] * 16 + j % 16

    def path(self, i):
        n, seen = self.query[i], []
        while n >= 0:
            seen.append(self.slots(n))
            if n == self.query[i] and self.pos is not None and self.pos[i] >= 0:
                seen[0] = seen[0][:self.pos[i] + 1]
            n = self.parent[n]
        return np.concatenate(seen[::-1])

    def expect(self, scale=None):
        """out, lse, and what each may be off by for a given way of summing:
        the weighted |v| and the largest sum of |q k|."""
        K, V = (ref.values(*ref.pages(p), g) for p, g in zip((self.k4, self.v4), self.g))
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        Q, Hq = len(self.query), self.hkv * self.group
        out, lse, wabs, big = np.zeros((Q, Hq, self.d)), np.full((Q, Hq), -np.inf), np.zeros((Q, Hq, self.d)), np.zeros((Q, Hq))
        n = np.zeros((Q, 1))
        for i in range(Q):
            s = self.path(i)
            if not len(s):
                continue
            n[i] = len(s)
            k, v = K[s // 16, :, s % 16], V[s // 16, :, s % 16]      # [tokens, heads, d]
            q = self.q[i].reshape(self.hkv, self.group, self.d)
            with np.errstate(invalid="ignore"):
                z = np.einsum("hgd,thd->hgt", q, k) * scale
                top = z.max(-1, keepdims=True)
                p = np.exp(z - top)
                total = p.sum(-1, keepdims=True)
                out[i] = (np.einsum("hgt,thd->hgd", p, v) / total).reshape(Hq, -1)
                wabs[i] = (np.einsum("hgt,thd->hgd", p, np.abs(v)) / total).reshape(Hq, -1)
                lse[i] = (top + np.log(total))[..., 0].reshape(-1)
                big[i] = (np.einsum("hgd,thd->hgt", np.abs(q), np.abs(k)) * scale).max(-1).reshape(-1)
        return out, lse, wabs, big, n

    def plan(self, chunk=256, pack=False):
        p = deft.Plan(self.parent, self.length, self.query, chunk, self.group, query_pos=self.pos, naive=False, tensor_pack=pack)
        p.upload()
        return p

    def tensors(self):
        return [torch.from_numpy(self.q.astype(np.float32)).bfloat16().cuda(), torch.from_numpy(self.k4).cuda(), torch.from_numpy(self.v4).cuda(), cu(self.off),
                cu(self.ids)]

    def run(self, plan, f32=True, **kw):
        out = deft.deft_tree_attn4(*self.tensors(), plan, out_dtype=deft.DEFT_OUT_F32 if f32 else deft.DEFT_OUT_BF16, k_scale=self.g[0], v_scale=self.g[1], **kw)
        assert plan.step_status() == 0
        return out


def check(t, got, f32=True, scale=None, rows=None):
    """fp32 sums of exact products: a logit is off by at most (d + 8) 2^-24 of
    its sum of |q k|, a weight by that, by 2^-11 for its rounding to fp16 and
    2^-21 for the exponentials (the rescaled ones included), a sum of n terms
    by n 2^-24; then the output's own rounding.  A weight below 2^-25 of the
    row's largest is an fp16 number without all of its bits: 2^11 times the
    weight is off by half of the smallest step, 2^-25, the weight by 2^-36,
    which shows where the largest weights meet values of 0."""
    out, lse, wabs, big, n = t.expect(scale)
    o, z = f64(got[0]), f64(got[1])
    assert o.shape == out.shape and z.shape == lse.shape
    logit = (t.d + 8) * 2.0 ** -24 * big
    if rows is None:
        rows = slice(None)
    w = 2 * logit + 2.0 ** -11 + 2.0 ** -21 + n * 2.0 ** -24
    vmax = max(6 * ref.E4M3[0x40], 6) * t.g[1]
    tol = w[..., None] * 2 * wabs + (n * 2.0 ** -36 * vmax)[..., None] + (0 if f32 else 2.0 ** -8) * np.abs(out) * (1 + 1e-2) + 1e-30
    err = np.abs(o - out)
    assert (err <= tol)[rows].all(), (np.nanmax((err / np.maximum(tol, 1e-30))[rows]))
    fin = np.isfinite(lse)
    assert np.array_equal(np.isfinite(z)[rows], fin[rows])
    lt = logit + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(fin, lse, 0))
    assert (np.abs(np.where(fin, z - np.where(fin, lse, 0), 0)) <= lt)[rows].all()
    assert (z[~fin] == -np.inf).all()


def forest(seed, nodes, longest, queries, positions=False):
    """A random forest with empty nodes; queries anywhere."""
    rng = np.random.default_rng(seed)
    parent = [-1] + [int(rng.integers(-1, i)) if rng.random() < 0.9 else -1 for i in range(1, nodes)]
    length = [int(x) for x in rng.choice([0, 1, 2, 15, 16, 17, 31, 32, 33, longest // 2, longest], nodes)]
    query = [int(x) for x in rng.integers(0, nodes, queries)]
    pos = [int(rng.integers(-1, length[n])) if length[n] else -1 for n in query] if positions else None
    return dict(parent=parent, length=length, query=query, pos=pos)


SHAPES = [(1, 1, 64), (2, 4, 128), (4, 1, 128), (3, 3, 64), (1, 7, 128), (2, 8, 64), (1, 12, 64), (1, 16, 128), (1, 33, 64), (2, 64, 128), (8, 4, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_forests(shape, seed):
    hkv, group, d = shape
    nodes, longest, queries = [(1, 40, 1), (5, 100, 7), (9, 300, 20), (30, 64, 70)][seed]
    t = Tree(**forest(seed, nodes, longest, queries, positions=seed % 2 == 1), hkv=hkv, group=group, d=d, seed=seed, kg=[1, 0.5, 0.37, 2][seed],
             vg=[1, 1, 1.9, 0.1][seed])
    for chunk, pack in ((256, False), (33, False), (1024, True)):
        check(t, t.run(t.plan(chunk, pack)))
    check(t, t.run(t.plan(64), f32=False), f32=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 31, 63, 64, 65, 128, 255, 513])
def test_one_node_of_any_length(d, n):
    t = Tree([-1], [n], [0], 2, 2, d, seed=n)
    check(t, t.run(t.plan()))


@pytest.mark.parametrize("queries,group", [(3, 5), (4, 4), (9, 1), (16, 1), (17, 1), (31, 1), (32, 2), (33, 1), (40, 2), (64, 1), (100, 1), (5, 13)])
def test_shared_prefix(queries, group):
    """Every row count of an item: a prefix under all the branches."""
    for d in (64, 128):
        t = Tree([-1] + [0] * queries, [700] + [5 + 3 * (i % 9) for i in range(queries)], list(range(1, queries + 1)), 2, group, d, seed=queries)
        check(t, t.run(t.plan(256)))


def test_speculative_tree():
    """Many one-token nodes in one chunk, every node a query."""
    rng = np.random.default_rng(3)
    parent, length = [-1, -1], [300, 77]
    for _ in range(150):
        parent.append(int(rng.integers(0, len(parent))))
        length.append(1)
    for d, pack in ((64, False), (128, True)):
        t = Tree(parent, length, list(range(2, 152)), 2, 2, d, seed=1)
        check(t, t.run(t.plan(256, pack)))


def test_chunk_of_256_segments():
    t = Tree([-1] + [0] * 300, [3] + [1] * 300, list(range(1, 301)), 1, 1, 128)
    check(t, t.run(t.plan(1024)))


def test_deep_chain():
    n = 400
    t = Tree([-1] + list(range(n - 1)), [i % 3 for i in range(n)], [n - 1, n // 2, 0], 2, 3, 64)
    check(t, t.run(t.plan(256)))


def test_empty_paths():
    """out = 0 and lse = -inf, alone and beside others; no query at all."""
    t = Tree([-1, 0, -1], [0, 0, 20], [0, 1, 2], 2, 2, 64)
    got = t.run(t.plan())
    check(t, got)
    assert (f64(got[0])[:2] == 0).all()
    t = Tree([-1], [0], [0, 0], 2, 2, 128)
    got = t.run(t.plan())
    assert (f64(got[0]) == 0).all() and (f64(got[1]) == -np.inf).all()
    t = Tree([-1], [5], [], 2, 2, 128)
    assert t.run(t.plan())[0].shape == (0, 4, 128)


@pytest.mark.parametrize("d", [64, 128])
def test_growing_logits_and_one_that_leads_all(d):
    """The running maximum raised over and over, and weights far below it."""
    t = Tree([-1, 0], [900, 40], [1] * 9, 1, 1, d, seed=5)
    codes, scales = t.k4[..., :8 * d], t.k4[..., 8 * d:]
    for j in range(900):
        s = t.slots(0)[j]
        scales.reshape(-1, 1, 16, d // 16)[s // 16, :, s % 16] = 0x10 + j // 16      # 2^-5.. to 2^2 and more
    check(t, t.run(t.plan(256)))
    check(t, t.run(t.plan(1024)))
    t = Tree([-1], [3000], [0], 1, 1, d, seed=6)
    t.q[:] = 0.25
    x = t.k4[..., :8 * d].reshape(-1, 1, 16, d // 2)
    sc = t.k4[..., 8 * d:].reshape(-1, 1, 16, d // 16)
    s = t.slots(0)
    x[s // 16, :, s % 16] = 0x99        # all -0.5 ...
    sc[s // 16, :, s % 16] = 0x38       # ... times 1
    x[s[5] // 16, :, s[5] % 16] = 0x55  # one token of 3
    sc[s[5] // 16, :, s[5] % 16] = 0x3C if d == 64 else 0x38
    check(t, t.run(t.plan(8192)), scale=None)


@pytest.mark.parametrize("queries", [4, 12, 20, 50])
@pytest.mark.parametrize("rising", [True, False])
def test_logits_that_rise_or_fall_over_a_chunk(queries, rising):
    """Every width: the maxima raised tile after tile (by 2^4 and more each),
    or once and then far above everything; branches that see half of it."""
    n = 1500
    t = Tree([-1] + [0] * queries, [n] + [1 + i % 40 for i in range(queries)], list(range(1, queries + 1)), 1, 1, 128, seed=queries)
    t.q[:] = np.abs(t.q) + 0.25
    t.q = f64(torch.from_numpy(t.q.astype(np.float32)).bfloat16())
    s = t.slots(0)
    codes, scales = t.k4[..., :8 * 128].reshape(-1, 1, 16, 64), t.k4[..., 8 * 128:].reshape(-1, 1, 16, 8)
    codes[s // 16, :, s % 16] &= 0x77           # keys of no negative element: logits follow the scales
    at = np.arange(n) if rising else np.arange(n)[::-1]
    scales[s // 16, :, s % 16] = (0x20 + at * 40 // n)[:, None, None]    # 2^-3 to 2^2
    for chunk in (256, 2048):
        check(t, t.run(t.plan(chunk)))


@pytest.mark.parametrize("scale", [1e-30, 1.0, 40.0])
def test_scales(scale):
    t = Tree([-1, 0, 0], [100, 9, 30], [1, 2, 0], 2, 3, 128)
    check(t, t.run(t.plan(), scale=scale), scale=scale)


@pytest.mark.parametrize("power", [-120, -60, -30, 30, 60])
def test_queries_of_any_magnitude(power):
    """A row's power of two is taken out before fp16 sees it: the same weights
    for q times 2^power and the scale times 2^-power."""
    t = Tree([-1, 0, 0], [200, 9, 30], [1, 2, 0, 1, 1, 1, 2, 2, 2], 2, 2, 128)
    if power < -80:     # (bf16's smallest number is 2^-133: elements that it holds times 2^power with all their bits)
        t.q = np.copysign(np.maximum(np.abs(t.q), 2.0 ** -6), t.q)
    else:
        t.q[1, :, :100] *= 2.0 ** -20       # a row of very uneven elements
    t.q[..., 3] = 0
    want = t.run(t.plan(), scale=0.25)
    t.q *= 2.0 ** power
    got = t.run(t.plan(), scale=0.25 * 2.0 ** -power)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    t.q *= 2.0 ** -power
    check(t, want, scale=0.25)


@pytest.mark.parametrize("queries", [3, 20, 50])
def test_rows_of_very_different_magnitudes(queries):
    """Rows of one item from 2^-40 to 2^20 of one another, one of zeros; and
    rows near one another, all tiny."""
    t = Tree([-1] + [0] * queries, [700] + [3 + i % 20 for i in range(queries)], list(range(1, queries + 1)), 2, 2, 128, seed=queries)
    q = t.q.copy()
    e = np.random.default_rng(1).integers(-40, 4, (queries, 4, 1))
    t.q = f64(torch.from_numpy((q * 2.0 ** e).astype(np.float32)).bfloat16())
    t.q[1, 2] = 0
    check(t, t.run(t.plan()))
    t.q = q * 2.0 ** -90
    check(t, t.run(t.plan(), scale=2.0 ** 86), scale=2.0 ** 86)


@pytest.mark.parametrize("d", [64, 128])
def test_pools_that_start_at_any_16_bytes(d):
    t = Tree([-1] + [0] * 20, [500] + [40] * 20, list(range(1, 21)), 2, 1, d)
    plan = t.plan()
    q, k4, v4, off, ids = t.tensors()
    want = deft.deft_tree_attn4(q, k4, v4, off, ids, plan)
    for by in (16, 48):
        moved = []
        for p in (k4, v4):
            flat = torch.empty(p.numel() + 64, dtype=torch.uint8, device="cuda")
            at = flat[by:by + p.numel()].view(p.shape)
            at.copy_(p)
            assert at.data_ptr() % 32 == 16
            moved.append(at)
        got = deft.deft_tree_attn4(q, *moved, off, ids, plan)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_that_are_not_finite():
    """An infinite or NaN query element, a NaN key: NaN in the rows that reach
    it, all others as without it."""
    t = Tree([-1, 0, 0], [300, 9, 30], [1, 2, 0, 1], 2, 4, 128)
    plan = t.plan(64)
    base = t.run(plan)
    q = t.q.copy()
    t.q[0, 1, 7], t.q[3, 6, 100], t.q[2, 0, 0] = np.nan, np.inf, -np.inf
    out, lse = (f64(x) for x in t.run(plan))
    hit = np.zeros((4, 8), bool)
    hit[0, 1] = hit[3, 6] = hit[2, 0] = True
    assert np.isnan(out[hit]).any(-1).all() and not np.isfinite(lse[hit]).any()
    assert (out[~hit] == f64(base[0])[~hit]).all() and (lse[~hit] == f64(base[1])[~hit]).all()
    t.q = q
    s = t.slots(1)[3]       # a key of node 1, of KV head 1: queries 0 and 3
    t.k4[..., 8 * 128:].reshape(-1, 2, 16, 8)[s // 16, 1, s % 16, 2] = 0x7F
    out, lse = (f64(x) for x in t.run(plan))
    hit = np.zeros((4, 8), bool)
    hit[[0, 3], 4:] = True
    assert np.isnan(out[hit]).all() and not np.isfinite(lse[hit]).any()
    assert (out[~hit] == f64(base[0])[~hit]).all()


def test_rows_that_are_not_finite_among_many():
    """The same where the prefix is one item of 40 rows."""
    t = Tree([-1] + [0] * 20, [600] + [17] * 20, list(range(1, 21)), 2, 2, 128)
    plan = t.plan()
    base = [f64(x) for x in t.run(plan)]
    t.q[4, 0, 9], t.q[11, 3, 100], t.q[19, 1, 0] = np.inf, np.nan, -np.inf
    out, lse = (f64(x) for x in t.run(plan))
    hit = np.zeros((20, 4), bool)
    hit[4, 0] = hit[11, 3] = hit[19, 1] = True
    assert np.isnan(out[hit]).any(-1).all() and np.isnan(lse[hit]).all()
    assert (out[~hit] == base[0][~hit]).all() and (lse[~hit] == base[1][~hit]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [1, 12, 40])
def test_logits_at_the_end_of_fp32(queries, d):
    """Rows of 2^100 and more: over keys of 0 every logit is 0, whatever the
    factor; a logit above fp32's largest is NaN in its row alone; logits of
    infinite rows the same, whatever rows are beside them."""
    t = Tree([-1] + [0] * queries, [600] + [3] * queries, list(range(1, queries + 1)), 2, 1, d, seed=queries)
    plan, g = t.plan(), 2.0 ** 60
    t.g = (g, 1.0)
    t.k4[..., :8 * d] = 0
    t.q[:] = 0
    t.q[..., 5] = 2.0 ** 120
    check(t, t.run(plan, scale=1.0), scale=1.0)
    t.g = (1.0, 1.0)
    t.k4[..., :8 * d] = 0x22                # all 1 ...
    x = t.k4[..., 8 * d:].reshape(-1, 2, 16, d // 16)
    s = np.concatenate([t.slots(n) for n in range(queries + 1)])
    x[s // 16, :, s % 16] = 0x38            # ... times 1
    t.q[:] = 2.0 ** -9
    base = [f64(v) for v in t.run(plan, scale=1.0)]
    check(t, t.run(plan, scale=1.0), scale=1.0)
    for value, at in ((2.0 ** 125, slice(None)), (np.inf, slice(3, 4)), (-np.inf, slice(3, 4)), (-np.inf, slice(None))):
        t.q[:] = 2.0 ** -9
        t.q[queries // 2, 1, at] = value    # (d 2^125: past fp32)
        out, lse = (f64(v) for v in t.run(plan, scale=1.0))
        hit = np.zeros((queries, 2), bool)
        hit[queries // 2, 1] = True
        assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
        assert (out[~hit] == base[0][~hit]).all() and (lse[~hit] == base[1][~hit]).all()


def test_long_path():
    """Offsets past 2^31 bytes and a path of 200000 tokens."""
    d, hkv = 128, 8
    t = Tree([-1, 0], [200000, 3], [1], 1, 2, d, seed=9)
    check(t, t.run(t.plan(8192)))
    pages = (1 << 32) // (hkv * 9 * d) + 10      # past 4 GB
    k4, v4 = (torch.zeros((pages, hkv, 9 * d), dtype=torch.uint8, device="cuda") for _ in "kv")
    t = Tree([-1], [100], [0], hkv, 2, d, seed=10, spare=0)
    ids = np.array([pages - 1, 3, pages // 2, pages - 7, 0, pages - 2, 11])
    for pool, rows in ((k4, t.k4), (v4, t.v4)):
        for page, i in zip(ids, t.ids):
            pool[int(page)] = torch.from_numpy(rows[i]).cuda()
    q, _, _, off, _ = t.tensors()
    got = deft.deft_tree_attn4(q, k4, v4, off, cu(ids), t.plan(32), out_dtype=deft.DEFT_OUT_F32)
    check(t, got)


def test_repeatable_and_two_at_once():
    """Bit for bit the same again, and two steps of one plan on two streams,
    each with buffers of its own; a step captured and replayed."""
    t = Tree([-1] + [0] * 20, [3000] + [100] * 20, list(range(1, 21)), 4, 2, 128)
    plan, args = t.plan(), t.tensors()
    want = deft.deft_tree_attn4(*args, plan)
    for _ in range(3):
        got = deft.deft_tree_attn4(*args, plan)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [deft.deft_tree_attn4(*args, plan, stream=s) for s in streams for _ in range(3)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    bufs = deft.alloc_buffers(plan, 20, 8, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        deft.deft_tree_attn4(*args, plan, bufs)
    for _ in range(2):
        for x in (bufs.out, bufs.lse, bufs.workspace):
            x.fill_(0x55)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.out, want[0]) and torch.equal(bufs.lse, want[1])


def test_refusals():
    t = Tree([-1], [20], [0, 0], 2, 2, 64)
    plan = t.plan()
    q, k4, v4, off, ids = t.tensors()
    bufs = deft.alloc_buffers(plan, 2, 4, 64)
    for call in (lambda: deft.deft_tree_attn4(q.float(), k4, v4, off, ids, plan), lambda: deft.deft_tree_attn4(q[:1], k4, v4, off, ids, plan),
                 lambda: deft.deft_tree_attn4(q, k4[..., :-9], v4[..., :-9], off, ids, plan), lambda: deft.deft_tree_attn4(q, k4.float(), v4, off, ids, plan),
                 lambda: deft.deft_tree_attn4(q, k4, v4, off.long(), ids, plan), lambda: deft.deft_tree_attn4(q, k4, v4, off[:0], ids, plan),
                 lambda: deft.deft_tree_attn4(q, k4, v4, off, ids.cpu(), plan),
                 lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, deft.StepBuffers(bufs.out[:1], bufs.lse, bufs.workspace)),
                 lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, deft.StepBuffers(bufs.out, bufs.lse.double(), bufs.workspace))):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, k_scale=0.0), -1),
                         (lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, v_scale=math.nan), -1),
                         (lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, scale=-1.0), -1),
                         (lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, plan, deft.StepBuffers(bufs.out, bufs.lse, bufs.workspace[:256])), -7),
                         (lambda: deft.deft_tree_attn4(q, k4, v4, off, ids, deft.Plan([-1], [20], [0, 0], 256, 2)), -8),
                         (lambda: deft.deft_tree_attn4(q.repeat(1, 2, 1), k4, v4, off, ids, plan), -8)):
        with pytest.raises(deft.DeftError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("d,group,rot", [(128, 4, 128), (64, 3, 32)])
def test_a_decode_loop(d, group, rot):
    """Requests grow by a token a step: page tables, appended rows in 4 bits,
    the step, against 64 bits from the projections on; the same cache through
    deft_kv_unpack4 by the bf16 step and by the prompts' attention."""
    rng = np.random.default_rng(d)
    hkv, B, steps = 2, 5, 20
    length = [0, 1, 15, 16, 300]
    pool = 64
    k4, v4 = deft.alloc_kv4_pages(pool, hkv, d)
    k4.fill_(0xFF)
    v4.fill_(0x7F)
    a = rng.uniform(-9, 9, (512, rot // 2))
    cos_sin = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    wt = torch.from_numpy(w).bfloat16().cuda()
    free = cu(rng.permutation(pool))
    table, prev, used = None, None, 0
    K, V = [np.zeros((0, hkv, d)) for _ in range(B)], [np.zeros((0, hkv, d)) for _ in range(B)]
    now = [n for n in length]
    first = True
    for step in range(steps):
        lens = [n + 1 for n in now] if not first else [max(1, n) for n in now]
        new = [b - (0 if first else c) for b, c in zip(lens, now)]
        table = deft.deft_page_table(cu(lens), free[used:], prev=prev, max_pages=pool, max_tokens=sum(new) + 3)
        used += int(table.counts[1])
        assert int(table.counts[3]) == 0
        T = sum(new)
        slot = table.slot[:T]
        pos = np.concatenate([np.arange(b - x, b) for b, x in zip(lens, new)])
        x = torch.from_numpy(rng.standard_normal((T, (group + 2) * hkv, d)).astype(np.float32)).bfloat16().cuda()
        q, k, v = x[:, :group * hkv], x[:, group * hkv:(group + 1) * hkv], x[:, (group + 1) * hkv:]
        kw = dict(position=cu(pos), cos_sin=cu(cos_sin, np.float32), q_norm=wt, k_norm=wt, eps=1e-6, k_scale=1.0, v_scale=0.5)
        qo = deft.deft_qkv_write4(q, k, v, slot, k4, v4, **kw)
        last = np.cumsum(new) - 1
        tok = 0
        for b in range(B):
            for arr, src, g, turn in ((K, k, 1.0, True), (V, v, 0.5, False)):
                y = f64(src)[tok:tok + new[b]]
                if turn:
                    y = ref.turned(y, f64(wt), 1e-6, cos_sin, pos[tok:tok + new[b]], False)
                c, s, _ = ref.quantise(ref.bf16(y), g)
                arr[b] = np.concatenate([arr[b], ref.values(c, s, g)])
            tok += new[b]
        now, first = lens, False
        prev = (cu(lens), table.page_off, table.page_id)
        if step in (0, 7, steps - 1):
            plan = deft.Plan([-1] * B, lens, list(range(B)), 64, group, naive=False)
            plan.upload()
            rows = qo[cu(last, np.int64)].contiguous()
            out, lse = deft.deft_tree_attn4(rows, k4, v4, table.page_off, table.page_id, plan, out_dtype=deft.DEFT_OUT_F32, k_scale=1.0, v_scale=0.5)
            q64 = f64(rows)
            for b in range(B):
                z = np.einsum("hgd,thd->hgt", q64[b].reshape(hkv, group, d), K[b]) / math.sqrt(d)
                p = np.exp(z - z.max(-1, keepdims=True))
                want = (np.einsum("hgt,thd->hgd", p, V[b]) / p.sum(-1, keepdims=True)).reshape(-1, d)
                # a key that 32-bit arithmetic puts on the other side of a
                # border differs by a code, at most 2 s of |k| up to 6 s
                assert np.abs(f64(out[b]) - want).max() < 2e-2
            n = int(table.counts[0])
            kp, vp = deft.deft_kv_unpack4(k4, v4, table.page_id[:n], k_scale=1.0, v_scale=0.5)
            ids = torch.arange(n, dtype=torch.int32, device="cuda")
            full = deft.Plan([-1] * B, lens, list(range(B)), 64, group)
            full.upload()
            o2, l2 = deft.deft_tree_attn(rows, kp, vp, table.page_off, ids, full, out_dtype=deft.DEFT_OUT_F32)
            pp = deft.PromptPlan(None, lens, list(range(B)), hkv, group, prompt_len=[1] * B)
            pp.upload()
            o3, l3 = deft.deft_prompt_attn(rows, kp, vp, table.page_off, ids, pp, out_dtype=deft.DEFT_OUT_F32)
            # weights rounded to bf16 there (2^-8 of a weighted |v| of at most 6 * 0.5 * 2)
            for o, z in ((o2, l2), (o3, l3)):
                assert (out - o).abs().max() < 2.0 ** -7 * 3 and (lse - z).abs().max() < 1e-4
