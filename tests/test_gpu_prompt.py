"""GPU parity of the prompt path: deft_page_table, deft_kv_write and
deft_prompt_attn against plain numpy / torch forms in 64 bits, and a run of
them together with the tree step.

Tolerances.  A bf16 rounding is off by at most 2^-8 of the value.  The
attention kernel rounds each probability p_j to bf16 before the product with
V, so its output is off by at most 2^-8 sum p_j |v_j| / sum p_j (`mean_abs`
below, from the reference), and a bf16 output by another 2^-8 |out|.  Logits
are fp32 sums of d exact products: off by at most d 2^-24 scale sum |q||k|;
the sum of n probabilities in fp32 by n 2^-24 of itself, ex2 by 2^-22.
"""
from __future__ import annotations

import ctypes
import math
import random

import numpy as np
import pytest
import torch

import shared_prefix_kv_deft_gb300 as deft
import workloads as W

pytestmark = pytest.mark.gpu
PAGE = 16
NAN = float("nan")


# ---------------------------------------------------------------------------
# Reference
# ---------------------------------------------------------------------------

class Case:
    """A tree whose nodes' K and V are kept per token (CPU, bf16) and
    scattered into pages; slots that hold no token are NaN."""

    def __init__(self, parent, node_len, prompt_node, prompt_len, hkv, group, d, seed=0, shuffle=True, q_pad=0, k_scale=1.0, fused=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.parent, self.node_len, self.prompt_node = list(parent), list(node_len), list(prompt_node)
        self.new = [node_len[n] if prompt_len is None or prompt_len[i] < 0 else prompt_len[i] for i, n in enumerate(prompt_node)]
        self.prompt_len, self.hkv, self.group, self.d = prompt_len, hkv, group, d
        rows, hq = sum(self.new), hkv * group
        self.k = [(torch.randn((n, hkv, d), generator=g) * k_scale).bfloat16() for n in node_len]
        self.v = [torch.randn((n, hkv, d), generator=g).bfloat16() for n in node_len]
        q = torch.randn((rows + q_pad, hq + 3 if fused else hq, d), generator=g).bfloat16()
        self.q = q[:, 2:2 + hq] if fused else q
        counts = [-(-n // PAGE) for n in node_len]
        total = sum(counts)
        self.num_pages = total + 5
        ids = rng.permutation(self.num_pages)[:total] if shuffle else np.arange(total)
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.ids = ids.astype(np.int32)
        kp = torch.full((self.num_pages, hkv, PAGE, d), NAN, dtype=torch.bfloat16)
        vp = kp.clone()
        for n, m in enumerate(node_len):
            for j in range(counts[n]):
                c = min(PAGE, m - j * PAGE)
                pg = int(ids[self.off[n] + j])
                kp[pg, :, :c] = self.k[n][j * PAGE:j * PAGE + c].transpose(0, 1)
                vp[pg, :, :c] = self.v[n][j * PAGE:j * PAGE + c].transpose(0, 1)
        self.kp, self.vp = kp.cuda(), vp.cuda()
        self.qd = q.cuda()[:, 2:2 + hq] if fused else q.cuda()
        self.npo = torch.from_numpy(self.off).cuda()
        # an empty table still needs an address
        self.pid = torch.from_numpy(self.ids if total else np.zeros(1, np.int32)).cuda()

    def plan(self):
        p = deft.PromptPlan(self.parent, self.node_len, self.prompt_node, self.hkv, self.group, prompt_len=self.prompt_len)
        p.upload()
        return p

    def run(self, out_dtype=deft.DEFT_OUT_BF16, plan=None, scale=None, bufs=None):
        plan = plan or self.plan()
        out, lse = deft.deft_prompt_attn(self.qd, self.kp, self.vp, self.npo, self.pid, plan, bufs, scale=scale, out_dtype=out_dtype)
        torch.cuda.synchronize()
        assert plan.step_status() == 0
        return out.cpu(), lse.cpu()

    def reference(self, scale=None):
        """(out, lse, sum p |v| / sum p, lse tolerance), 64 bits, row by row block."""
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        dev = "cuda"
        outs, lses, means, tols = [], [], [], []
        row = 0
        for p, n in enumerate(self.prompt_node):
            way, a = [n], self.parent[n]
            while a >= 0:
                way.insert(0, a)
                a = self.parent[a]
            K = torch.cat([self.k[x] for x in way]).to(dev).double()
            V = torch.cat([self.v[x] for x in way]).to(dev).double()
            m, T = self.new[p], K.shape[0]
            if m == 0:
                continue
            q = self.q[row:row + m].to(dev).double()
            K, V = (x.repeat_interleave(self.group, 1) for x in (K, V))
            s = torch.einsum("ihd,jhd->hij", q, K) * scale
            hidden = torch.arange(T, device=dev)[None, :] > T - m + torch.arange(m, device=dev)[:, None]
            big = torch.einsum("ihd,jhd->hij", q.abs(), K.abs()).masked_fill(hidden, 0).amax(-1) * scale
            s.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[..., None])
            outs.append(torch.einsum("hij,jhd->ihd", w, V))
            means.append(torch.einsum("hij,jhd->ihd", w, V.abs()))
            lses.append(lse.T)
            # the logits' error (and that of the shift by the maximum and of
            # the sum's logarithm, each a rounding of the lse), the sum's
            tols.append((big * (self.d + 4) * 2 ** -24 + (T + 8) * 2 ** -24 + lse.abs() * 2 ** -22 + 2 ** -20).T)
            row += m
        cat = lambda x, *s: torch.cat(x).cpu() if x else torch.zeros(0, *s)  # noqa: E731
        hq = self.hkv * self.group
        return cat(outs, hq, self.d), cat(lses, hq), cat(means, hq, self.d), cat(tols, hq)

    def check(self, out_dtype=deft.DEFT_OUT_BF16, scale=None, plan=None):
        out, lse = self.run(out_dtype, scale=scale, plan=plan)
        self.compare(out, lse, scale)
        return out, lse

    def compare(self, out, lse, scale=None):
        ref, rlse, mean, tol = self.reference(scale)
        rows = sum(self.new)
        f32 = out.dtype == torch.float32
        # a probability's relative error besides its rounding is the logits'
        # absolute error, twice (once through the sum)
        bound = (2 ** -8 + 2 * tol[..., None]) * mean + (0 if f32 else 2 ** -8) * (ref.abs() + 2 ** -8 * mean) + 2 ** -24
        err = (out[:rows].double() - ref).abs()
        assert torch.isfinite(out[:rows]).all()
        assert (err <= bound).all(), f"out: {(err / bound).max():.3f} of the bound"
        lerr = (lse[:rows].double() - rlse).abs()
        assert (lerr <= tol).all(), f"lse: {(lerr / tol).max():.3f} of the bound"


def forest(lens, new=None, **kw):
    return dict(parent=[-1] * len(lens), node_len=lens, prompt_node=list(range(len(lens))), prompt_len=new, **kw)


# ---------------------------------------------------------------------------
# deft_prompt_attn
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_one_prompt(n, d):
    Case(**forest([n]), hkv=2, group=1, d=d, seed=n).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 16, 33, 64])
def test_groups(group, d):
    Case(**forest([150, 1, 37]), hkv=2, group=group, d=d, seed=group).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(10))
def test_random_trees(seed, d):
    rng = random.Random(100 + seed)
    n = rng.randint(2, 12)
    parent = [-1 if i == 0 or rng.random() < 0.15 else rng.randrange(i) for i in range(n)]
    lens = [0 if rng.random() < 0.15 else rng.choice([1, 16, rng.randint(1, 40), rng.randint(1, 500)]) for _ in range(n)]
    nodes = [rng.randrange(n) for _ in range(rng.randint(1, 8))]
    new = None if seed % 2 else [rng.choice([-1, 0, rng.randint(0, lens[x])]) for x in nodes]
    Case(parent, lens, nodes, new, hkv=rng.choice([1, 2, 3]), group=rng.choice([1, 2, 4, 6]), d=d, seed=seed, shuffle=seed % 3 != 0,
         q_pad=seed % 4).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,hkv,group", [
    ([4096], [1], 1, 8), ([4099], [3], 2, 4), ([5000, 31, 700], [40, 31, 1], 2, 3), ([2047, 1, 129], [64, 1, 129], 1, 1),
    ([3000], [200], 1, 4), ([2500, 2500], [1, 1], 4, 64)])
def test_split_ranges(lens, new, hkv, group, d):
    c = Case(**forest(lens, new), hkv=hkv, group=group, d=d, seed=7)
    plan = c.plan()
    assert plan.stats["num_split_items"] > 0
    c.check(plan=plan)
    c.check(out_dtype=deft.DEFT_OUT_F32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,hkv,group", [
    ([2227, 1960, 2297, 2209], [20] * 4, 8, 64), ([2768, 3693, 4128, 3056, 2370], [160] * 5, 4, 8)])
def test_only_the_shortest_ranges_are_cut(lens, new, hkv, group, d):
    c = Case(**forest(lens, new), hkv=hkv, group=group, d=d, seed=8)
    plan = c.plan()
    assert 0 < plan.stats["num_split_items"] < plan.stats["num_items"] // 3
    c.check(plan=plan)


@pytest.mark.parametrize("d", [64, 128])
def test_chain_of_one_token_nodes(d):
    n = 40      # every page of the path holds one token
    Case([-1] + list(range(n - 1)), [1] * n, [n - 1, 17, 0], None, hkv=1, group=2, d=d).check()


@pytest.mark.parametrize("d", [64, 128])
def test_growing_logits(d):
    """Keys scaled up along the node: later tiles exceed earlier maxima by far
    more than the rescale threshold."""
    c = Case(**forest([700]), hkv=1, group=2, d=d, seed=3)
    ramp = (1 + torch.arange(700) * 0.1)[:, None, None]
    c.k[0] = (c.k[0].float() * ramp).bfloat16()
    for j in range(44):
        m = min(16, 700 - 16 * j)
        c.kp[int(c.ids[j]), :, :m] = c.k[0][16 * j:16 * j + m].transpose(0, 1).cuda()
    c.check()
    c.check(out_dtype=deft.DEFT_OUT_F32)


@pytest.mark.parametrize("d", [64, 128])
def test_fused_projection_view_and_padding(d):
    """q as a view of a wider row, more q rows than the plan's: rows past the
    plan's are left as they were."""
    c = Case(**forest([90, 33]), hkv=2, group=2, d=d, q_pad=50, fused=True)
    assert not c.qd.is_contiguous()
    plan = c.plan()
    bufs = deft.alloc_buffers(plan, 173, 4, d)
    bufs.out.fill_(7)
    bufs.lse.fill_(9)
    out, lse = c.run(plan=plan, bufs=bufs)
    c.compare(out, lse)
    assert (out[123:] == 7).all() and (lse[123:] == 9).all()


def test_closed_forms():
    """q = 0: the mean of the values seen and ln of their number."""
    c = Case(parent=[-1, 0], node_len=[100, 60], prompt_node=[1], prompt_len=None, hkv=1, group=1, d=128)
    c.qd.zero_()
    out, lse = c.run(out_dtype=deft.DEFT_OUT_F32)
    seen = torch.arange(101, 161).double()
    assert ((lse[:, 0].double() - seen.log()).abs() < 2 ** -20).all()
    mean = torch.cat([c.v[0], c.v[1]]).double()[:, 0].cumsum(0)[100:] / seen[:, None]
    # every probability is 1: no rounding but the fp32 sums
    assert ((out[:, 0].double() - mean).abs() < 160 * 2 ** -24 * 4).all()


def test_scale_and_types():
    c = Case(**forest([200]), hkv=1, group=4, d=64)
    for scale in (0.01, 1.0):
        c.check(scale=scale)
    a, la = c.run(out_dtype=deft.DEFT_OUT_F32)
    b, lb = c.run()
    assert torch.equal(a.bfloat16(), b) and torch.equal(la, lb)


def test_repeatable_and_streams():
    """Bitwise repeatable; one plan on two streams at once, each with its own
    outputs and workspace."""
    c = Case(**forest([3000, 500], [100, 500]), hkv=2, group=4, d=128)
    plan = c.plan()
    ref = c.run(plan=plan)
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [deft.alloc_buffers(plan, 600, 8, 128) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, b in zip(streams, bufs):
            deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, b, stream=s)
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.equal(b.out.cpu(), ref[0]) and torch.equal(b.lse.cpu(), ref[1])
    assert plan.step_status() == 0


def test_captured_and_replayed():
    c = Case(**forest([2000, 77], [60, 77]), hkv=2, group=4, d=128)
    plan = c.plan()
    bufs = deft.alloc_buffers(plan, 137, 8, 128)
    ref = c.run(plan=plan)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, bufs)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, bufs)
    bufs.out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs.out.cpu(), ref[0]) and torch.equal(bufs.lse.cpu(), ref[1])


def test_rebuilt_and_uploaded_before_every_step():
    """One plan rebuilt for another batch before every step: the step reads
    the plan its upload has just copied, never the one before (both batches
    are cut into pieces, so the merge reads it too)."""
    cases = [Case(**forest([5000, 31, 700], [40, 31, 1]), hkv=2, group=3, d=64, seed=7), Case(**forest([5000], [40]), hkv=2, group=3, d=64, seed=8),
             Case(**forest([2000] * 30, [9] * 30), hkv=2, group=3, d=64, seed=9)]
    refs = [c.run() for c in cases]
    plan = cases[0].plan()
    outs = []
    for i in range(60):
        c = cases[(i * 7 + i // 3) % 3]
        plan.rebuild(c.parent, c.node_len, c.prompt_node, c.hkv, c.group, prompt_len=c.prompt_len)
        plan.upload()
        outs.append((c, deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan)))
    torch.cuda.synchronize()
    for c, (out, lse) in outs:
        out_ref, lse_ref = refs[cases.index(c)]
        assert torch.equal(out.cpu(), out_ref) and torch.equal(lse.cpu(), lse_ref)


def test_no_rows_and_refusals():
    c = Case(**forest([40], [0]), hkv=1, group=1, d=64)
    out, lse = c.run()
    assert out.shape[0] == 0
    c = Case(**forest([40]), hkv=1, group=1, d=64)
    plan = c.plan()
    with pytest.raises((ValueError, deft.DeftError)):     # fewer q rows than the plan's
        deft.deft_prompt_attn(c.qd[:39], c.kp, c.vp, c.npo, c.pid, plan)
    with pytest.raises(ValueError):
        deft.deft_prompt_attn(c.qd.float(), c.kp, c.vp, c.npo, c.pid, plan)
    with pytest.raises(ValueError):
        deft.deft_prompt_attn(c.qd.cpu(), c.kp, c.vp, c.npo, c.pid, plan)
    with pytest.raises(ValueError):
        deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo.long(), c.pid, plan)
    small = deft.alloc_buffers(plan, 40, 1, 64)
    small.workspace = small.workspace[:0]
    with pytest.raises(deft.DeftError):
        deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, small)


def test_long_prompt_against_the_definition():
    """One 6001-token prompt with grouped heads: 47 query tiles a head."""
    Case(**forest([6001]), hkv=1, group=4, d=128, seed=11).check()


def test_wide_batch():
    """More units than CTAs, so every CTA runs several in turn."""
    rng = random.Random(5)
    lens = [rng.randint(1, 400) for _ in range(120)]
    Case(**forest(lens), hkv=4, group=2, d=128, seed=12).check()
    Case(**forest(lens), hkv=4, group=3, d=64, seed=12).check()


# ---------------------------------------------------------------------------
# deft_page_table
# ---------------------------------------------------------------------------

def table_reference(lens, prev, prev_off, prev_id, free):
    off, ids, tok, slot, took = [0], [], [0], [], 0
    for n, x in enumerate(lens):
        p = prev[n] if n < len(prev) else 0
        pages = -(-x // PAGE)
        kept = min(-(-p // PAGE), pages)
        own = [int(prev_id[prev_off[n] + j]) for j in range(kept)] + [int(free[took + j]) for j in range(pages - kept)]
        took += pages - kept
        ids += own
        off.append(len(ids))
        slot += [own[t // PAGE] * PAGE + t % PAGE for t in range(p, x)]
        tok.append(len(slot))
    return off, ids, tok, slot, took


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


@pytest.mark.parametrize("nodes", [1, 2, 31, 257, 2047, 2048, 2049, 5000, 70000])
@pytest.mark.parametrize("with_prev", [False, True])
def test_page_table(nodes, with_prev):
    rng = np.random.default_rng(nodes)
    hi = 40 if nodes > 10000 else 200
    lens = rng.integers(0, hi, nodes)
    if nodes > 2:
        lens[nodes // 2] = 30000       # one node over several CTAs' shares
    n_prev = nodes - nodes // 3 if with_prev else 0
    # grown, unchanged and shrunken nodes
    prev = np.maximum(0, lens[:n_prev] + rng.integers(-40, 20, n_prev)) if n_prev else np.zeros(0, int)
    prev_pages = -(-prev // PAGE)
    prev_off = np.concatenate([[0], np.cumsum(prev_pages)])
    pool = rng.permutation(int(prev_off[-1]) + int((-(-lens // PAGE)).sum()) + 5)
    prev_id, free = pool[:prev_off[-1]], pool[prev_off[-1]:]
    off, ids, tok, slot, took = table_reference(lens, prev, prev_off, prev_id, free)
    t = deft.deft_page_table(cu(lens), cu(free), prev=(cu(prev), cu(prev_off), cu(prev_id)) if n_prev else None, max_pages=len(ids) + 3,
                             max_tokens=len(slot) + 37)
    assert t.counts.tolist() == [len(ids), took, len(slot), 0]
    assert t.page_off.tolist() == off and t.page_id[:len(ids)].tolist() == ids
    assert t.tok_off.tolist() == tok and t.slot.tolist() == slot + [-1] * 37


def test_page_table_leaves_the_rest_and_reuses_tensors():
    t = deft.alloc_page_table(3, 10, 40)
    t.page_id.fill_(-7)
    for lens in ([20, 0, 5], [1, 1, 1]):
        deft.deft_page_table(cu(lens), cu(range(9)), table=t)
        used = sum(-(-x // PAGE) for x in lens)
        assert t.counts.tolist() == [used, used, sum(lens), 0]
        assert t.slot.tolist()[sum(lens):] == [-1] * (40 - sum(lens))
    assert t.page_id.tolist()[3:] == [-7] * 7


@pytest.mark.parametrize("nodes", [3, 3000])
def test_page_table_reports(nodes):
    """Every shortage is reported, nothing is written past a capacity, tokens
    without a page get -1."""
    lens = [33] + [1] * (nodes - 1)
    need, toks = nodes + 2, nodes + 32
    t = deft.deft_page_table(cu(lens), cu(range(2)), max_pages=need, max_tokens=toks)
    assert t.counts.tolist() == [need, need, toks, deft.TABLE_NO_FREE_PAGE]
    assert t.page_id.tolist() == [0, 1] + [-1] * (need - 2) and t.slot.tolist() == list(range(32)) + [-1] * (toks - 32)
    big = deft.alloc_page_table(nodes, need, toks)
    big.page_id.fill_(-7)
    big.slot.fill_(-7)
    full_p, full_s = big.page_id, big.slot
    big.page_id, big.slot = full_p[:2], full_s[:5]
    deft.deft_page_table(cu(lens), cu(range(need)), table=big)
    assert big.counts.tolist() == [need, need, toks, deft.TABLE_PAGE_CAP | deft.TABLE_TOKEN_CAP]
    assert full_p.tolist() == [0, 1] + [-7] * (need - 2) and full_s.tolist() == list(range(5)) + [-7] * (toks - 5)
    bad = list(lens)
    bad[-1] = -5
    t = deft.deft_page_table(cu(bad), cu(range(need)), max_pages=need, max_tokens=toks)
    assert t.counts.tolist() == [need - 1, need - 1, toks - 1, deft.TABLE_BAD_LENGTH]
    # earlier pages outside the earlier table
    t = deft.deft_page_table(cu(lens), cu(range(need)), prev=(cu([16]), cu([5]), cu([3, 4])), max_pages=need, max_tokens=toks)
    assert t.counts.tolist()[3] == deft.TABLE_BAD_PREV and t.page_id.tolist()[0] == -1
    # sums past 31 bits
    t = deft.deft_page_table(cu([2 ** 31 - 1] * nodes), cu(range(4)), max_pages=4, max_tokens=8)
    assert t.counts.tolist()[2:] == [2 ** 31 - 1, deft.TABLE_NO_FREE_PAGE | deft.TABLE_PAGE_CAP | deft.TABLE_TOKEN_CAP]
    assert t.page_id.tolist() == [0, 1, 2, 3] and t.slot.tolist() == list(range(8))


def test_page_table_captured():
    lens, free = cu([40, 3]), cu(range(10, 20))
    t = deft.alloc_page_table(2, 8, 64)
    deft.deft_page_table(lens, free, table=t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        deft.deft_page_table(lens, free, table=t)
    lens.copy_(cu([1, 17]))
    g.replay()
    assert t.counts.tolist() == [3, 3, 18, 0] and t.page_id.tolist()[:3] == [10, 11, 12]
    assert t.slot.tolist()[:18] == [160] + list(range(176, 193))


# ---------------------------------------------------------------------------
# deft_kv_write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,hkv", [(1, 1), (5, 3), (33, 8), (1000, 2), (4097, 1)])
def test_kv_write(tokens, hkv, d, dtype):
    g = torch.Generator().manual_seed(tokens)
    rng = np.random.default_rng(tokens)
    qkv = torch.randn((tokens, 3 * hkv, d), generator=g).to(dtype).cuda()
    k, v = qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:]
    pages = -(-tokens // PAGE) + 3
    slot = rng.permutation(pages * PAGE)[:tokens]
    slot[rng.random(tokens) < 0.1] = -1
    if tokens > 2:
        slot[1] = pages * PAGE          # behind the pool: skipped as well
    kp = torch.full((pages, hkv, PAGE, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, 4.0)
    wk, wv = kp.cpu(), vp.cpu()
    for t, s in enumerate(slot):
        if 0 <= s < pages * PAGE:
            wk[s // PAGE, :, s % PAGE] = k[t].cpu().bfloat16()
            wv[s // PAGE, :, s % PAGE] = v[t].cpu().bfloat16()
    deft.deft_kv_write(k, v, cu(slot), kp, vp)
    assert torch.equal(kp.cpu(), wk) and torch.equal(vp.cpu(), wv)


def test_kv_write_specials_and_refusals():
    k = torch.tensor([NAN, math.inf, -math.inf, 1e-40, 3.4e38, 1 + 2 ** -8, 1 + 3 * 2 ** -8, -0.0] * 8).view(1, 1, 64).cuda()
    kp = torch.zeros((1, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    deft.deft_kv_write(k, -k, cu([3]), kp, vp)
    assert torch.equal(kp[0, 0, 3].isnan(), k[0, 0].bfloat16().isnan())
    assert torch.equal(kp[0, 0, 3].nan_to_num(1).view(torch.int16), k[0, 0].bfloat16().nan_to_num(1).view(torch.int16))
    deft.deft_kv_write(k[:0], k[:0], cu([]), kp, vp)
    with pytest.raises(ValueError):
        deft.deft_kv_write(k, k.bfloat16(), cu([0]), kp, vp)
    with pytest.raises(ValueError):
        deft.deft_kv_write(k.half(), k.half(), cu([0]), kp, vp)
    with pytest.raises(ValueError):
        deft.deft_kv_write(k, k, cu([0, 1]), kp, vp)
    with pytest.raises(ValueError):
        deft.deft_kv_write(k, k, cu([0]).cpu(), kp, vp)
    with pytest.raises(deft.DeftError):     # rows that are not 16-byte aligned
        deft.deft_kv_write(*(torch.zeros(65, device="cuda")[1:].view(1, 1, 64) for _ in "kv"), cu([0]), kp, vp)


# ---------------------------------------------------------------------------
# Together: prefill of a prefix, prefill of branches under it, a decode step
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,group,d", [(2, 4, 128), (4, 1, 64)])
def test_prefill_then_tree_decode(hkv, group, d):
    """A 300-token prefix and 20 branches of 45 tokens under it enter the
    cache through deft_page_table and deft_kv_write, attend through
    deft_prompt_attn, then grow by a token each and take a tree step."""
    hq, pool = hkv * group, deft.PagePool(200)
    parent = [-1] + [0] * 20
    lens_at = [[300] + [0] * 20, [300] + [45] * 20, [300] + [46] * 20]
    c = Case(parent, lens_at[2], list(range(21)), None, hkv, group, d, seed=21)      # every token's K and V, and q rows
    kp = torch.full((200, hkv, PAGE, d), NAN, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    prev, spec = None, None
    qrow = dict(zip(range(21), np.concatenate([[0], np.cumsum(lens_at[2])[:-1]])))
    ref, rlse, mean, tol = c.reference()
    before = [0] * 21
    for lens in lens_at[:2]:
        free = pool.alloc(sum(-(-x // PAGE) for x in lens) - sum(-(-x // PAGE) for x in before))
        t = deft.deft_page_table(cu(lens), cu(free), prev=prev, max_pages=200, max_tokens=1500)
        total = sum(lens) - sum(before)
        assert t.counts.tolist() == [sum(-(-x // PAGE) for x in lens), len(free), total, 0]
        pad = torch.zeros((1500 - total, hkv, d), dtype=torch.bfloat16)
        k, v = (torch.cat([x[n][before[n]:lens[n]] for n in range(21)] + [pad]).cuda() for x in (c.k, c.v))
        deft.deft_kv_write(k, v, t.slot, kp, vp)
        nodes = [n for n in range(21) if lens[n] > before[n]]
        plan = deft.PromptPlan(parent, lens, nodes, hkv, group, prompt_len=[lens[n] - before[n] for n in nodes])
        plan.upload()
        rows = np.concatenate([qrow[n] + np.arange(before[n], lens[n]) for n in nodes])
        out, lse = deft.deft_prompt_attn(c.q[rows].cuda(), kp, vp, t.page_off, t.page_id, plan)
        err = (out.cpu().double() - ref[rows]).abs()
        bound = (2 ** -8 + 2 * tol[rows][..., None]) * mean[rows] + 2 ** -8 * (ref[rows].abs() + 2 ** -8 * mean[rows]) + 2 ** -24
        assert (err <= bound).all() and ((lse.cpu().double() - rlse[rows]).abs() <= tol[rows]).all()
        prev, before = (cu(lens), t.page_off, t.page_id), lens
    lens = lens_at[2]
    free = pool.alloc(sum(-(-x // PAGE) for x in lens) - sum(-(-x // PAGE) for x in before))
    t = deft.deft_page_table(cu(lens), cu(free), prev=prev, max_pages=200, max_tokens=20)
    assert t.counts.tolist()[3] == 0
    k, v = (torch.cat([x[n][45:46] for n in range(1, 21)]).cuda() for x in (c.k, c.v))
    deft.deft_kv_write(k, v, t.slot, kp, vp)
    assert deft.deft_check_pages(lens, t.page_off.cpu().numpy(), t.page_id.cpu().numpy(), 200) == 0
    plan = deft.Plan(parent, lens, list(range(1, 21)), 256, group)
    plan.upload()
    rows = [qrow[n] + 45 for n in range(1, 21)]
    out, lse = deft.deft_tree_attn(c.q[rows].cuda(), kp, vp, t.page_off, t.page_id, plan)
    # the tree step's own tolerances
    assert (out.cpu().double() - ref[rows]).abs().max() <= 1e-2 and (lse.cpu().double() - rlse[rows]).abs().max() <= 1e-3
    # and the prompt step on the same single tokens
    plan = deft.PromptPlan(parent, lens, list(range(1, 21)), hkv, group, prompt_len=[1] * 20)
    plan.upload()
    out, lse = deft.deft_prompt_attn(c.q[rows].cuda(), kp, vp, t.page_off, t.page_id, plan)
    err = (out.cpu().double() - ref[rows]).abs()
    assert (err <= (2 ** -8 + 2 * tol[rows][..., None]) * mean[rows] + 2 ** -8 * (ref[rows].abs() + 2 ** -8 * mean[rows]) + 2 ** -24).all()


def test_pages_behind_four_gigabytes():
    """A cache of 6.4 GB a pool: pages whose offsets pass 32 bits, in elements
    and in bytes, written and read."""
    hkv, d, pages = 8, 128, 200000
    kp, vp = (torch.empty((pages, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    c = Case(**forest([300, 77], [300, 20]), hkv=hkv, group=1, d=d, seed=31)
    free = np.concatenate([[0, 70000, 140000], np.arange(pages - 40, pages)]).astype(np.int32)
    t = deft.deft_page_table(cu([300, 77]), cu(free), max_pages=30, max_tokens=377)
    assert t.counts.tolist() == [24, 24, 377, 0] and t.slot.max().item() > 3 * 10 ** 6
    deft.deft_kv_write(*(torch.cat(x).cuda() for x in (c.k, c.v)), t.slot, kp, vp)
    plan = c.plan()
    out, lse = deft.deft_prompt_attn(c.qd, kp, vp, t.page_off, t.page_id, plan)
    c.compare(out.cpu(), lse.cpu())


@pytest.mark.parametrize("raw", [False, True])
def test_buffers_allocated_by_a_call_on_another_stream(raw):
    """Outputs and workspace that the call allocates itself belong to its
    stream: what the current stream allocates and fills right behind the call
    is other memory, although the call still waits for a busy stream."""
    c = Case(**forest([3000, 500], [100, 500]), hkv=2, group=4, d=128, seed=41)
    plan = c.plan()
    ref = c.run(plan=plan)
    ws = plan.workspace_bytes(8, 128)
    lens, free = cu([700, 3]), cu(np.arange(60))
    table = deft.deft_page_table(lens, free, max_pages=50, max_tokens=800)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            x = big @ big      # the side stream is busy when the call is enqueued
        s = side.cuda_stream if raw else side
        out, lse = deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, stream=s)
        t = deft.deft_page_table(lens, free, max_pages=50, max_tokens=800, stream=s)
        for n in (ws, out.numel() * 2, 4 * lse.numel(), 3200, 200):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])
        assert torch.equal(t.slot, table.slot) and torch.equal(t.counts, table.counts)
        del out, lse, t, x


def test_two_layers_share_a_plan_and_a_workspace():
    """Layer after layer with one plan, one workspace and one set of pages
    each, as a model runs them on one stream."""
    cases = [Case(**forest([3000, 40], [70, 40]), hkv=2, group=4, d=128, seed=s, shuffle=False) for s in (1, 2)]
    plan = cases[0].plan()
    ws = deft.alloc_buffers(plan, 110, 8, 128)
    outs = []
    for c in cases * 3:
        b = deft.StepBuffers(torch.empty_like(ws.out), torch.empty_like(ws.lse), ws.workspace)
        outs.append((c, deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, b)))
    torch.cuda.synchronize()
    for c, (out, lse) in outs:
        c.compare(out.cpu(), lse.cpu())


def test_behind_other_kernels_of_the_stream():
    """The step behind kernels that make its inputs (it may start while they
    end): q, the pages and the page table all written right before it."""
    c = Case(**forest([700, 130], [300, 130]), hkv=2, group=2, d=128, seed=33)
    plan = c.plan()
    ref = c.run(plan=plan)
    q, kp, vp = c.qd.clone(), c.kp.clone(), c.vp.clone()
    for _ in range(20):
        c.qd.zero_(), c.kp.zero_(), c.vp.zero_(), c.pid.zero_()
        big = torch.randn(4096, 4096, device="cuda")
        big = big @ big      # keeps the device busy while the rest is enqueued
        c.qd.copy_(q), c.kp.copy_(kp), c.vp.copy_(vp)
        c.pid.copy_(torch.from_numpy(c.ids))
        out, lse = deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan)
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])


@pytest.mark.parametrize("i", [1, 4])
def test_workload_prefill(i):
    """Every node of a benchmark tree as a prompt."""
    s = W.config(i)
    Case(s.parent.tolist(), s.node_len.tolist(), list(range(s.num_nodes)), None, min(s.num_kv_heads, 2), s.gqa_group, s.head_dim, seed=i).check()


@pytest.mark.parametrize("out_dtype", [deft.DEFT_OUT_BF16, deft.DEFT_OUT_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("cut", [False, True])
def test_partly_filled_tiles(cut, group, d, out_dtype):
    """Query tiles whose last warp holds 1 to 31 rows, as tile A and as tile
    B, of whole and of cut ranges, both output types."""
    tile = 128 // group
    m = sorted({1, 2, 10, 11, 21, 31, 33, tile - 1, tile + 1, tile + 11, 2 * tile - 1} - {tile, 2 * tile})
    c = Case(**forest([3000 + 16 * x for x in m] if cut else m, m), hkv=1, group=group, d=d, seed=51)
    plan = c.plan()
    assert (plan.stats["num_split_items"] > 0) == cut
    c.check(out_dtype=out_dtype, plan=plan)


def memory_stream(t):
    """The stream whose memory tensor t lies in."""
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]][0]


@pytest.mark.parametrize("default", [True, False])
def test_memory_of_raw_handles(default):
    """A raw handle, the default stream's 0 among them: what a call allocates
    comes from that stream's memory, and goes back to it call after call."""
    c = Case(**forest([3000, 500], [100, 500]), hkv=2, group=4, d=128, seed=42)
    plan = c.plan()
    ref = c.run(plan=plan)
    lens, free = cu([700, 3]), cu(np.arange(60))
    side = torch.cuda.Stream()
    handle = 0 if default else side.cuda_stream
    torch.cuda.synchronize()
    held = None
    for i in range(40):
        with torch.cuda.stream(side if default else torch.cuda.default_stream()):
            out, lse = deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, stream=handle)
            t = deft.deft_page_table(lens, free, max_pages=50, max_tokens=800, stream=handle)
        assert {memory_stream(x) for x in (out, lse, t.page_off, t.page_id, t.tok_off, t.slot, t.counts)} == {handle}
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])
        if i == 2:
            held = torch.cuda.memory_reserved()
    assert torch.cuda.memory_reserved() == held


def test_buffers_of_the_default_stream_by_its_handle():
    """As test_buffers_allocated_by_a_call_on_another_stream, the streams
    exchanged: the default stream is busy and named by its handle, 0, and a
    side stream is the current one."""
    c = Case(**forest([3000, 500], [100, 500]), hkv=2, group=4, d=128, seed=43)
    plan = c.plan()
    ref = c.run(plan=plan)
    ws = plan.workspace_bytes(8, 128)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        x = big @ big
        with torch.cuda.stream(side):
            out, lse = deft.deft_prompt_attn(c.qd, c.kp, c.vp, c.npo, c.pid, plan, stream=0)
            for n in (ws, out.numel() * 2, 4 * lse.numel()):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])
        del out, lse, x


@pytest.mark.parametrize("default", [True, False])
@pytest.mark.parametrize("raw", [True, False])
def test_tree_step_memory(raw, default):
    """The tree steps' own buffers belong to the stream the step runs on too."""
    s = W.tiny_tree()
    layout = W.paged_layout(s)
    t = W.make_tensors(s, layout, device="cuda:0")
    plan = deft.Plan(s.parent, s.node_len, s.query_node, 64, s.gqa_group)
    plan.upload()
    args = (t.q, t.k_pages, t.v_pages, cu(layout.node_page_off), cu(layout.page_id), plan)
    ref = deft.deft_tree_attn(*args)
    side = torch.cuda.Stream()
    on, current = (torch.cuda.default_stream(), side) if default else (side, torch.cuda.default_stream())
    torch.cuda.synchronize()
    for step in (deft.deft_tree_attn, deft.deft_naive_attn):
        with torch.cuda.stream(current):
            out, lse = step(*args, stream=on.cuda_stream if raw else on)
        assert memory_stream(out) == memory_stream(lse) == on.cuda_stream
        torch.cuda.synchronize()
        assert (out - ref[0]).abs().max() <= 1e-2 and (lse - ref[1]).abs().max() <= 1e-3


def check_special(c, plan, out_dtype):
    """out and lse of a case with non-finite q or K: NaN exactly where the
    64-bit form is, the other rows within their bounds (of the finite values:
    a logit of -infinity is exact)."""
    out, lse = c.run(out_dtype, plan=plan)
    ref, rlse, mean, _ = c.reference()
    kept = c.q, c.k
    c.q, c.k = c.q.nan_to_num(0, 0, 0), [x.nan_to_num(0, 0, 0) for x in c.k]
    tol = c.reference()[3]
    c.q, c.k = kept
    bad = ref.isnan()
    assert bad.any() and (bad.any(-1) == bad.all(-1)).all()
    assert torch.equal(out.isnan(), bad)
    good = ~bad.all(-1)
    f32 = out.dtype == torch.float32
    bound = (2 ** -8 + 2 * tol[..., None]) * mean + (0 if f32 else 2 ** -8) * (ref.abs() + 2 ** -8 * mean) + 2 ** -24
    assert ((out.double() - ref).abs() <= bound)[good].all()
    assert ((lse.double() - rlse).abs() <= tol)[good].all()
    return lse, ~good


SPECIAL = [([200], None, False), ([300, 40], [70, 40], False), ([4099, 150], [70, 150], True), ([5000], [200], True)]


@pytest.mark.parametrize("out_dtype", [deft.DEFT_OUT_BF16, deft.DEFT_OUT_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("lens,new,cut", SPECIAL)
def test_non_finite_queries(lens, new, cut, value, d, out_dtype):
    """A row whose query holds a NaN or an infinity (logits of both signs) is
    NaN in out and lse, whole or cut; the rows beside it are not touched."""
    c = Case(**forest(lens, new), hkv=2, group=3, d=d, seed=61)
    plan = c.plan()
    assert (plan.stats["num_split_items"] > 0) == cut
    for row in (33, 60, 69):
        c.q[row, 1, 5] = value      # one head of KV head 0
    # the keys of the first two tokens: logits of both signs for every row
    c.k[0][0, 0, 5], c.k[0][1, 0, 5] = 1, -1
    c.kp[int(c.ids[c.off[0]]), 0, 0, 5], c.kp[int(c.ids[c.off[0]]), 0, 1, 5] = 1, -1
    c.qd = c.q.cuda()
    lse, bad = check_special(c, plan, out_dtype)
    assert bad.sum() == 3 and lse[bad].isnan().all()


@pytest.mark.parametrize("out_dtype", [deft.DEFT_OUT_BF16, deft.DEFT_OUT_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,cut", SPECIAL)
def test_logits_of_minus_infinity(lens, new, cut, d, out_dtype):
    """A row whose logits are all -infinity has no softmax: out NaN, lse
    -infinity, whole or cut."""
    c = Case(**forest(lens, new), hkv=2, group=3, d=d, seed=62)
    plan = c.plan()
    assert (plan.stats["num_split_items"] > 0) == cut
    c.k[0][:, 0, 5] = -1
    for j in range(-(-lens[0] // PAGE)):
        c.kp[int(c.ids[c.off[0] + j]), 0, :min(PAGE, lens[0] - PAGE * j), 5] = -1
    c.q[33, 1, 5] = math.inf
    c.q[60, 2, 5] = math.inf
    c.qd = c.q.cuda()
    lse, bad = check_special(c, plan, out_dtype)
    assert bad.sum() == 2 and lse[33, 1] == lse[60, 2] == -math.inf


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, math.inf])
@pytest.mark.parametrize("place", [3, -50, -1])
@pytest.mark.parametrize("lens,new,cut", SPECIAL)
def test_non_finite_keys(lens, new, cut, place, value, d):
    """A non-finite key reaches the rows that attend it, in whichever piece it
    lies, and no other: NaN where its logit is NaN or +infinity."""
    c = Case(**forest(lens, new), hkv=2, group=3, d=d, seed=63)
    plan = c.plan()
    assert (plan.stats["num_split_items"] > 0) == cut
    at = place % lens[0]
    c.k[0][at, 1, 7] = value
    c.kp[int(c.ids[c.off[0] + at // PAGE]), 1, at % PAGE, 7] = value
    # KV head 1's query heads 3, 4 and 5: logits of +, - and any sign there
    c.q[:, 3, 7] = 1 + c.q[:, 3, 7].abs()
    c.q[:, 4, 7] = -1 - c.q[:, 4, 7].abs()
    c.qd = c.q.cuda()
    lse, bad = check_special(c, plan, deft.DEFT_OUT_BF16)
    assert not lse[bad].isfinite().any()
    seen = torch.arange(sum(c.new)) < c.new[0]
    seen[:c.new[0]] = torch.arange(lens[0] - c.new[0], lens[0]) >= at
    assert not bad[~seen].any() and not bad[:, :3].any()
    assert bad[seen][:, 3].all() and bad[seen][:, 4].all() == math.isnan(value)


@pytest.mark.parametrize("nodes", [3, 3000])
def test_page_table_highest_page(nodes):
    """Page numbers up to 2^27 - 1, whose last slot is 2^31 - 1; a listed
    number outside 0 .. 2^27 - 1 is copied to page_id and its slots are -1."""
    top = 2 ** 27 - 1
    lens, prev = [40, 20, 5] + [0] * (nodes - 3), [3, 0, 0]
    free = [top - 1, top, 7, -4, 2 ** 27]
    t = deft.deft_page_table(cu(lens), cu(free), prev=(cu(prev), cu([0, 1, 1]), cu([top])), max_pages=6, max_tokens=62)
    assert t.counts.tolist() == [6, 5, 62, 0] and t.page_id.tolist() == [top] + free
    base = [16 * top + i for i in range(3, 16)] + [16 * (top - 1) + i for i in range(16)] + [16 * top + i for i in range(8)]
    assert t.slot.tolist() == base + [7 * 16 + i for i in range(16)] + [-1] * 9


@pytest.mark.parametrize("nodes", [511 * 2048 + 1, 1 << 20])
def test_page_table_largest(nodes):
    """The most nodes a call takes, 512 blocks of 2048, and one node in the
    last block."""
    rng = np.random.default_rng(nodes)
    lens = rng.integers(0, 24, nodes)
    n_prev = nodes - nodes // 3
    prev = np.maximum(0, lens[:n_prev] + rng.integers(-20, 12, n_prev))
    pages, prev_pages = -(-lens // PAGE), -(-prev // PAGE)
    prev_off = np.concatenate([[0], np.cumsum(prev_pages)])
    pool = rng.permutation(int(prev_off[-1]) + int(pages.sum()) + 5)
    prev_id, free = pool[:prev_off[-1]], pool[prev_off[-1]:]
    all_prev = np.concatenate([prev, np.zeros(nodes - n_prev, int)])
    kept = np.minimum(-(-all_prev // PAGE), pages)
    fresh = np.maximum(lens - all_prev, 0)
    off, tok, take = (np.concatenate([[0], np.cumsum(x)]) for x in (pages, fresh, pages - kept))
    node = np.repeat(np.arange(nodes), pages)
    j = np.arange(off[-1]) - off[node]
    old = j < kept[node]
    ids = np.where(old, prev_id[np.where(old, np.concatenate([prev_off[:-1], np.zeros(nodes - n_prev, int)])[node] + j, 0)],
                   free[np.where(old, 0, take[node] + j - kept[node])])
    node = np.repeat(np.arange(nodes), fresh)
    t = all_prev[node] + np.arange(tok[-1]) - tok[node]
    slot = ids[off[node] + t // PAGE] * PAGE + t % PAGE
    got = deft.deft_page_table(cu(lens), cu(free), prev=(cu(prev), cu(prev_off), cu(prev_id)), max_pages=len(ids) + 3, max_tokens=len(slot) + 37)
    assert got.counts.tolist() == [off[-1], take[-1], tok[-1], 0]
    assert np.array_equal(got.page_off.cpu().numpy(), off) and np.array_equal(got.tok_off.cpu().numpy(), tok)
    assert np.array_equal(got.page_id.cpu().numpy()[:len(ids)], ids)
    assert np.array_equal(got.slot.cpu().numpy(), np.concatenate([slot, np.full(37, -1)]))


@pytest.mark.parametrize("d", [64, 128])
def test_replays_write_everything(d):
    """A captured step with a cut range: every replay writes out, lse and the
    partial rows anew, whatever lies there before."""
    c = Case(**forest([2000, 77], [60, 77]), hkv=2, group=4, d=d, seed=71)
    plan = c.plan()
    assert plan.stats["num_split_items"] > 0
    bufs = deft.alloc_buffers(plan, 137, 8, d)
    ref = c.run(plan=plan)
    args = (c.qd, c.kp, c.vp, c.npo, c.pid, plan, bufs)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        deft.deft_prompt_attn(*args)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        deft.deft_prompt_attn(*args)
    for _ in range(3):
        bufs.out.fill_(7)
        bufs.lse.fill_(NAN)
        bufs.workspace.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.out.cpu(), ref[0]) and torch.equal(bufs.lse.cpu(), ref[1])
    assert plan.step_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_and_one_long_range(d):
    """A decode batch of 160 requests and 8 KV heads with one context far
    longer than the rest, whether the plan cuts it or not."""
    Case(**forest([20000] + [300 + i for i in range(159)], [1] * 160), hkv=8, group=1, d=d, seed=72).check()


@pytest.mark.parametrize("lens,new,hkv,group", [([2200] * 4, [20] * 4, 8, 64), ([8192] * 8, [512] * 8, 2, 4), ([1000] * 40, [9] * 40, 4, 5)])
def test_equal_lengths(lens, new, hkv, group):
    """Batches of one length, whose units do not divide among the CTAs."""
    c = Case(**forest(lens, new), hkv=hkv, group=group, d=128, seed=73)
    c.check()


def test_launches_report_their_own_errors():
    """A call that failed before (a status read of a capturing stream: refused
    by CUDA on the host, the graph dropped unused) does not show in the calls
    behind it."""
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    plan = deft.PromptPlan(None, [5], [0], 1)
    plan.upload()
    side = torch.cuda.Stream()
    raw, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    k = torch.ones((40, 1, 64), dtype=torch.bfloat16, device="cuda")
    kp, vp = (torch.zeros((3, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lens = {n: cu([1] * n) for n in (40, 4000)}
    free = cu(range(4000))
    torch.cuda.synchronize()

    def fail():
        assert rt.cudaStreamBeginCapture(raw, 2) == 0      # relaxed
        with pytest.raises(deft.DeftError):
            plan.step_status(stream=side)
        assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()

    fail()
    deft.deft_kv_write(k, k, cu(range(40)), kp, vp)
    assert (kp.transpose(1, 2).reshape(48, 64)[:40] == 1).all()
    for n in (40, 4000):
        fail()
        t = deft.deft_page_table(lens[n], free, max_pages=n, max_tokens=n)
        assert t.counts.tolist() == [n, n, n, 0] and t.slot.tolist() == list(range(0, 16 * n, 16))
