"""The append calls (head norms, rotation, K and V into bf16 or 4-bit pages)
and the way back from 4-bit pages, against numpy in 64 bits."""
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


def table(rot, n, seed=3):
    """cos and sin of random angles, as a table."""
    a = np.random.default_rng(seed).uniform(-50, 50, (n, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Rows:
    """A projection's output, the pools and slots for it."""

    def __init__(self, T, hq, hkv, d, f32=False, rot=0, interleaved=False, norm=True, seed=0, pad=0, skip=(), scale=1.0):
        rng = np.random.default_rng(seed)
        dt = torch.float32 if f32 else torch.bfloat16
        self.T, self.hq, self.hkv, self.d = T, hq, hkv, d
        fused = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv + pad, d)).astype(np.float32) * scale).to(dt).cuda()
        self.q, self.k, self.v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:hq + 2 * hkv]
        self.pages = -(-T // 16) + 3
        self.slot = rng.permutation(self.pages * 16)[:T].astype(np.int32)
        self.slot[list(skip)] = -1
        self.kw = {"eps": 1e-5}
        self.w = [None, None]
        if norm:
            self.w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(d).astype(np.float32)).to(dt).cuda() for _ in "qk"]
            self.kw.update(q_norm=self.w[0], k_norm=self.w[1])
        self.cos_sin = self.position = None
        self.interleaved = interleaved
        if rot:
            self.cos_sin, self.position = table(rot, 97), rng.integers(0, 97, T)
            self.kw.update(cos_sin=cu(self.cos_sin, np.float32), position=cu(self.position), interleaved=interleaved)

    def pools(self):
        return [torch.full((self.pages, self.hkv, 16, self.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def pools4(self):
        return [torch.full((self.pages, self.hkv, 9 * self.d), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]

    def expect(self, which):
        """float64 rows of q or k, and a bound on what fp32 arithmetic leaves
        open: ten roundings of at most 2^-24, each of terms no larger than the
        pair's magnitudes (and the weights' share of the norm)."""
        x, w = ((self.q, self.w[0]), (self.k, self.w[1]))[which]
        y = ref.turned(f64(x), None if w is None else f64(w), 1e-5, self.cos_sin, self.position, self.interleaved)
        big = np.abs(ref.turned(f64(x), None if w is None else f64(w), 1e-5, None, None, False)).max(-1, keepdims=True)
        # the sum of squares: log2(d) + 1 roundings more
        return y, (10 + math.log2(self.d)) * 2.0 ** -24 * 2 * big

    def at(self, pool, rows):
        s = self.slot[rows]
        return pool[s // 16, :, s % 16]


def close(got, want, slack):
    """bf16 of a value known to `slack`: half a step, relative to the value, and what lies under it."""
    assert got.shape == want.shape
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + slack) + slack).all()


CASES = [
    dict(T=1, hq=1, hkv=1, d=64), dict(T=1, hq=32, hkv=8, d=128, rot=128), dict(T=2, hq=3, hkv=1, d=64, rot=64, interleaved=True),
    dict(T=17, hq=12, hkv=4, d=64, rot=16), dict(T=33, hq=5, hkv=5, d=128, rot=16, interleaved=True), dict(T=40, hq=7, hkv=1, d=128, rot=48),
    dict(T=19, hq=9, hkv=3, d=128, rot=64, f32=True), dict(T=300, hq=32, hkv=8, d=128, rot=128, skip=(0, 7, 299)),
    dict(T=23, hq=4, hkv=2, d=64, rot=48, f32=True, interleaved=True, pad=1), dict(T=31, hq=16, hkv=2, d=64, rot=64, f32=True),
    dict(T=9, hq=6, hkv=6, d=128, norm=False, rot=128), dict(T=9, hq=6, hkv=6, d=64, norm=False, pad=2), dict(T=5, hq=64, hkv=33, d=128, rot=112),
    dict(T=1000, hq=8, hkv=8, d=64, rot=64, f32=True), dict(T=5000, hq=4, hkv=1, d=128, rot=128), dict(T=3001, hq=2, hkv=3, d=64, rot=32),
]


@pytest.mark.parametrize("c", CASES)
def test_qkv_write(c):
    r = Rows(**c)
    kp, vp = r.pools()
    q = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw)
    close(f64(q), *r.expect(0))
    kept = np.nonzero(r.slot >= 0)[0]
    close(r.at(f64(kp), kept), *(x[kept] for x in r.expect(1)))
    assert (r.at(f64(vp), kept) == f64(r.v.to(torch.bfloat16))[kept]).all()
    free = np.setdiff1d(np.arange(r.pages * 16), r.slot)
    for pool in (kp, vp):       # nothing else is written
        assert (f64(pool)[free // 16, :, free % 16] == 7).all()


@pytest.mark.parametrize("c", CASES)
def test_each_operation_rounds_by_itself(c):
    """Bit for bit what 32-bit arithmetic gives, operation by operation."""
    r = Rows(**c)
    kp, vp = r.pools()
    q = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw)
    kept = np.nonzero(r.slot >= 0)[0]
    for got, x, w, rows in ((f64(q), r.q, r.w[0], slice(None)), (r.at(f64(kp), kept), r.k, r.w[1], kept)):
        want = ref.turned32(f64(x), None if w is None else f64(w), 1e-5, r.cos_sin, r.position, r.interleaved)
        assert want.dtype == np.float32 and (got == ref.bf16(want)[rows]).all()


@pytest.mark.parametrize("g", [(1.0, 1.0), (0.25, 4.0), (0.37, 1.9)])
@pytest.mark.parametrize("c", CASES)
def test_qkv_write4(c, g):
    """The queries are deft_qkv_write's, and the 4-bit rows are what the
    format makes of its bf16 rows, bit for bit."""
    r = Rows(**c)
    kp, vp = r.pools()
    q = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw)
    k4, v4 = r.pools4()
    q4 = deft.deft_qkv_write4(r.q, r.k, r.v, cu(r.slot), k4, v4, k_scale=g[0], v_scale=g[1], **r.kw)
    assert torch.equal(q, q4)
    kept = np.nonzero(r.slot >= 0)[0]
    for pool, pool4, x in ((kp, k4, g[0]), (vp, v4, g[1])):
        codes, scales = ref.pages(pool4.cpu().numpy())
        want_c, want_s, _ = ref.quantise(r.at(f64(pool), kept), x)
        assert (r.at(codes, kept) == want_c).all() and (r.at(scales, kept) == want_s).all()
    free = np.setdiff1d(np.arange(r.pages * 16), r.slot)
    for pool in (k4, v4):
        codes, scales = ref.pages(pool.cpu().numpy())
        assert (scales[free // 16, :, free % 16] == 0xA5).all()
        c4 = codes[free // 16, :, free % 16]
        assert (c4[..., 0::2] == 5).all() and (c4[..., 1::2] == 0xA).all()


def test_write4_halfway_values():
    """Elements halfway between two codes, for every scale that the largest
    element can make: to the even code.  All seven borders times 127 scales."""
    d = 64
    s = ref.E4M3[1:]
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    rows = []
    for v in s:
        b = np.zeros(16)
        b[0] = 6 * v
        b[1:8], b[8:15] = mids * v, -mids * v
        rows.append(b)
    x = np.zeros((-(-len(rows) // 4) * 4, 16))
    x[:len(rows)] = rows
    x = x.reshape(-1, 1, d)
    assert (ref.bf16(x) == x).all()
    t = cu(x, np.float32).bfloat16()
    slot = cu(np.arange(len(x)))
    k4, v4 = deft.alloc_kv4_pages(-(-len(x) // 16), 1, d)
    assert deft.deft_qkv_write4(None, t, -t, slot, k4, v4) is None
    for pool, sign in ((k4, 1), (v4, -1)):
        codes, scales = ref.pages(pool.cpu().numpy())
        want_c, want_s, _ = ref.quantise(f64(sign * t), 1.0)
        got = codes.transpose(0, 2, 1, 3).reshape(-1, 1, d)[:len(x)]
        assert (got == want_c).all()
        assert (scales.transpose(0, 2, 1, 3).reshape(-1, 1, d // 16)[:len(x)] == want_s).all()


@pytest.mark.parametrize("f32", [False, True])
def test_write4_extremes(f32):
    """Zeros of both signs, the smallest and the largest numbers, infinities,
    NaN: each block by itself."""
    d = 128
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, 2, d)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2, 0, :16], x[2, 0, 16:32] = 2.0 ** -133, 2.0 ** -20
    x[2, 1, :16] = -2.0 ** -12
    x[3] *= 1e38 / np.abs(x[3]).max()
    x[4, 0, 5], x[4, 1, 100] = np.inf, -np.inf
    x[5, 0, 3] = np.nan
    x[6, 1, 17:32] = np.inf
    x[7, 0] *= 2688
    t = cu(x, np.float32).to(torch.float32 if f32 else torch.bfloat16)
    k4, v4 = deft.alloc_kv4_pages(1, 2, d)
    deft.deft_qkv_write4(None, t, t, cu(np.arange(8)), k4, v4, v_scale=0.0625)
    for pool, g in ((k4, 1.0), (v4, 0.0625)):
        codes, scales = ref.pages(pool.cpu().numpy())
        want_c, want_s, nan = ref.quantise(f64(t.bfloat16()), g)
        got_c, got_s = codes[0].transpose(1, 0, 2)[:8], scales[0].transpose(1, 0, 2)[:8]
        assert (got_s == want_s).all()
        assert (got_c == want_c)[~np.repeat(nan, 16, -1)].all()
        kp, vp = deft.deft_kv_unpack4(k4, v4, cu([0]), k_scale=1.0, v_scale=0.0625)
        back = f64((kp if g == 1.0 else vp)[0].transpose(0, 1))[:8]
        assert np.isnan(back[5, 0, :16]).all() and np.isfinite(np.delete(back, 5, 0)).all() and np.isfinite(back[5, 0, 16:]).all()
        assert back[4, 0, 5] == 2688 * g and back[4, 1, 100] == -2688 * g


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [(1.0, 0.5), (0.37, 3.3)])
def test_unpack4_every_code(d, g):
    """All 256 scale bytes with all 16 codes, pages in any order, some listed
    twice, some outside the pool (left as they were)."""
    rng = np.random.default_rng(d)
    n, h = 40, 3
    pool = rng.integers(0, 256, (2, n, h, 9 * d), dtype=np.uint8)
    pool[0, 0, 0, 8 * d:8 * d + 64] = np.arange(64)
    every = np.resize(np.arange(256, dtype=np.uint8), (n, h, d))
    pool[0, ..., 8 * d:] = every
    ids = np.concatenate([rng.permutation(n), [3, 3, -1, n, 2 ** 31 - 1, -2 ** 31, 0]]).astype(np.int64)
    out = [torch.full((len(ids) + 2, h, 16, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k4, v4 = (torch.from_numpy(p).cuda() for p in pool)
    kp, vp = deft.deft_kv_unpack4(k4, v4, cu(ids), *out, k_scale=g[0], v_scale=g[1])
    ok = (ids >= 0) & (ids < n)
    for p, pages, x in zip(pool, (kp, vp), g):
        x32 = np.float32(x)
        exact = ref.values(*ref.pages(p), 1.0).astype(np.float32)      # exact in fp32
        want = ref.bf16((exact * x32).astype(np.float64))
        got = f64(pages)
        assert np.array_equal(got[:len(ids)][ok], want[ids[ok]], equal_nan=True)
        assert (got[:len(ids)][~ok] == 5).all() and (got[len(ids):] == 5).all()


def test_positions_outside_the_table():
    """NaN in the rotated elements of such a row, and nowhere else; in 4 bits
    in the blocks that hold them."""
    r = Rows(T=6, hq=2, hkv=2, d=64, rot=32, norm=True)
    pos = np.array([0, -1, 96, 97, 2 ** 31 - 1, -2 ** 31])
    r.position = pos
    r.kw["position"] = cu(pos)
    kp, vp = r.pools()
    q = f64(deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw))
    bad = np.array([1, 3, 4, 5])
    rows = np.arange(6)
    for got, want in ((q, r.expect(0)), (r.at(f64(kp), rows), r.expect(1))):
        assert np.isnan(got[bad][..., :32]).all()
        fine = np.isfinite(want[0])
        assert (np.isfinite(got) == fine).all()
        close(np.where(fine, got, 0), np.where(fine, want[0], 0), want[1])
    k4, v4 = r.pools4()
    deft.deft_qkv_write4(r.q, r.k, r.v, cu(r.slot), k4, v4, **r.kw)
    s = r.at(ref.pages(k4.cpu().numpy())[1], rows)
    assert (s[bad][..., :2] == 0x7F).all() and (s[bad][..., 2:] < 0x7F).all() and (s[[0, 2]] < 0x7F).all()


def test_in_place_queries_and_no_queries():
    r = Rows(T=50, hq=4, hkv=2, d=128, rot=128)
    kp, vp = r.pools()
    want = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw)
    q = r.q.contiguous()
    k2, v2 = r.pools()
    assert deft.deft_qkv_write(q, r.k, r.v, cu(r.slot), k2, v2, q_out=q, **r.kw) is q
    assert torch.equal(q, want) and torch.equal(kp, k2) and torch.equal(vp, v2)
    k3, v3 = r.pools()
    kw = {n: v for n, v in r.kw.items() if n != "q_norm"}
    assert deft.deft_qkv_write(None, r.k, r.v, cu(r.slot), k3, v3, **kw) is None
    assert torch.equal(kp, k3) and torch.equal(vp, v3)


def test_plain_rows_are_kv_writes():
    """Without norm and rotation the call is deft_kv_write, bit for bit."""
    for f32 in (False, True):
        r = Rows(T=70, hq=3, hkv=3, d=64, f32=f32, norm=False, skip=(4,))
        a, b = r.pools(), r.pools()
        q = deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), *a)
        deft.deft_kv_write(r.k, r.v, cu(r.slot), *b)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(q, r.q.to(torch.bfloat16))


def test_no_tokens_and_no_pages():
    r = Rows(T=1, hq=2, hkv=1, d=64)
    kp, vp = r.pools()
    q = deft.deft_qkv_write(r.q[:0], r.k[:0], r.v[:0], cu([]), kp, vp, **r.kw)
    assert q.shape == (0, 2, 64) and (kp == 7).all()
    k4, v4 = r.pools4()
    assert deft.deft_kv_unpack4(k4, v4, cu([]))[0].shape == (0, 1, 16, 64)


def test_binding_refusals():
    r = Rows(T=4, hq=2, hkv=1, d=64, rot=64)
    kp, vp = r.pools()
    k4, v4 = r.pools4()
    slot = cu(r.slot)
    q, k, v, kw = r.q, r.k, r.v, r.kw
    for call in (
            lambda: deft.deft_qkv_write(q, k, v.float(), slot, kp, vp), lambda: deft.deft_qkv_write(q.float(), k, v, slot, kp, vp),
            lambda: deft.deft_qkv_write(q, k, v, slot[:3], kp, vp), lambda: deft.deft_qkv_write(q, k, v, slot.long(), kp, vp),
            lambda: deft.deft_qkv_write(q, k, v, slot, kp.float(), vp.float()), lambda: deft.deft_qkv_write(q, k, v, slot, kp[:, :, :8], vp[:, :, :8]),
            lambda: deft.deft_qkv_write(q[:3], k, v, slot, kp, vp), lambda: deft.deft_qkv_write(None, k, v, slot, kp, vp, q_norm=r.w[0]),
            lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, q_norm=r.w[0].float()), lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, q_norm=r.w[0][:32]),
            lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, cos_sin=kw["cos_sin"]), lambda: deft.deft_qkv_write(
                q, k, v, slot, kp, vp, cos_sin=kw["cos_sin"].double(), position=kw["position"]),
            lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, cos_sin=kw["cos_sin"], position=kw["position"][:2]),
            lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, q_out=torch.empty_like(q)[:3]), lambda: deft.deft_qkv_write(q, k, v, slot.cpu(), kp, vp),
            lambda: deft.deft_qkv_write4(q, k, v, slot, kp, vp), lambda: deft.deft_qkv_write4(q, k, v, slot, k4[:, :, :-1], v4[:, :, :-1]),
            lambda: deft.deft_qkv_write4(q, k, v, slot, k4.repeat(1, 2, 1), v4.repeat(1, 2, 1)),
            lambda: deft.deft_kv_unpack4(k4, v4[:1], slot), lambda: deft.deft_kv_unpack4(k4, v4, slot, kp[:1], vp[:1]),
            lambda: deft.deft_kv_unpack4(k4, v4, slot, kp), lambda: deft.deft_kv_unpack4(k4, v4, slot.float())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: deft.deft_qkv_write4(q, k, v, slot, k4, v4, k_scale=0.0), lambda: deft.deft_kv_unpack4(k4, v4, slot, v_scale=math.inf),
                 lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, q_norm=r.w[0], eps=-1.0),
                 lambda: deft.deft_qkv_write(q, k, v, slot, kp, vp, cos_sin=kw["cos_sin"][:, :24].contiguous(), position=kw["position"])):
        with pytest.raises(deft.DeftError):
            call()
    assert (kp == 7).all() and (k4 == 0xA5).all()


def test_slots_outside_the_pool():
    r = Rows(T=8, hq=1, hkv=2, d=64)
    slot = r.slot.copy()
    slot[:6] = [-1, r.pages * 16, 2 ** 31 - 1, -2 ** 31, -16, r.pages * 16 + 5]
    for pools, call in ((r.pools(), deft.deft_qkv_write), (r.pools4(), deft.deft_qkv_write4)):
        before = [p.clone() for p in pools]
        call(r.q[:6], r.k[:6], r.v[:6], cu(slot[:6]), *pools, **r.kw)
        assert all(torch.equal(a, b) for a, b in zip(pools, before))


def test_rows_behind_4gb():
    """Slots whose bytes lie past 32-bit offsets."""
    d, h = 128, 8
    pages = (1 << 33) // (h * 16 * d * 2) + 8     # 8 GB a pool
    r = Rows(T=4, hq=2, hkv=h, d=d, rot=128)
    kp, vp = (torch.empty((pages, h, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    r.slot = np.array([5, (pages // 2) * 16 + 3, (pages - 1) * 16 + 15, (pages - 1) * 16], dtype=np.int32)
    deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), kp, vp, **r.kw)
    want, slack = r.expect(1)
    for t, s in enumerate(r.slot.tolist()):
        close(f64(kp[s // 16, :, s % 16]), want[t], slack[t])
    del kp, vp
    pages = (1 << 33) // (h * 9 * d) + 8
    k4, v4 = (torch.empty((pages, h, 9 * d), dtype=torch.uint8, device="cuda") for _ in "kv")
    r.slot[1:] = [(pages // 2) * 16 + 3, (pages - 1) * 16 + 15, (pages - 1) * 16]
    deft.deft_qkv_write4(r.q, r.k, r.v, cu(r.slot), k4, v4, **r.kw)
    ids = r.slot // 16
    kp, vp = deft.deft_kv_unpack4(k4, v4, cu(ids))
    for t, s in enumerate(r.slot.tolist()):
        c, sc, _ = ref.quantise(f64(r.v[t]), 1.0)
        assert (f64(vp[t, :, s % 16]) == ref.values(c, sc, 1.0)).all()


def test_pools_that_start_at_any_16_bytes():
    r = Rows(T=20, hq=2, hkv=2, d=64, rot=64)
    a = r.pools4()
    q = deft.deft_qkv_write4(r.q, r.k, r.v, cu(r.slot), *a, **r.kw)
    b = [torch.empty(p.numel() + 16, dtype=torch.uint8, device="cuda")[16:].view(p.shape).fill_(0xA5) for p in a]
    q2 = deft.deft_qkv_write4(r.q, r.k, r.v, cu(r.slot), *b, **r.kw)
    assert torch.equal(q, q2) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids = cu(np.arange(r.pages))
    assert torch.equal(deft.deft_kv_unpack4(*a, ids)[0], deft.deft_kv_unpack4(*b, ids)[0])
    n = r.pages * 2 * 16 * 64
    out = [torch.empty(n + 8, dtype=torch.bfloat16, device="cuda")[8:].view(r.pages, 2, 16, 64) for _ in "kv"]
    with pytest.raises(deft.DeftError):      # 32-byte stores
        deft.deft_kv_unpack4(*a, ids, *out)
    deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), *out, **r.kw)
    c = r.pools()
    deft.deft_qkv_write(r.q, r.k, r.v, cu(r.slot), *c, **r.kw)
    kept = np.arange(r.T)
    assert (r.at(f64(out[0]), kept) == r.at(f64(c[0]), kept)).all() and (r.at(f64(out[1]), kept) == r.at(f64(c[1]), kept)).all()


def test_stream_and_graph():
    """On a stream of its own, allocating its output there, and captured."""
    r = Rows(T=64, hq=8, hkv=2, d=128, rot=128)
    a, b = r.pools4(), r.pools4()
    slot, ids = cu(r.slot), cu(np.arange(r.pages))
    want = deft.deft_qkv_write4(r.q, r.k, r.v, slot, *a, **r.kw)
    kp, vp = deft.deft_kv_unpack4(*a, ids)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q = deft.deft_qkv_write4(r.q, r.k, r.v, slot, *b, stream=st, **r.kw)
    k2, v2 = deft.deft_kv_unpack4(*b, ids, stream=st)
    st.synchronize()
    assert torch.equal(q, want) and torch.equal(a[0], b[0]) and torch.equal(kp, k2) and torch.equal(vp, v2)
    c = r.pools4()
    q3 = torch.empty_like(want)
    out = [torch.zeros_like(kp), torch.zeros_like(vp)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        deft.deft_qkv_write4(r.q, r.k, r.v, slot, *c, q_out=q3, **r.kw)
        deft.deft_kv_unpack4(*c, ids, *out)
    for _ in range(2):
        for x in (*c, *out):
            x.fill_(0xA5)
        q3.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q3, want) and torch.equal(c[0], a[0]) and torch.equal(out[1], vp)
