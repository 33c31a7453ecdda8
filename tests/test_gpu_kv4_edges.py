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
