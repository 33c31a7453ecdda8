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
