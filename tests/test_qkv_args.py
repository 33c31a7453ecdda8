"""Argument checks of the append and unpack calls, and the tests' own form of
the 4-bit format (no GPU)."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref
import shared_prefix_kv_deft_gb300 as deft
from shared_prefix_kv_deft_gb300 import build as deft_build

A = 1 << 20     # a 16-byte aligned address that no call reaches
EINVAL, EUNSUPPORTED = -1, -5


@pytest.fixture(scope="module", autouse=True)
def _built():
    deft_build.build()
    deft.load()


def qkv_args(**kw):
    turn = dict(q_norm=None, k_norm=None, eps=1e-6, rot_dim=0, interleaved=0, num_positions=0, cos_sin=None, position=None)
    turn.update({n: kw.pop(n) for n in list(kw) if n in turn})
    d = dict(q=A, k=2 * A, v=3 * A, in_dtype=0, qs=256, ks=128, vs=128, slot=A, num_tokens=3, turn=ctypes.byref(deft.QkTurn(**turn)), q_out=7 * A,
             kp=4 * A, vp=5 * A, num_pages=4, hq=4, hkv=2, head_dim=64, page_size=16, stream=None)
    d.update(kw)
    return list(d.values())


REFUSED = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(q=None), EINVAL), (dict(q_out=None), EINVAL), (dict(slot=None), EINVAL),
    (dict(kp=None), EINVAL), (dict(vp=4 * A), EINVAL), (dict(num_tokens=-1), EINVAL), (dict(num_pages=0), EINVAL), (dict(hkv=0), EINVAL),
    (dict(hq=-1), EINVAL), (dict(in_dtype=2), EINVAL), (dict(q=A + 8), EINVAL), (dict(k=A + 8), EINVAL), (dict(q_out=A + 2), EINVAL),
    (dict(kp=A + 8), EINVAL), (dict(qs=248), EINVAL), (dict(ks=120), EINVAL), (dict(vs=132), EINVAL), (dict(in_dtype=1, qs=258), EINVAL),
    (dict(rot_dim=16), EINVAL), (dict(rot_dim=80, cos_sin=A, position=A, num_positions=9), EINVAL), (dict(rot_dim=-16), EINVAL),
    (dict(rot_dim=16, cos_sin=A, position=None, num_positions=9), EINVAL), (dict(rot_dim=16, cos_sin=A + 4, position=A, num_positions=9), EINVAL),
    (dict(rot_dim=16, cos_sin=A, position=A, num_positions=0), EINVAL), (dict(rot_dim=16, cos_sin=A, position=A, num_positions=9, interleaved=2), EINVAL),
    (dict(rot_dim=24, cos_sin=A, position=A, num_positions=9), EUNSUPPORTED), (dict(q_norm=A, eps=-1.0), EINVAL),
    (dict(k_norm=A, eps=float("nan")), EINVAL), (dict(k_norm=A + 2), EINVAL), (dict(head_dim=32), EUNSUPPORTED), (dict(page_size=64), EUNSUPPORTED),
    (dict(num_pages=1 << 27), EUNSUPPORTED), (dict(q_out=A, in_dtype=1), EINVAL), (dict(q_out=A, qs=512), EINVAL), (dict(num_tokens=0), 0),
    (dict(num_tokens=0, q=None, k=None, v=None, slot=None, q_out=None), 0), (dict(num_tokens=1 << 30, hq=4, hkv=2, turn=None, head_dim=128, qs=512,
                                                                                  ks=256, vs=256), EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_qkv_write_argument_checks(kw, status):
    assert deft.load().deft_qkv_write(*qkv_args(**dict(kw))) == status


@pytest.mark.parametrize("kw,status", REFUSED + [
    (dict(kg=0.0), EINVAL), (dict(vg=-1.0), EINVAL), (dict(kg=float("nan")), EINVAL), (dict(vg=float("inf")), EINVAL), (dict(kg=2.0 ** -61), EINVAL)])
def test_qkv_write4_argument_checks(kw, status):
    kw = dict(kw)
    g = [kw.pop("kg", 1.0), kw.pop("vg", 1.0)]
    a = qkv_args(**kw)
    assert deft.load().deft_qkv_write4(*a[:13], *g, *a[13:]) == status


def unpack_args(**kw):
    d = dict(k4=A, v4=2 * A, kg=1.0, vg=1.0, num_pages=4, page_id=A, listed=2, kp=3 * A, vp=4 * A, hkv=2, head_dim=64, page_size=16, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(k4=None), EINVAL), (dict(v4=None), EINVAL), (dict(page_id=None), EINVAL), (dict(kp=None), EINVAL), (dict(vp=3 * A), EINVAL),
    (dict(kp=A), EINVAL), (dict(vp=2 * A), EINVAL), (dict(kp=3 * A + 16), EINVAL), (dict(k4=A + 8), EINVAL), (dict(num_pages=0), EINVAL), (dict(listed=-1), EINVAL),
    (dict(hkv=0), EINVAL), (dict(kg=0.0), EINVAL), (dict(vg=float("nan")), EINVAL), (dict(head_dim=96), EUNSUPPORTED),
    (dict(page_size=32), EUNSUPPORTED), (dict(listed=0), 0), (dict(hkv=1 << 19), EINVAL)])
def test_unpack4_argument_checks(kw, status):
    assert deft.load().deft_kv_unpack4(*unpack_args(**kw)) == status


def test_page_bytes():
    assert [deft.kv4_page_bytes(d) for d in (64, 128, 96, 0, -1)] == [576, 1152, 0, 0, 0]


def test_the_tests_own_format():
    """Each code's value rounds to itself, halfway values to the even code."""
    for grid in (ref.E2M1, ref.E4M3):
        assert (ref.nearest(grid, grid) == np.arange(len(grid))).all()
        mid = (grid[1:] + grid[:-1]) / 2
        code = ref.nearest(mid, grid)
        assert (code % 2 == 0).all() and (np.abs(code - np.arange(len(mid)) - 0.5) == 0.5).all()
        assert (ref.nearest(mid * (1 + 2.0 ** -30), grid) == np.arange(1, len(grid))).all()
    x = ref.bf16(np.random.default_rng(0).standard_normal((64, 128)))
    code, s, _ = ref.quantise(x, 1.0)
    y = ref.values(code, s, 1.0)
    # a step of the largest codes is 2 s, half of it an element's error at most;
    # s is within 2^-4 of amax / 6 (the largest code's overflow included)
    assert (np.abs(y - x) <= np.repeat(ref.E4M3[s], 16, -1) * (1 + 6 * 2.0 ** -4)).all()


def attn4_args(of, **kw):
    d = dict(q=A, kp=2 * A, vp=3 * A, kg=1.0, vg=1.0, off=A, ids=A, num_pages=9, hq=4, hkv=2, head_dim=64, page_size=16, scale=0.1, plan=of.handle,
             out=4 * A, out_dtype=0, lse=5 * A, ws=6 * A, ws_bytes=1 << 30, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(kp=None), EINVAL), (dict(vp=None), EINVAL), (dict(off=None), EINVAL), (dict(ids=None), EINVAL), (dict(out=None), EINVAL),
    (dict(lse=None), EINVAL), (dict(plan=None), EINVAL), (dict(kg=0.0), EINVAL), (dict(vg=float("nan")), EINVAL), (dict(kg=2.0 ** 61), EINVAL),
    (dict(vg=-1.0), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(num_pages=0), EINVAL), (dict(hq=5), EINVAL), (dict(hkv=0), EINVAL),
    (dict(q=A + 8), EINVAL), (dict(kp=A + 8), EINVAL), (dict(out=4 * A + 8), EINVAL), (dict(out_dtype=7), EINVAL), (dict(head_dim=80), EUNSUPPORTED),
    (dict(page_size=32), EUNSUPPORTED), (dict(hq=8), -8), (dict(), -8)])
def test_tree_attn4_argument_checks(kw, status):
    """Of a plan that has not been uploaded: nothing reaches a GPU."""
    plan = deft.Plan([-1, 0, 0], [100, 5, 7], [1, 2], 256, 2, naive=False)
    assert deft.load().deft_tree_attn4(*attn4_args(plan, **kw)) == status
