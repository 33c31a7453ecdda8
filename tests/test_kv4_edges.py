"""The calls around the 4-bit cache at their edges, as far as no GPU is needed:
empty batches, argument ranges, the arithmetic of the format."""
import ctypes

import pytest

import shared_prefix_kv_deft_gb300 as deft
from shared_prefix_kv_deft_gb300 import build as deft_build

A = 1 << 20     # a 16-byte aligned address that no call reaches
EINVAL, EUNSUPPORTED, ESTATE = -1, -5, -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    deft_build.build()
    deft.load()


@pytest.mark.parametrize("tokens,status", [(0, 0), (3, EINVAL)])
@pytest.mark.parametrize("four", [False, True])
def test_no_tokens_need_no_positions(tokens, status, four):
    """An empty batch's tensors have no address, its positions' among them."""
    turn = deft.QkTurn(None, None, 1e-6, 16, 0, 9, A, None)
    args = [A, 2 * A, 3 * A, 0, 256, 128, 128, A, tokens, ctypes.byref(turn), 7 * A, 4 * A, 5 * A]
    tail = [4, 4, 2, 64, 16, None]
    lib = deft.load()
    assert (lib.deft_qkv_write4(*args, 1.0, 1.0, *tail) if four else lib.deft_qkv_write(*args, *tail)) == status
