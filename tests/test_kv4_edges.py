"""The calls around the 4-bit cache at their edges, as far as no GPU is needed:
empty batches, argument ranges, the arithmetic of the format."""
import contextlib
import ctypes
import subprocess
from fractions import Fraction

import pytest
import torch

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


RING = r"""
#include <cstdio>
#include <vector>

#include "kv4_internal.h"

// Barriers as the GPU's: one arrival a phase, and a wait for a parity is
// answered when the phase before the present one had it.
struct Ring {
    std::vector<int> phase;                 // completed, by stage
    std::vector<std::vector<int>> flying;   // copies on their way, by stage
    int asked = 0, vain = 0;
    explicit Ring(int stages) : phase(stages), flying(stages) {}
    void issue(int j) { flying[j % phase.size()].push_back(j); }
    void land(int s)
    {
        phase[s]++;
        flying[s].clear();
    }
    // A wait that lets the stage's copy land, if the parity asked for is that copy's.
    bool operator()(int s, unsigned parity)
    {
        asked++;
        if (((phase[s] & 1) ^ 1) == (int)parity && phase[s] > 0)
            return true;
        if (flying[s].empty() || (phase[s] & 1) != (int)parity) {
            vain++;
            return false;
        }
        land(s);
        return true;
    }
};

int main()
{
    int bad = 0, runs = 0;
    for (int stages = 1; stages <= 4; ++stages)
        for (int mine = 1; mine <= 13; ++mine)
            for (int failed = 0; failed < mine; ++failed) {
                Ring r(stages);
                auto wait = [&](int s, unsigned p) { return r(s, p); };
                int issued = 0;
                while (issued < mine && issued < stages)
                    r.issue(issued++);
                for (int i = 0; i < failed; ++i) {
                    bad += !deft::ring_wait(i, stages, wait);
                    if (issued < mine)
                        r.issue(issued++);
                }
                r.asked = 0;
                deft::ring_drain(failed, issued, stages, wait);
                for (auto &f : r.flying)
                    bad += !f.empty();
                bad += r.vain != 0 || r.asked != issued - failed;
                ++runs;
            }
    std::printf("%d %d\n", runs, bad);
    return bad != 0;
}
"""


def test_a_failed_wait_leaves_no_copy_behind(tmp_path):
    """Whichever copy of whichever ring does not land in time: the drain waits
    for every copy that is still on its way, and for nothing else."""
    src = tmp_path / "ring.cpp"
    src.write_text(RING)
    exe = tmp_path / "ring"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{deft_build.CSRC}", f"-I{deft_build.INCLUDE}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == [str(4 * 13 * 14 // 2), "0"]


@pytest.mark.parametrize("pages,heads,status", [((1 << 31) - 1, 2, ESTATE), (1 << 28, 16, ESTATE), ((1 << 28) + 1, 16, EUNSUPPORTED),
                                                ((1 << 31) - 1, 4, EUNSUPPORTED), ((1 << 31) - 1, 1 << 20, EUNSUPPORTED)])
def test_pages_of_heads_are_numbered_in_32_bits(pages, heads, status):
    """Of a plan that has not been uploaded: nothing reaches a GPU."""
    plan = deft.Plan([-1, 0, 0], [100, 5, 7], [1, 2], 256, 2, naive=False)
    rc = deft.load().deft_tree_attn4(A, 2 * A, 3 * A, 1.0, 1.0, A, A, pages, 2 * heads, heads, 128, 16, 0.1, plan.handle, 4 * A, 0, 5 * A, 6 * A, 1 << 30, None)
    assert rc == status


def test_alloc_kv4_pages_refuses_other_heads():
    assert [p.shape for p in deft.alloc_kv4_pages(3, 2, 64, "cpu")] == [(3, 2, 576)] * 2
    for d in (0, -64, 32, 96, 256):
        with pytest.raises(ValueError):
            deft.alloc_kv4_pages(3, 2, d, "cpu")


def rounded(x: Fraction) -> Fraction:
    """x > 0 to 24 significant bits, halfway to even."""
    e = x.numerator.bit_length() - x.denominator.bit_length() - 24
    unit = Fraction(2) ** (e + (x / Fraction(2) ** e >= 1 << 24))
    return round(x / unit) * unit       # (Fraction's round is to even)


def test_quotients_are_the_correctly_rounded_ones():
    """The append's quotient (the product with the reciprocal, and one step on
    the exact residual) gives the code of the correctly rounded x / sg for
    every bf16 x and every fp32 sg.  Both are within two units in the last
    place of x / sg, so they can only lie on two sides of a border t (or one
    on it) where sg is within a few units of x / t: all of those are tried,
    for all 128 significands of x and all seven borders.  Powers of two change
    nothing (the residual is far from fp32's least numbers)."""
    borders = [Fraction(b) / 4 for b in (1, 3, 5, 7, 10, 14, 20)]

    def code(y):        # halfway to the even code
        return sum(y > t if i % 2 == 0 else y >= t for i, t in enumerate(borders))

    assert [code(t) for t in borders] == [0, 2, 2, 4, 4, 6, 6]
    off = changed = 0
    for m in range(128):
        x = 1 + Fraction(m, 128)
        for t in borders:
            near = rounded(x / t)
            unit = Fraction(2) ** (near.numerator.bit_length() - near.denominator.bit_length() - 25)
            for u in range(-24, 25):
                sg = rounded(near + u * unit)
                r = rounded(1 / sg)
                y0 = rounded(x * r)
                left = y0 * sg - x
                step = rounded(abs(left)) * r if left else Fraction(0)
                y = rounded(y0 - step if left > 0 else y0 + step)
                want = rounded(x / sg)
                off += code(y) != code(want)
                changed += code(y0) != code(want)
    assert off == 0
    assert changed > 0      # (the product alone would not do)


@pytest.mark.parametrize("call", ["deft_qkv_write", "deft_qkv_write4", "deft_kv_unpack4", "deft_tree_attn4"])
@pytest.mark.parametrize("stream", [0, 0x77])
def test_outputs_come_from_the_launch_streams_memory(monkeypatch, call, stream):
    """Every call that allocates its outputs does so inside
    _allocating_for(its stream)."""
    class Allocated(Exception):
        pass

    inside = []

    @contextlib.contextmanager
    def allocating_for(st):
        inside.append(st)
        yield
        inside.pop()

    def empty(*a, **kw):
        raise Allocated(list(inside))

    rows, pages = torch.zeros((2, 1, 64), dtype=torch.bfloat16), torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    four, index = torch.zeros((1, 1, 576), dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    plan = deft.Plan([-1], [5], [0, 0], 256, 1, naive=False)
    args = {"deft_qkv_write": (rows, rows, rows, index, pages, pages), "deft_qkv_write4": (rows, rows, rows, index, four, four),
            "deft_kv_unpack4": (four, four, index), "deft_tree_attn4": (rows, four, four, index, index, plan)}[call]
    monkeypatch.setattr(deft, "_allocating_for", allocating_for)
    monkeypatch.setattr(torch, "empty", empty)
    with pytest.raises(Allocated) as e:
        getattr(deft, call)(*args, stream=stream)
    assert e.value.args[0] == [stream]
