"""How linear attention cuts sequences, on the host: what one workgroup may have to walk, whatever the lengths of packed sequences
are, and what is not worth a cut."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(CXX is None, reason="no host C++ compiler")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "driver")
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", os.path.join(HERE, "attn_plan_driver.cpp"), "-o", exe], check=True)

    def answer(T, nseq, units, packed, backward):
        out = subprocess.run([exe], input="plan %d %d %d %d %d\n" % (T, nseq, units, packed, backward), capture_output=True, text=True, check=True).stdout
        return [int(w) for w in out.split()]

    return answer


@pytest.mark.parametrize("units", [1, 8, 16, 100])
@pytest.mark.parametrize("nseq", [2, 10, 63, 64, 65, 300, 2000])
@pytest.mark.parametrize("T", [300, 2049, 20000, 131072])
def test_one_long_sequence_among_many(plan, T, nseq, units):
    """Nearly all packed tokens may be one sequence's: no workgroup walks more than its heads' share of the card, 2048 tokens, or
    4096 backwards, unless the sequences are shorter than a chunk in the mean."""
    share = -(-T * units // 512)
    for backward, most in ((0, 2048), (1, 4096)):
        seg, _, _ = plan(T, nseq, units, 1, backward)
        assert (seg or T) <= max(most, share + 63) or (not backward and T < 64 * nseq)


@pytest.mark.parametrize("T", [257, 1024, 4096])
@pytest.mark.parametrize("nseq,units", [(12, 16), (23, 16), (3, 64), (1, 380), (383, 1)])
def test_batches_that_fill_most_of_the_card_are_whole(plan, T, nseq, units):
    assert plan(T, nseq, units, 0, 0) == [0, 1, nseq] and plan(T, nseq, units, 0, 1) == [0, 1, nseq]


@pytest.mark.parametrize("backward,units", [(0, 8), (0, 128), (0, 191), (1, 8), (1, 64), (1, 95)])
def test_fewer_are_cut(plan, backward, units):
    seg, per, slots = plan(4096, 1, units, 0, backward)
    assert 0 < seg <= 2048 and per == slots >= 2


def test_backward_segments_end_where_sums_cancel(plan):
    for packed, nseq, units in ((0, 1, 96), (0, 3, 32), (1, 32, 32), (1, 5, 400)):
        assert plan(5000, nseq, units, packed, 1)[0] == 4096


def test_workgroups_are_numbered_in_31_bits(tmp_path):
    """At the largest calls that are taken, and any others, no launch has 2^31 workgroups; a little larger ones are refused."""
    exe = str(tmp_path / "driver")
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", os.path.join(HERE, "attn_launch_driver.cpp"), "-o", exe], check=True)
    r, cases = random.Random(5), []
    for _ in range(20000):
        packed, group, dk, dv = r.randint(0, 1), r.choice([1, 2, 3, 8]), r.choice([64, 128]), 32 * r.randint(1, 8)
        Hk = r.choice([1, 2, 5, 16, 64, 1000, 100000])
        Hv, T = Hk * group, int(2 ** r.uniform(0, 31)) - 1
        # sequences up to about what the rule leaves room for
        room = max(1, (2 ** 26 // Hv - (T // 256 + 1 if packed else 0)) // (1 if packed else 1 + T // 256 + 1))
        nseq = max(1, int(room * r.choice([1, 0.999, 0.5, 1e-3, 1e-6])))
        cases.append((1 if packed else nseq, T, nseq, packed, Hk, Hv, dk, dv))
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    out = [line.split() for line in subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()]
    taken = [int(most) for ok, most in out if ok == "1"]
    assert len(out) == len(cases) and len(taken) > 2000 and max(taken) > 2 ** 30 and max(taken) < 2 ** 31 - 4096
    assert any(ok == "0" for ok, _ in out)
