"""Which kernel the norms' calls of tens of thousands of tokens take, on the host."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests._qk_cases import LONG, MANY

HERE = os.path.dirname(os.path.abspath(__file__))
CXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(CXX is None, reason="no host C++ compiler")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "driver")
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", os.path.join(HERE, "qk_plan_driver.cpp"), "-o", exe], check=True)

    def answer(case):
        out = subprocess.run([exe], input=" ".join(map(str, case[:5])), capture_output=True, text=True, check=True).stdout
        return [int(w) for w in out.split()]

    return answer


@pytest.mark.parametrize("case", MANY)
def test_many_tokens_a_workgroup(plan, case):
    tokens, tiles, _, _, _ = plan(case)
    assert tokens == (8 if case[4] > 128 else 16)
    assert case == MANY[-1] or case[0] * case[1] % tokens and case[1] % tokens  # tiles over two batch rows, the last one part full


@pytest.mark.parametrize("case", LONG)
def test_more_steps_than_are_summed_in_32_bits(plan, case):
    """A backward workgroup's turns hold more than the 64 steps after which its sums go on in 64 bits, in every form."""
    tokens, tiles, steps, _, groups = plan(case)
    assert groups == 1024 and tiles * steps // groups > 64
    assert tokens == {8: 16, 136: 4, 40: 4, 64: 16, 256: 8}[case[4]]
