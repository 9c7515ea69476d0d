"""How the layer operators lay calls out, on the host: the sizes of tests/_layer_shapes.py take the kernels they are
there for, and every kernel of the products is taken by one of the GPU tests' sizes."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests._layer_shapes import CES, FFNS, SCANS

HERE = os.path.dirname(os.path.abspath(__file__))
CXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(CXX is None, reason="no host C++ compiler")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "driver")
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", os.path.join(HERE, "layer_plan_driver.cpp"), "-o", exe], check=True)

    def ask(*words):
        text = " ".join(str(w) for w in words)
        return subprocess.run([exe], input=text + "\n", capture_output=True, text=True, check=True).stdout.strip()

    return ask


@pytest.mark.parametrize("lens,D,packed,es,want", SCANS)
def test_scans(plan, lens, D, packed, es, want):
    T = sum(lens) if packed else lens[0]
    assert plan("scan", T, D, len(lens), int(packed), es) == "%d %d %d" % want


def test_scans_without_sequences(plan):
    for T in (0, 1, 256, 257, 100000):
        assert plan("scan", T, 20, 0, 0, 4) == "0 0 2"


@pytest.mark.parametrize("M,D,F,es,want", FFNS)
def test_feed_forward(plan, M, D, F, es, want):
    assert plan("ffn", M, D, F, es) == want


@pytest.mark.parametrize("N,D,V,es,want", CES)
def test_cross_entropy(plan, N, D, V, es, want):
    assert plan("ce", N, D, V, es) == want


def test_the_large_tile_is_taken_by_every_product():
    for k in range(3):
        assert any(f[4].split()[k].startswith("256") for f in FFNS)
    for k in (0, 2, 3, 4):
        assert any(c[4].split()[k].startswith("256") for c in CES)
