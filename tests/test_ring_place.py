"""A warp that fills the ring of the block's products waits, before its CTA
leaves, for every slot that it filled to be handed back: an arrival from the
pair's other CTA must not find the shared memory gone.  Followed on the host
for every number of fills, those of short contractions (fewer than there are
slots) among them."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "norm_quant_gb300", "csrc")


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = tmp_path_factory.mktemp("ring") / "libring.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(so),
                    os.path.join(HERE, "cuda", "ring_place_check.cpp")], check=True)
    return ctypes.CDLL(str(so)).arrivals_left


def test_no_arrival_is_left_behind(check):
    assert [check(used) for used in range(40)] == [0] * 40
