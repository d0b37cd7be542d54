"""The few-token products at sizes that take several panels, several 16-row
tiles to a slot and several passes, as real layers do, with copies of scales by
tensor and by hand, and with fewer tokens to a part than an expert has.

On 152 SMs a CTA of the second kernel has one tile up to H = 2432, two up to
4864, three up to 7296 and a second pass beyond; the streaming linear has a
second pass from N = 9729 on.  Rows of scales are copied by tensor copies where
they are multiples of 16 bytes."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

from test_gpu_layer import Problem, _check_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group,zeros", [("none", 0, False), ("nvfp4", 16, False), ("int4", 64, False),
                                             ("int4", 128, True)])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 7168, 128, 3, 2), (4, 7168, 128, 4, 2), (2, 128, 8192, 2, 1),
                                       (5, 256, 7168, 2, 2), (3, 2560, 128, 3, 2), (9, 5120, 128, 2, 2),
                                       (2, 7424, 128, 2, 2), (12, 16384, 128, 3, 2)])
def test_layer_panels_tiles_and_passes(T, H, I, E, k, fmt, group, zeros, io):
    p = Problem(T, H, I, E, k, fmt, group, zeros, io)
    p.check()
    assert p.status == 0


# rows that end inside a panel, and scales that lanes copy, in several tiles and passes
@pytest.mark.parametrize("T,H,I,fmt,group,zeros", [
    (3, 7184, 48, "nvfp4", 16, False), (2, 5136, 80, "nvfp4", 16, False), (10, 2576, 1408, "nvfp4", 16, False),
    (2, 7312, 4112, "nvfp4", 16, False), (3, 7040, 192, "int4", 64, True), (2, 2496, 64, "int4", 64, False),
    (9, 5184, 320, "int4", 64, True), (1, 7360, 1344, "int4", 64, True), (4, 5120, 768, "int4", 128, True),
    (2, 7304, 72, "none", 0, False), (9, 2440, 1000, "none", 0, False), (17, 4888, 520, "none", 0, False)])
def test_layer_rows_that_end_inside_a_panel(T, H, I, fmt, group, zeros):
    for io in ("bf16", "fp16"):
        p = Problem(T, H, I, 3, 2, fmt, group, zeros, io)
        p.check("gelu_tanh")
        assert p.status == 0


@pytest.mark.parametrize("group", [128, 512, 1024])
@pytest.mark.parametrize("H,I", [(1024, 1024), (5120, 1024), (1024, 7168)])
def test_layer_int4_groups(H, I, group):
    for zeros in (False, True):
        Problem(3, H, I, 2, 2, "int4", group, zeros).check()


@pytest.mark.parametrize("fmt,group,zeros", [("none", 0, False), ("nvfp4", 16, False), ("int4", 64, True)])
@pytest.mark.parametrize("H", [12288, 16384, 32768])
def test_layer_parts_that_shared_memory_makes_smaller(H, fmt, group, zeros):
    for T in (8, 11):
        p = Problem(T, H, 64, 2, 1, fmt, group, zeros)
        p.ids[:] = 1
        p.check()
        assert p.status == 0


@pytest.mark.parametrize("fmt,group,zeros,io", [("nvfp4", 16, False, "fp16"), ("nvfp4", 16, False, "bf16"),
                                                ("int4", 64, True, "bf16"), ("int4", 128, False, "fp16")])
@pytest.mark.parametrize("M,N,K", [(1, 9745, 256), (3, 12301, 384), (8, 20000, 256), (12, 9729, 512), (20, 12301, 640),
                                   (40, 19999, 256), (64, 9745, 1024), (2, 65535, 128)])
def test_linear_second_pass(M, N, K, fmt, group, zeros, io):
    _check_linear(M, N, K, fmt, group, zeros, io)
