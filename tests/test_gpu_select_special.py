"""Expert selection where logits are infinite, NaN of either sign, the type's
lowest value or all closed, for every logit type and on each side of the sizes
at which another kernel takes over (E = 256: registers sorted or not; E = 1024:
a CTA a token; 4096 tokens: 32-bit logits sorted)."""
import math

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _layer_ref as ref
from test_gpu_layer import DEV, DT, _check_select, _gen, _select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def _special(E, dt, seed=2):
    """Ten rows, one for each thing that a row can hold."""
    inf, low = math.inf, torch.finfo(DT[dt]).min
    x = torch.randn((10, E), generator=_gen(seed)).to(DT[dt])
    bits = torch.int32 if dt == "fp32" else torch.int16
    quiet = {"fp32": 0x7FC00000, "bf16": 0x7FC0, "fp16": 0x7E00}[dt]
    least = {"fp32": 0x7F800001, "bf16": 0x7F81, "fp16": 0x7C01}[dt]  # next to the infinity
    sign = -(1 << (31 if dt == "fp32" else 15))
    x[0] = -inf                       # nothing open
    x[1].view(bits)[:] = quiet        # NaNs of both signs, nothing open
    x[1].view(bits)[::2] = quiet + sign
    x[2, 3:] = -inf                   # three open, six asked for
    x[3].view(bits)[::3] = least + sign
    x[3].view(bits)[1::3] = least
    x[4, E // 2] = inf                # takes the softmax
    x[5, [E // 4, E - 1]] = inf       # share it
    x[6] = low                        # the lowest value is not closed
    x[7, 1:] = -inf
    x[7, E - 2] = inf                 # two open, one of them infinite
    x[8] = -inf
    x[8, E - 1] = inf                 # +inf alone
    x[9] = low
    x[9, 2::2].view(bits)[:] = quiet + sign
    return x


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [12, 33, 64, 128, 256, 257, 512, 1024, 1025, 3000])
def test_select_special_values(E, dt):
    x = _special(E, dt)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check_select(x, 6, dt, scoring, renorm, 1.0)


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
def test_select_special_values_in_a_large_batch(dt):
    x, k = _special(200, dt), 7
    T = 5000
    ids, w = _select(x.repeat(T // 10, 1).to(DEV), k, dt)
    want_ids, want_w = ref.select(x, k, "softmax", True, 1.0)
    assert torch.equal(ids, want_ids.repeat(T // 10, 1))
    # exponentials of arguments below 10 in magnitude, a sum of 7 and a division in fp32
    assert (w.double() - want_w.repeat(T // 10, 1)).abs().le(40 * 2.0 ** -24 * want_w.repeat(T // 10, 1)).all()


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
def test_select_renormalised_sigmoid_far_below_zero(dt):
    """Ratios of sigmoids hold down to the smallest normal float, wherever the largest logit lies."""
    for most in (5.0, 0.0, -3.0, -16.0, -18.0, -59.0, -61.0, -200.0):
        down = torch.tensor([0.0, -1.0, -20.0, -45.0, -70.0, -80.0, -86.0])
        x = (most + down).expand(3, 7).contiguous()
        for renorm in (True, False):
            _check_select(x, 7, dt, "sigmoid", renorm, 1.0)
    x = torch.randn((400, 5), generator=_gen(8)) * 60
    _check_select(x, 4, dt, "sigmoid", True, 2.5)


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
def test_select_sigmoid_of_equal_lowest_values(dt):
    x = torch.full((2, 40), torch.finfo(DT[dt]).min, dtype=DT[dt])
    _check_select(x, 8, dt, "sigmoid", True, 1.0)
