"""Waits that run out part of the way through the few-token products: a ring
whose filling stops after a few slots, inside a row of panels, with slots
filled by tensor copies and by lanes.  The consumers that give up hand no slot
back, the call ends within a few seconds, what depends on the missing weights
is NaN, everything else is as it was, and the context stays usable."""
import time

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _layer_ref as ref
from test_gpu_layer import Problem, _gen, _linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def _stalled(slots, call):
    t0 = time.monotonic()
    try:
        nqg.moe_debug_stall(slots)
        got = call()
    finally:
        nqg.moe_debug_stall(-1)
    assert time.monotonic() - t0 < 20  # 2 s for each wait that runs out after another
    return got


# resident kernel; streamed with tensor copies, with lanes' copies, and with several passes
@pytest.mark.parametrize("slots", [1, 3])
@pytest.mark.parametrize("M,N,K,fmt,group", [(1, 8000, 16384, "nvfp4", 16), (5, 8000, 16384, "int4", 128),
                                             (3, 8000, 7184, "nvfp4", 16), (40, 12000, 4096, "int4", 64)])
def test_linear_filling_that_stops(M, N, K, fmt, group, slots):
    gen = _gen(slots)
    W = ref.Weights(gen, (), N, K, fmt, group, False)
    x = torch.randn((M, K), generator=gen).to(torch.bfloat16)
    good = _linear(x, W, "bf16")
    got = _stalled(slots, lambda: _linear(x, W, "bf16"))
    late = got.isnan().all(0)
    assert 0 < int(late.sum()) <= -(-N // 16 // 152) * 16
    assert torch.equal(got[:, ~late], good[:, ~late])
    assert torch.equal(_linear(x, W, "bf16"), good)


# the first block makes eight values of one expert, from 4 panels and more
@pytest.mark.parametrize("slots", [1, 3])
@pytest.mark.parametrize("H,fmt,group", [(32768, "none", 0), (32752, "nvfp4", 16), (32768, "int4", 64)])
def test_layer_filling_that_stops(H, fmt, group, slots):
    p = Problem(4, H, 128, 2, 1, fmt, group)
    p.ids[:] = torch.tensor([[0], [1], [0], [1]])
    good = p.run()
    got = _stalled(slots, p.run)
    assert p.status == nqg.MOE_ERR_DEVICE_TIMEOUT
    # the first part is expert 0 with token 0, and with token 2 where the columns of both fit
    assert got[0].isnan().all()
    assert got[2].isnan().all() or torch.equal(got[2], good[2])
    assert torch.equal(got[[1, 3]], good[[1, 3]])
    assert torch.equal(p.run(), good) and p.status == 0
