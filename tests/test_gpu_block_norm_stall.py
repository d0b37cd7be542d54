"""Copies that stop in the norms' gradients without a second norm: what depends
on a row that never came is NaN, a token's gate gradient among it."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

from test_gpu_block import DEV, gen, normal
from test_gpu_block_stall import stalled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


@pytest.mark.parametrize("slots", [1])
@pytest.mark.parametrize("H", [96, 4096])
@pytest.mark.parametrize("post,pre,residual", [(False, False, True), (False, False, False), (True, False, True), (False, True, True),
                                               (True, True, False)])
def test_rows_that_stop(post, pre, residual, H, slots):
    T = 12000 if H == 96 else 3000
    g = gen(H + slots)
    y, r, d, dn = (normal(g, T, H).to(DEV) for _ in range(4))
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    gate = torch.rand(T, generator=g).to(DEV)
    d_y, d_gate = torch.empty_like(y), torch.empty(T, device=DEV)
    d_res = torch.empty_like(y) if residual else None

    def call():
        nqg.moe_block_norm_backward(y, r if residual else None, post_gamma=gamma if post else None, pre_gamma=gamma if pre else None,
                                    gate=gate, gate_kind="token", d_residual_out=d, d_norm_out=dn if pre else None, d_y=d_y,
                                    d_residual=d_res, d_gate=d_gate)

    call()
    outs = [t for t in (d_y, d_gate, d_res) if t is not None]
    good = [t.clone() for t in outs]
    assert all(bool(t.isfinite().all()) for t in good)
    stalled(slots, call)
    late = d_y.isnan().all(1)
    assert 0 < int(late.sum()) <= T // 152 + 1
    for t, was in zip(outs, good):
        assert bool(t[late].isnan().all()) and torch.equal(t[~late], was[~late])
    call()
    assert all(torch.equal(a, b) for a, b in zip(outs, good))
