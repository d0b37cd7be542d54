"""The gated product's gradients where a gate is so large that its square leaves
fp32: both activations are straight there, so their slopes are 1 and 0."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


@pytest.mark.parametrize("rows", [1, 200])  # dg and du held as sums of two, or rounded once
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("io", ["bf16", "fp16"])
def test_slopes_of_large_gates(io, kind, rows):
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    big = [200.0, 4096.0, 60000.0] if io == "fp16" else [200.0, 1e9, 1.8e19, 1.9e19, 1e25, 1e30, 2.0 ** 126, torch.finfo(dt).max]
    g = torch.tensor([s * v for v in big for s in (1, -1)] + [0.0] * 16).to(dt)[:16]
    I, H = 16, 8
    gate_up = torch.zeros((rows, 2 * I), dtype=dt, device=DEV)
    gate_up[0, :I], gate_up[0, I:] = g.to(DEV), 1
    d = torch.zeros((rows, I), dtype=dt, device=DEV)
    d[0] = 0.5
    x = torch.ones((rows, H), dtype=dt, device=DEV)
    dw = torch.empty((1, 2 * I, H), dtype=torch.float32, device=DEV)
    ws = torch.empty(nqg.moe_gated_linear_backward_workspace_size(rows, I), dtype=torch.uint8, device=DEV)
    nqg.moe_gated_linear_backward(d, gate_up, x=x, d_w13=dw, workspace=ws, activation=kind, io_dtype=io, grad_dtype="fp32")
    # one row with values: its dg and du, exact here (a half is a power of two, and act(g) is g or 0)
    slope = torch.where(g > 0, 1.0, torch.where(g < 0, 0.0, 0.5))
    want = torch.cat((0.5 * slope, 0.5 * g.float().clamp(min=0)))
    assert torch.equal(dw[0].cpu(), want[:, None].expand(-1, H)), dw[0, :, 0]
