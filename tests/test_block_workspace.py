"""A workspace of the gated gradients that is large enough for some rows is large
enough for fewer: a program makes one for its largest batch."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


@pytest.mark.parametrize("I", [8, 16, 24, 32, 40, 56, 64, 72, 104, 128, 200, 456, 512, 968, 1408, 1992, 4032, 4040, 4048, 8192])
def test_size_never_falls_as_rows_grow(I):
    sizes = [nqg.moe_gated_linear_backward_workspace_size(rows, I) for rows in range(600)]
    assert sizes == sorted(sizes)
    assert all(size >= 4 * rows * I for rows, size in enumerate(sizes))


@pytest.mark.gpu
@pytest.mark.parametrize("I", [8, 24, 72, 200])
def test_one_workspace_for_all_batches(I):
    """A workspace for 100 rows, for fewer of them in turn: the results that each call has with one of its own."""
    most, H = 100, 64
    g = torch.Generator().manual_seed(I)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to("cuda")  # noqa: E731
    d, gate_up, x, w = normal(most, I), normal(most, 2 * I), normal(most, H), normal(1, 2 * I, H)
    size = nqg.moe_gated_linear_backward_workspace_size
    shared = torch.empty(size(most, I), dtype=torch.uint8, device="cuda")
    for rows in (100, 65, 64, 51, 33, 32, 20, 7, 1):
        got = []
        for ws in (shared, torch.empty(size(rows, I), dtype=torch.uint8, device="cuda")):
            dx, dw = torch.empty_like(x[:rows]), torch.empty_like(w)
            nqg.moe_gated_linear_backward(d[:rows], gate_up[:rows], x=x[:rows], w13=w, d_x=dx, d_w13=dw, workspace=ws)
            got.append((dx, dw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), rows
