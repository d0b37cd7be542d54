"""A product whose one expert alone takes longer than the 2 s that a wait is
given: waits that begin long before their tile does are given the time of
the tiles in front of it."""
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


def test_few_rows_behind_an_expert_of_many():
    """600000 rows of one expert (2.4 to 2.9 s of matrix instructions in its weights' gradient) and 8 of another, whose only step
    reads beyond its rows."""
    rows, more, width = 600_000, 8, 65536
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 190 * 2 ** 30:
        pytest.skip("less than 190 GB of memory free")
    a = (1.0 + torch.arange(width) % 2).to(torch.bfloat16).to(DEV)
    b = (1.0 - 2.0 * (torch.arange(width) % 3 == 1)).to(torch.bfloat16).to(DEV)
    dy, x = (torch.empty((rows + more, width), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dy.copy_(a)
    x.copy_(b)
    off = torch.tensor([0, rows, rows + more], dtype=torch.int32, device=DEV)
    dw, status = torch.empty((2, width, width), dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    nqg.moe_grouped_linear_backward(dy, x=x, d_w=dw, offsets=off, status=status)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 2000, "not as long as meant"
    assert int(status) == 0
    # sums of ones and twos, exact in fp32: rows a b
    for e, n in enumerate((rows, more)):
        for at in range(0, width, 4096):
            want = (n * a[at:at + 4096].float()[:, None] * b.float()).to(torch.bfloat16)
            assert torch.equal(dw[e, at:at + 4096], want), (e, at)
    del dy, x, dw
    torch.cuda.empty_cache()
