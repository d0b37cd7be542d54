"""Waits that run out in the block's products: the first CTA's copies stop after
a few slots.  The call ends within a few seconds, the status says why, results
of the first pair from that tile on are NaN, everything else is as it was, and the
context stays usable."""
import time

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

from test_gpu_block import DEV, dev_offsets, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def stalled(slots, call):
    t0 = time.monotonic()
    try:
        nqg.moe_debug_stall(slots)
        call()
        torch.cuda.synchronize()
    finally:
        nqg.moe_debug_stall(-1)
    assert time.monotonic() - t0 < 30


@pytest.mark.parametrize("slots", [0, 3, 12])  # in the first tile or the second, or a later one
@pytest.mark.parametrize("what", ["linear", "gated", "input", "weight"])
def test_copies_that_stop(what, slots):
    bounds, rows, K, N = [0, 100, 900, 1000], 1000, 520, 8192
    g = gen(slots)
    x, w, dy = normal(g, rows, K).to(DEV), normal(g, 3, N, K, std=K ** -0.5).to(DEV), normal(g, rows, N).to(DEV)
    off, status = dev_offsets(bounds), torch.zeros(1, dtype=torch.int32, device=DEV)
    shape = {"linear": (rows, N), "gated": (rows, N // 2), "input": (rows, K), "weight": (3, N, K)}[what]
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)

    def call():
        kw = dict(offsets=off, status=status)
        if what == "linear":
            nqg.moe_grouped_linear(x, w, out, **kw)
        elif what == "gated":
            nqg.moe_gated_linear(x, w, out, **kw)
        elif what == "input":
            nqg.moe_grouped_linear_backward(dy, w=w, d_x=out, **kw)
        else:
            nqg.moe_grouped_linear_backward(dy, x=x, d_w=out, **kw)

    call()
    good = out.clone()
    assert bool(good.isfinite().all()) and int(status) == 0
    stalled(slots, call)
    assert int(status) == nqg.MOE_ERR_DEVICE_TIMEOUT
    late = out.isnan()
    # the first pair has the first tile of each round of tiles
    assert 0 < float(late.double().mean()) <= 0.5
    assert torch.equal(out[~late], good[~late])
    status.zero_()
    call()
    assert torch.equal(out, good) and int(status) == 0


@pytest.mark.parametrize("slots", [0, 2])
@pytest.mark.parametrize("rows,K,N", [(20, 4096, 256), (300, 4096, 1024)])
def test_copies_that_stop_in_a_shared_tile(rows, K, N, slots):
    """The pairs that share the tile make it NaN; other tiles are as they were."""
    g = gen(rows)
    x, w = normal(g, rows, K).to(DEV), normal(g, 1, N, K, std=K ** -0.5).to(DEV)
    out, status = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda: nqg.moe_grouped_linear(x, w, out, status=status)  # noqa: E731
    call()
    good = out.clone()
    assert bool(good.isfinite().all())
    stalled(slots, call)
    assert int(status) == nqg.MOE_ERR_DEVICE_TIMEOUT
    late = out.isnan()
    assert bool(late[:20, :256].all()) and bool((late.sum() <= 256 * 128))
    assert torch.equal(out[~late], good[~late])
    status.zero_()
    call()
    assert torch.equal(out, good) and int(status) == 0


@pytest.mark.parametrize("slots", [0, 1, 3])
@pytest.mark.parametrize("H", [96, 4096, 16384])
def test_norm_rows_that_stop(slots, H):
    """Rows of the first CTA's first group from that one on are NaN, and so are the sums over tokens that they are part of."""
    T = 12000 if H == 96 else 3000
    g = gen(H)
    y, r, d = (normal(g, T, H).to(DEV) for _ in range(3))
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    out = [torch.empty_like(y) for _ in range(4)]
    sums = [torch.empty(H, device=DEV) for _ in range(2)]
    ws = torch.empty(nqg.moe_block_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)

    def forward():
        nqg.moe_block_norm(y, r, post_gamma=gamma, pre_gamma=gamma, residual_out=out[0], norm_out=out[1])

    def backward():
        nqg.moe_block_norm_backward(y, r, post_gamma=gamma, pre_gamma=gamma, d_residual_out=d, d_norm_out=d, d_y=out[2], d_residual=out[3],
                                    d_post_gamma=sums[0], d_pre_gamma=sums[1], workspace=ws)

    for call, results in ((forward, out[:2]), (backward, out[2:])):
        if call is backward and H > 8192:
            continue  # rows this wide are not copied ahead there
        call()
        good = [t.clone() for t in results]
        assert all(bool(t.isfinite().all()) for t in good)
        stalled(slots, call)
        for t, was in zip(results, good):
            late = t.isnan().all(1)
            assert 0 < int(late.sum()) <= T // 152 + 1
            assert torch.equal(t[~late], was[~late])
        if call is backward:
            assert all(bool(s.isnan().all()) for s in sums)
        call()
        assert all(torch.equal(a, b) for a, b in zip(results, good))
