"""Weights' gradients of experts that end anywhere within a step of 64 rows, each
between neighbours whose rows are not finite: nothing of these is read into
them, whatever the number of rows, the widths and the form."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _block_ref as ref
from test_gpu_block import DEV, dev_offsets, gen, near, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(256, 256), (512, 128), (72, 136), (1288, 64), (8, 8)])  # in boxes of two chunks, one, or parts of one
def test_every_end_between_bad_neighbours(K, N, io, bad):
    counts = []
    for rest in range(1, 64):
        counts += [rest + 64 * (rest % 3), 1 + rest % 5]  # the rows that count, and a neighbour's
    bounds = [3]
    for c in counts:
        bounds.append(bounds[-1] + c)
    rows = bounds[-1] + 40
    g = gen(K + N)
    x, dy = normal(g, rows, K, io=io), normal(g, rows, N, io=io)
    good = torch.zeros(rows, dtype=torch.bool)
    for e in range(0, len(counts), 2):
        good[bounds[e]:bounds[e + 1]] = True
    xs, ds = x.clone(), dy.clone()
    xs[~good], ds[~good] = bad, bad
    dw = torch.full((len(counts), N, K), 13.0, device=DEV)
    nqg.moe_grouped_linear_backward(ds.to(DEV), x=xs.to(DEV), d_w=dw, offsets=dev_offsets(bounds), io_dtype=io, grad_dtype="fp32")
    want, bound = ref.weight_grad(dy.double(), torch.zeros(rows, N, dtype=torch.float64), x, bounds, io, "fp32")
    near(dw[::2], want[::2], bound[::2])
    assert not bool(dw[1::2].isfinite().any())


@pytest.mark.parametrize("first,rest", [(0, 1), (64, 17), (200, 63), (128, 48), (4000, 29), (4096, 3)])
def test_ends_of_one_expert_before_bad_rows(first, rest):
    """One expert whose rows end before the tensor's, with a contraction that pairs share where it is long."""
    rows, K, N = first + rest, 264, 520
    g = gen(rows)
    x, dy = normal(g, rows + 9, K), normal(g, rows + 9, N)
    xs, ds = x.clone(), dy.clone()
    xs[rows:], ds[rows:] = float("inf"), float("nan")
    dw = torch.full((1, N, K), 13.0, device=DEV)
    nqg.moe_grouped_linear_backward(ds.to(DEV), x=xs.to(DEV), d_w=dw, offsets=dev_offsets([0, rows]), grad_dtype="fp32")
    want, bound = ref.weight_grad(dy.double(), torch.zeros(rows + 9, N, dtype=torch.float64), x, [0, rows], "bf16", "fp32")
    near(dw, want, bound)


@pytest.mark.parametrize("I", [8, 40, 72])
def test_ends_of_held_sums(I):
    """The same with dg and du held as sums of two values: each of the last two steps ends there."""
    counts, H = [1, 2, 7, 3, 9, 1, 5], 72
    bounds = [0]
    for c in counts:
        bounds.append(bounds[-1] + c)
    rows = bounds[-1] + 2
    g = gen(I)
    x, gu, d = normal(g, rows, H), normal(g, rows, 2 * I), normal(g, rows, I)
    dgu, err = ref.gate_grad(d, gu, "silu", "bf16")
    want, bound = ref.weight_grad(dgu, err, x, bounds, "bf16", "fp32")
    xs, ds = x.clone(), d.clone()
    for e in range(1, len(counts), 2):
        xs[bounds[e]:bounds[e + 1]], ds[bounds[e]:bounds[e + 1]] = float("inf"), float("nan")
    xs[bounds[-1]:], ds[bounds[-1]:] = float("nan"), float("nan")
    dw = torch.full((len(counts), 2 * I, H), 13.0, device=DEV)
    ws = torch.full((nqg.moe_gated_linear_backward_workspace_size(rows, I),), 255, dtype=torch.uint8, device=DEV)
    nqg.moe_gated_linear_backward(ds.to(DEV), gu.to(DEV), x=xs.to(DEV), d_w13=dw, workspace=ws, offsets=dev_offsets(bounds),
                                  grad_dtype="fp32")
    near(dw[::2], want[::2], bound[::2])
    assert not bool(dw[1::2].isfinite().any())
