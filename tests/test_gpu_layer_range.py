"""NVFP4 products of bf16 rows at the ends of the range: rows and global scales
for which factors or products leave fp32's normal range, and elements far below
the largest of their strip.

Beside the error of the sums (the bound of ``_layer_ref.linear``) the operator
states what is lost: with few rows and much K an element of x is off by at most
2^-39 of the largest of its 256, or by 2^-150 max(g, 1) if that is more; in all
other cases a product is off by at most 2^-123 / g."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _layer_ref as ref
from test_gpu_layer import _gen, _linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def _weights(gen, N, K, g):
    W = ref.Weights(gen, (), N, K, "nvfp4")
    W.value = W.value * W.glob.double() / g
    W.glob = torch.tensor([g], dtype=torch.float64)
    return W


def _bound(x, W, g, resident):
    M, K = x.shape
    want, tol = ref.linear(x, W.value, "bf16")
    if resident:
        strips = x.double().abs().view(M, -1, 256).amax(2, keepdim=True) * 2.0 ** -39
        off = strips.clamp(min=2.0 ** -150 * max(g, 1.0)).expand(M, K // 256, 256).reshape(M, K)
        return want, tol + off @ W.value.abs().t()
    return want, tol + K * 2.0 ** -123 / g


# g: a float as the call takes it
@pytest.mark.parametrize("size,g", [(2.0 ** -120, 1.0), (2.0 ** -120, 2.0 ** -10), (2.0 ** -8, 1.9375 * 2.0 ** 126),
                                    (1.0, 1.9375 * 2.0 ** 127), (2.0 ** -60, 1.25 * 2.0 ** 70),
                                    (2.0 ** 100, 1.5 * 2.0 ** 110), (2.0 ** -30, 2.0 ** -40)])
@pytest.mark.parametrize("M,N,K", [(1, 40, 4096), (2, 4100, 4096), (3, 20, 512), (20, 24, 1024), (40, 24, 1024)])
def test_linear_small_rows_and_large_scales(M, N, K, size, g):
    gen = _gen(M + N)
    W = _weights(gen, N, K, g)
    x = (torch.randn((M, K), generator=gen) * size).to(torch.bfloat16)
    got = _linear(x, W, "bf16")
    want, tol = _bound(x, W, g, resident=K >= 4096)
    assert want.abs().max() > 64 * tol.max()  # the bound is far below the results
    assert (got.double() - want).abs().le(tol).all()


@pytest.mark.parametrize("below", [29, 36, 38, 39, 40, 45])
def test_linear_elements_far_below_the_largest(below):
    N, K = 24, 4096
    gen = _gen(below)
    W = _weights(gen, N, K, 1.0)
    x = (torch.ones((1, K)) * 2.0 ** -below).to(torch.bfloat16)
    x[0, ::2] *= 1.5
    x[0, ::256] = 1.0                  # the largest of each strip meets a zero
    codes = W.codes & 0x77             # and all other codes are positive
    codes[:, ::128] &= 0xF0
    W.codes = codes
    W.value = ref.E2M1[ref.unpack(codes)] * ref.e4m3(W.scales).repeat_interleave(16, -1)
    got = _linear(x, W, "bf16")
    want, tol = _bound(x, W, 1.0, resident=True)
    assert (got.double() - want).abs().le(tol).all()
    if below <= 29:                    # exact so far: the sums' error alone
        assert (got.double() - want).abs().le(ref.linear(x, W.value, "bf16")[1]).all()
