"""The block operators' host side without a GPU: argument layouts, workspace
sizes, the refusals of the C ABI (none of these calls reaches CUDA), and the
binding's checks of shapes, types and places."""
import ctypes as C

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return nqg.lib()


def test_argument_layouts(L):
    sizes = {"moe_gated_linear": 104, "moe_gated_linear_backward": 144, "moe_grouped_linear": 80,
             "moe_grouped_linear_backward": 112, "moe_block_norm": 96, "moe_block_norm_backward": 152}
    for name, size in sizes.items():
        cls = nqg._BLOCK_ARGS[name]
        assert getattr(L, name + "_args_size")() == C.sizeof(cls) == nqg._PACK[name].size == size, name


def call(L, name, base, kw):
    args = nqg._BLOCK_ARGS[name](**{**base, **kw})
    return getattr(L, name)(C.byref(args), None)


SHARED = [(dict(rows=-1), 1), (dict(E=0), 1), (dict(io_dtype=2), 1), (dict(io_dtype=-1), 1), (dict(rows=(1 << 31) - (1 << 16)), 2),
          (dict(E=1025), 2), (dict(offsets=None), 1), (dict(offsets=0x1002), 1), (dict(status=0x1002), 1)]

GATED = dict(rows=4, H=64, I=32, E=2, offsets=0x1000, x=0x2000, x_stride=64, w13=0x3000, out=0x4000, out_stride=32)


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(H=0), 1), (dict(H=60), 1), (dict(I=0), 1), (dict(I=4), 1), (dict(H=65544, x_stride=65544), 2),
    (dict(I=65544, out_stride=65544), 2), (dict(activation=2), 1), (dict(activation=-1), 1), (dict(x=None), 1),
    (dict(w13=None), 1), (dict(out=None), 1), (dict(x=0x2008), 1), (dict(w13=0x3008), 1), (dict(out=0x4002), 1),
    (dict(x_stride=56), 1), (dict(x_stride=68), 1), (dict(out_stride=24), 1), (dict(out_stride=36), 1),
    (dict(gate_up=0x5000), 1), (dict(gate_up=0x5000, gate_up_stride=56), 1), (dict(gate_up=0x5008, gate_up_stride=64), 1),
    (dict(rows=0), 0), (dict(rows=0, x=None, w13=None, out=None, offsets=None), 0)])
def test_gated_linear_refusals(L, kw, want):
    assert call(L, "moe_gated_linear", GATED, kw) == want


# a stride that no tensor map takes (2^40 bytes and more), of every matrix of rows of the products
@pytest.mark.parametrize("name,fields", [
    ("moe_gated_linear", ["x", "out", "gate_up"]), ("moe_gated_linear_backward", ["x", "d_out", "gate_up", "d_x"]),
    ("moe_grouped_linear", ["x", "out"]), ("moe_grouped_linear_backward", ["x", "d_out", "d_x"])])
def test_strides_beyond_a_tensor_map(L, name, fields):
    base = {"moe_gated_linear": dict(GATED, gate_up=0x5000, gate_up_stride=64), "moe_gated_linear_backward": GATED_GRAD,
            "moe_grouped_linear": GROUPED, "moe_grouped_linear_backward": GROUPED_GRAD}[name]
    for field in fields:
        for stride in (1 << 39, (1 << 63) - 8):
            assert call(L, name, base, {f"{field}_stride": stride}) == 1, (field, stride)


GATED_GRAD = dict(rows=4, H=64, I=32, E=2, offsets=0x1000, d_out=0x2000, d_out_stride=32, gate_up=0x3000, gate_up_stride=64,
                  x=0x4000, x_stride=64, w13=0x5000, d_x=0x6000, d_x_stride=64, d_w13=0x7000, workspace=0x8000,
                  workspace_bytes=1024, grad_dtype=1)


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(H=60), 1), (dict(I=4), 1), (dict(activation=2), 1), (dict(grad_dtype=2), 1), (dict(grad_dtype=3), 1),
    (dict(io_dtype=1, grad_dtype=1), 1), (dict(d_out=None), 1), (dict(gate_up=None), 1), (dict(x=None), 1), (dict(w13=None), 1),
    (dict(d_x=None, d_w13=None), 1), (dict(d_x=0x6008), 1), (dict(d_w13=0x7008), 1), (dict(d_x_stride=56), 1),
    (dict(d_out_stride=24), 1), (dict(gate_up_stride=60), 1), (dict(x_stride=60), 1), (dict(workspace=None), 3),
    (dict(workspace_bytes=1023), 3), (dict(workspace=0x8008), 1), (dict(rows=0, d_w13=None), 0)])
def test_gated_linear_backward_refusals(L, kw, want):
    assert call(L, "moe_gated_linear_backward", GATED_GRAD, kw) == want


GROUPED = dict(rows=4, K=64, N=32, E=2, offsets=0x1000, x=0x2000, x_stride=64, w=0x3000, out=0x4000, out_stride=32)


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(K=60), 1), (dict(N=4), 1), (dict(K=65544, x_stride=65544), 2), (dict(N=65544, out_stride=65544), 2), (dict(x=None), 1),
    (dict(w=None), 1), (dict(out=None), 1), (dict(x=0x2008), 1), (dict(w=0x3008), 1), (dict(out=0x4008), 1), (dict(x_stride=56), 1),
    (dict(out_stride=24), 1), (dict(rows=0), 0)])
def test_grouped_linear_refusals(L, kw, want):
    assert call(L, "moe_grouped_linear", GROUPED, kw) == want


GROUPED_GRAD = dict(rows=4, K=64, N=32, E=2, offsets=0x1000, d_out=0x2000, d_out_stride=32, x=0x4000, x_stride=64, w=0x5000,
                    d_x=0x6000, d_x_stride=64, d_w=0x7000, grad_dtype=0)


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(K=60), 1), (dict(N=4), 1), (dict(grad_dtype=2), 1), (dict(d_out=None), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(d_x=None, d_w=None), 1), (dict(d_x=0x6008), 1), (dict(d_w=0x7008), 1), (dict(d_x_stride=60), 1),
    (dict(rows=0, d_w=None), 0)])
def test_grouped_linear_backward_refusals(L, kw, want):
    assert call(L, "moe_grouped_linear_backward", GROUPED_GRAD, kw) == want


NORM_SHARED = [(dict(T=-1), 1), (dict(H=0), 1), (dict(H=60), 1), (dict(H=16392), 2), (dict(T=1 << 31), 2), (dict(io_dtype=2), 1),
               (dict(y=None), 1), (dict(y=0x1008), 1), (dict(residual=0x2008), 1), (dict(post_gamma=0x3002), 1),
               (dict(pre_gamma=0x4002), 1), (dict(gate=0x5000), 1), (dict(gate_kind=1), 1), (dict(gate_kind=3, gate=0x5000), 1),
               (dict(gate_kind=-1, gate=0x5000), 1), (dict(gate_kind=1, gate=0x5008), 1), (dict(gate_kind=2, gate=0x5002), 1),
               (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(block_scale=float("nan")), 1),
               (dict(residual_scale=float("inf")), 1), (dict(weight_bias=float("nan")), 1)]
NORM = dict(T=4, H=64, y=0x1000, residual=0x2000, post_gamma=0x3000, pre_gamma=0x4000, block_scale=1.0, residual_scale=1.0,
            eps=1e-6, residual_out=0x6000, norm_out=0x7000)


@pytest.mark.parametrize("kw,want", NORM_SHARED + [
    (dict(residual_out=None, norm_out=None), 1), (dict(pre_gamma=None), 1), (dict(norm_out=0x6000), 1), (dict(residual_out=0x6008), 1),
    (dict(norm_out=0x7008), 1), (dict(T=0), 0), (dict(T=0, y=None, residual_out=None, norm_out=None), 0)])
def test_block_norm_refusals(L, kw, want):
    assert call(L, "moe_block_norm", NORM, kw) == want


NORM_GRAD = dict(T=4, H=64, y=0x1000, residual=0x2000, post_gamma=0x3000, pre_gamma=0x4000, block_scale=1.0, residual_scale=1.0,
                 eps=1e-6, d_residual_out=0x6000, d_norm_out=0x7000, d_y=0x8000, d_residual=0x9000, d_post_gamma=0xA000,
                 d_pre_gamma=0xB000, workspace=0xC000, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,want", NORM_SHARED + [
    (dict(d_residual_out=None, d_norm_out=None, d_pre_gamma=None), 1), (dict(pre_gamma=None), 1), (dict(d_norm_out=None), 1),
    (dict(post_gamma=None), 1), (dict(residual=None), 1), (dict(d_gate=0xD000), 1), (dict(gate=0x5000, gate_kind=1, d_gate=0xD004), 1),
    (dict(gate=0x5000, gate_kind=2, d_gate=0xD002), 1), (dict(d_residual=0x8000), 1), (dict(d_y=0x8008), 1),
    (dict(d_residual=0x9008), 1), (dict(d_post_gamma=0xA004), 1), (dict(d_pre_gamma=0xB004), 1), (dict(d_residual_out=0x6008), 1),
    (dict(d_norm_out=0x7008), 1), (dict(d_y=None, d_residual=None, d_post_gamma=None, d_pre_gamma=None), 1),
    (dict(workspace=None), 3), (dict(workspace_bytes=64), 3), (dict(workspace=0xC008), 1),
    (dict(T=0, d_post_gamma=None, d_pre_gamma=None), 0)])
def test_block_norm_backward_refusals(L, kw, want):
    assert call(L, "moe_block_norm_backward", NORM_GRAD, kw) == want


def test_null_arguments(L):
    for name in nqg._BLOCK_ARGS:
        assert getattr(L, name)(None, None) == 1, name


def test_workspace_sizes(L):
    assert nqg.moe_gated_linear_backward_workspace_size(0, 8) == 0
    assert nqg.moe_gated_linear_backward_workspace_size(100, 24) == 100 * 24 * 4
    # few values are held as sums of two, each part rounded up to 64 columns
    assert nqg.moe_gated_linear_backward_workspace_size(4, 32) == 4 * 2 * 64 * 2
    assert nqg.moe_gated_linear_backward_workspace_size(1, 4040) == 2 * 8128 * 2
    assert nqg.moe_gated_linear_backward_workspace_size(1, 4048) == 4048 * 4
    for rows in (1, 2, 16, 64, 65):
        sizes = [nqg.moe_gated_linear_backward_workspace_size(rows, i) for i in range(8, 8192, 8)]
        assert all(s <= 4 * rows * i + 65536 for s, i in zip(sizes, range(8, 8192, 8)))
    assert nqg.moe_gated_linear_backward_workspace_size(1 << 30, 65536) == 1 << 48
    n = C.c_size_t(0)
    for rows, inner, want in ((-1, 8, 1), (1, 0, 1), (1, 12, 1), (1, 65544, 2), (1 << 31, 8, 2)):
        assert L.moe_gated_linear_backward_workspace_size(rows, inner, C.byref(n)) == want
    assert L.moe_gated_linear_backward_workspace_size(1, 8, None) == 1
    assert nqg.moe_block_norm_backward_workspace_size(0, 64) == 0
    assert 0 < nqg.moe_block_norm_backward_workspace_size(1, 64) <= nqg.moe_block_norm_backward_workspace_size(1 << 20, 64) <= 12 * 64 * 1024
    for T, H, want in ((-1, 8, 1), (1, 0, 1), (1, 12, 1), (1, 16392, 2), (1 << 31, 8, 2)):
        assert L.moe_block_norm_backward_workspace_size(T, H, C.byref(n)) == want


# --------------------------------------------------- the binding's own checks


class _OnGpu(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor, so that it reaches every check; nothing is launched."""
    is_cuda = property(lambda self: True)


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def refused(what, fn, *a, **kw):
    with pytest.raises(ValueError) as e:
        fn(*a, stream=0, **kw)
    assert what in str(e.value), str(e.value)


F32, I32, I64 = torch.float32, torch.int32, torch.int64


def test_binding_of_the_products(L):
    x, w, out = t(5, 64), t(2, 32, 64), t(5, 32)
    off = t(3, dtype=I32)
    refused("CUDA", nqg.moe_grouped_linear, torch.zeros(5, 64, dtype=torch.bfloat16), w, out, offsets=off)
    refused("offsets", nqg.moe_grouped_linear, x, w, out, offsets=t(3, dtype=I64))
    refused("offsets", nqg.moe_grouped_linear, x, w, out, offsets=t(2, dtype=I32))
    refused("out", nqg.moe_grouped_linear, x, w, t(4, 32), offsets=off)
    refused("out", nqg.moe_grouped_linear, x, w, t(5, 40), offsets=off)
    refused("w is", nqg.moe_grouped_linear, x, t(2, 32, 72), out, offsets=off)
    refused("w is", nqg.moe_grouped_linear, x, t(32, 64), out, offsets=off)
    refused("w has 4-byte", nqg.moe_grouped_linear, x, t(2, 32, 64, dtype=F32), out, offsets=off)
    refused("x is", nqg.moe_grouped_linear, t(5, 64, dtype=F32), w, out, offsets=off)
    refused("x: the elements", nqg.moe_grouped_linear, t(64, 5).t(), w, out, offsets=off)
    refused("contiguous", nqg.moe_grouped_linear, x, t(2, 64, 32).transpose(1, 2), out, offsets=off)
    refused("status", nqg.moe_grouped_linear, x, w, out, offsets=off, status=t(1, dtype=I64))
    refused("out", nqg.moe_gated_linear, x, w, out, offsets=off)  # I is 16
    refused("as many of W3", nqg.moe_gated_linear, x, t(2, 33, 64), t(5, 16), offsets=off)
    refused("gate_up", nqg.moe_gated_linear, x, w, t(5, 16), gate_up=t(5, 16), offsets=off)


def test_binding_of_their_gradients(L):
    dy, x, w, dx, dw = t(5, 32), t(5, 64), t(2, 32, 64), t(5, 64), t(2, 32, 64)
    fn = nqg.moe_grouped_linear_backward
    refused("needs", fn, dy, x=x, d_x=dx)
    refused("needs", fn, dy, w=w, d_w=dw)
    refused("has to be given", fn, dy)
    refused("columns", fn, t(5, 40), w=w, d_x=dx)
    refused("x is", fn, dy, x=t(5, 72), w=w, d_w=dw)
    refused("d_x is", fn, dy, w=w, d_x=t(5, 72))
    refused("d_w is", fn, dy, x=x, w=w, d_w=t(1, 32, 64))
    refused("d_w has", fn, dy, x=x, w=w, d_w=dw, grad_dtype="fp32")
    refused("d_w has", fn, dy, x=x, w=w, d_w=t(2, 32, 64, dtype=F32))
    fn, d, gu, w13 = nqg.moe_gated_linear_backward, t(5, 16), t(5, 32), t(2, 32, 64)
    refused("needs", fn, d, gu, d_x=dx)
    refused("gate_up", fn, d, t(5, 16), w13=w13, d_x=dx)
    refused("rows an expert", fn, t(5, 24), t(5, 48), w13=w13, d_x=dx)
    refused("d_w13", fn, d, gu, x=x, d_w13=t(2, 32, 64, dtype=F32))


def test_binding_of_the_norms(L):
    y, gamma = t(3, 64), t(64)
    fn = nqg.moe_block_norm
    refused("residual has", fn, y, t(3, 64, dtype=F32), residual_out=y)
    refused("residual holds", fn, y, t(2, 64), residual_out=y)
    refused("post_gamma", fn, y, y, post_gamma=t(56), residual_out=y)
    refused("gate_kind", fn, y, y, gate=gamma, residual_out=y)
    refused("gate_kind", fn, y, y, gate_kind="token", residual_out=y)
    refused("gate has", fn, y, y, gate=gamma, gate_kind="token", residual_out=y)
    refused("gate holds", fn, y, y, gate=t(56), gate_kind="channel", residual_out=y)
    refused("norm_out", fn, y, y, pre_gamma=gamma, norm_out=t(2, 64))
    fn = nqg.moe_block_norm_backward
    refused("d_post_gamma has", fn, y, y, post_gamma=gamma, d_residual_out=y, d_post_gamma=gamma)
    refused("d_gate holds", fn, y, y, gate=t(3, dtype=F32), gate_kind="token", d_residual_out=y, d_gate=t(2, dtype=F32))
    refused("CUDA", fn, torch.zeros(3, 64, dtype=torch.bfloat16), d_residual_out=y, d_y=y)
