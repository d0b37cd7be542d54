"""The few-token operators' host side without a GPU: argument layouts,
workspace sizes, the refusals of the C ABI (none of these calls reaches CUDA),
and the binding's size checks."""
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
    assert L.moe_linear_w4_args_size() == C.sizeof(nqg.MoeLinearW4Args) == 88
    assert L.moe_layer_args_size() == C.sizeof(nqg.MoeLayerArgs) == 192


@pytest.mark.parametrize("T,k,I,want", [(1, 8, 2048, 32768), (0, 1, 8, 0), (3, 1, 8, 1536), (64, 32, 65536, 1 << 28)])
def test_workspace_size(L, T, k, I, want):
    assert nqg.moe_layer_workspace_size(T, k, I) == want


@pytest.mark.parametrize("T,k,I,want", [(-1, 1, 8, 1), (1, 0, 8, 1), (1, 1, 0, 1), (65, 1, 8, 2), (1, 33, 8, 2),
                                        (1, 1, 65544, 2)])
def test_workspace_size_refusals(L, T, k, I, want):
    n = C.c_size_t(0)
    assert L.moe_layer_workspace_size(T, k, I, C.byref(n)) == want
    assert L.moe_layer_workspace_size(1, 1, 8, None) == 1


def _select(L, **kw):
    a = dict(logits=0x1000, T=4, E=16, stride=16, dt=0, k=2, scoring=0, renorm=1, scale=1.0, ids=0x2000, w=0x3000,
             wd=0)
    a.update(kw)
    return L.moe_select_experts(a["logits"], a["T"], a["E"], a["stride"], a["dt"], a["k"], a["scoring"], a["renorm"],
                                a["scale"], a["ids"], a["w"], a["wd"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=17), 1), (dict(stride=15), 1), (dict(dt=3), 1),
    (dict(dt=-1), 1), (dict(wd=3), 1), (dict(scoring=2), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(E=8193, stride=8193), 2), (dict(E=64, stride=64, k=33), 2),
    (dict(T=1 << 40), 2), (dict(logits=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(logits=0x1002), 1),
    (dict(logits=0x1001, dt=1), 1), (dict(ids=0x2002), 1), (dict(w=0x3002), 1), (dict(w=0x3001, wd=2), 1),
    (dict(T=0), 0), (dict(T=0, logits=None, ids=None, w=None), 0)])
def test_select_refusals(L, kw, want):
    assert _select(L, **kw) == want


def _linear(**kw):
    a = dict(M=2, N=8, K=128, x=0x1000, x_stride=128, w=0x2000, w_scales=0x3000, w_zeros=None, global_scale=1.0,
             w_format=1, group_size=0, io_dtype=0, out=0x4000, out_stride=8)
    a.update(kw)
    return nqg.MoeLinearW4Args(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=24, x_stride=24), 1), (dict(w_format=0), 1),
    (dict(w_format=3), 1), (dict(io_dtype=2), 1), (dict(global_scale=0.0), 1), (dict(global_scale=-1.0), 1),
    (dict(global_scale=float("inf")), 1), (dict(global_scale=float("nan")), 1), (dict(w_zeros=0x5000), 1),
    (dict(w_format=2, group_size=32), 1), (dict(w_format=2, group_size=96), 1), (dict(w_format=2, group_size=0), 1),
    (dict(w_format=2, group_size=256), 1), (dict(M=65), 2), (dict(N=65537), 2), (dict(K=65552, x_stride=65552), 2),
    (dict(x=None), 1), (dict(w=None), 1), (dict(w_scales=None), 1), (dict(out=None), 1), (dict(x=0x1008), 1),
    (dict(w=0x2008), 1), (dict(out=0x4001), 1), (dict(w_format=2, group_size=64, w_scales=0x3001), 1),
    (dict(x_stride=120), 1), (dict(x_stride=132), 1), (dict(out_stride=7), 1),
    (dict(M=0), 0), (dict(M=0, x=None, w=None, out=None, w_scales=None), 0)])
def test_linear_refusals(L, kw, want):
    assert L.moe_linear_w4(C.byref(_linear(**kw)), None) == want


def test_null_arguments(L):
    assert L.moe_linear_w4(None, None) == 1 and L.moe_layer(None, None) == 1


def _layer(**kw):
    a = dict(T=2, H=128, I=64, E=4, top_k=2, x=0x1000, x_stride=128, topk_ids=0x2000, router_weights=0x3000,
             w13=0x4000, w2=0x5000, out=0x6000, workspace=0x7000, workspace_bytes=512)
    a.update(kw)
    return nqg.MoeLayerArgs(**a)


NV = dict(w_format=1, w13_scales=0x8000, w2_scales=0x9000)
I4 = dict(w_format=2, group_size=64, w13_scales=0x8000, w2_scales=0x9000)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(I=0), 1), (dict(E=0), 1), (dict(top_k=0), 1), (dict(H=124), 1),
    (dict(I=60), 1), (dict(w_format=3), 1), (dict(w_format=-1), 1), (dict(io_dtype=2), 1), (dict(weight_dtype=3), 1),
    (dict(activation=2), 1), (dict(T=65), 2), (dict(E=1025), 2), (dict(top_k=33), 2),
    (dict(H=65544, x_stride=65544), 2), (dict(I=65544), 2), (dict(x=None), 1), (dict(topk_ids=None), 1),
    (dict(router_weights=None), 1), (dict(w13=None), 1), (dict(w2=None), 1), (dict(out=None), 1),
    (dict(x=0x1008), 1), (dict(w13=0x4008), 1), (dict(w2=0x5008), 1), (dict(topk_ids=0x2002), 1),
    (dict(router_weights=0x3002), 1), (dict(router_weights=0x3001, weight_dtype=1), 1), (dict(out=0x6001), 1),
    (dict(shared_out=0xA001), 1), (dict(residual=0xA001), 1), (dict(status=0xA002), 1), (dict(x_stride=120), 1),
    (dict(x_stride=132), 1), (dict(workspace=None), 3), (dict(workspace_bytes=511), 3), (dict(workspace=0x7008), 1),
    (dict(w13_global=0xB000), 1), (dict(w13_zeros=0xB000), 1), (dict(NV, w13_scales=None), 1),
    (dict(NV, w2_scales=None), 1), (dict(NV, w2_zeros=0xB000), 1), (dict(NV, w2_global=0xB002), 1),
    (dict(NV, H=136, x_stride=136), 1), (dict(I4, group_size=48), 1), (dict(I4, group_size=128), 1),
    (dict(I4, w13_global=0xB000), 1), (dict(I4, w2_scales=0x9001), 1),
    (dict(T=0), 0), (dict(T=0, x=None, w13=None, w2=None, out=None, workspace=None), 0)])
def test_layer_refusals(L, kw, want):
    assert L.moe_layer(C.byref(_layer(**kw)), None) == want


# --------------------------------------------------- the binding's own checks

def _expect(what, fn, *a, **kw):
    with pytest.raises(ValueError) as e:
        fn(*a, **kw)
    assert what in str(e.value), str(e.value)


def test_binding_refuses_cpu_and_misshapen_tensors(L):
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    _expect("CUDA", nqg.linear_w4_args, h(2, 64), torch.zeros((8, 32), dtype=torch.uint8),
            torch.zeros((8, 4), dtype=torch.uint8), h(2, 8))
    kw = dict(topk_ids=torch.zeros((2, 2), dtype=torch.int32), router_weights=torch.zeros(2, 2), w13=h(4, 128, 64),
              w2=h(4, 64, 64), out=h(2, 64), workspace=torch.zeros(1024, dtype=torch.uint8))
    _expect("CUDA", nqg.layer_args, x=h(2, 64), **kw)
    _expect("w2 has rows", nqg.layer_args, x=h(2, 72), **kw)
    _expect("CUDA", nqg.moe_select_experts, torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int32),
            torch.zeros((2, 2)))
