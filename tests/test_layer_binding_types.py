"""The few-token operators' binding refuses tensors whose elements are not of
the size that the call reads or writes, by name (ValueError), instead of taking
their bytes for something else.  CPU tensors that say they are CUDA tensors reach
every check; nothing is launched."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


class _OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)


def _t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


BF16, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def _layer_kw(fmt="none"):
    T, H, I, E, k = 3, 256, 128, 4, 2
    kw = dict(x=_t(BF16, T, H), topk_ids=_t(I32, T, k), router_weights=_t(F32, T, k), out=_t(BF16, T, H),
              shared_out=_t(BF16, T, H), residual=_t(BF16, T, H), status=_t(I32, 1), workspace=_t(U8, 4096))
    if fmt == "none":
        return dict(kw, w13=_t(BF16, E, 2 * I, H), w2=_t(BF16, E, H, I))
    kw.update(w_format=fmt, w13=_t(U8, E, 2 * I, H // 2), w2=_t(U8, E, H, I // 2))
    if fmt == "nvfp4":
        kw.update(w13_scales=_t(U8, E, 2 * I, H // 16), w2_scales=_t(U8, E, H, I // 16), w13_global=_t(F32, E),
                  w2_global=_t(F32, E))
    else:
        kw.update(group_size=64, w13_scales=_t(BF16, E, 2 * I, H // 64), w2_scales=_t(BF16, E, H, I // 64),
                  w13_zeros=_t(U8, E, 2 * I, H // 64), w2_zeros=_t(U8, E, H, I // 64))
    return kw


def _refused(name, fn, *a, **kw):
    with pytest.raises(ValueError) as e:
        fn(*a, **kw)
    assert name in str(e.value) and "byte" in str(e.value), str(e.value)


WIDE = {1: torch.int32, 2: torch.float32, 4: torch.int64}


@pytest.mark.parametrize("fmt", ["none", "nvfp4", "int4"])
def test_layer_refuses_elements_of_another_size(fmt):
    kw = _layer_kw(fmt)
    args = nqg.layer_args(**kw)
    assert (args.T, args.H, args.I, args.E, args.top_k) == (3, 256, 128, 4, 2)
    for name, t in kw.items():
        if name in ("workspace", "x") or not isinstance(t, torch.Tensor):
            continue
        wide = _t(WIDE[t.element_size()], *t.shape)  # as many elements, more bytes
        _refused(name, nqg.layer_args, **dict(kw, **{name: wide}))


def test_layer_refuses_codes_packed_in_wider_words():
    kw = _layer_kw("int4")
    # eight codes to an int32: the same bytes, but a quarter of the columns
    kw["w2"] = _t(I32, 4, 256, 16)
    _refused("w2", nqg.layer_args, **kw)


@pytest.mark.parametrize("weight_dtype,dtype", [("fp32", torch.float64), ("bf16", torch.float32), ("fp16", torch.float32)])
def test_router_weights_of_another_size(weight_dtype, dtype):
    _refused("router_weights", nqg.layer_args, **dict(_layer_kw(), router_weights=_t(dtype, 3, 2),
                                                      weight_dtype=weight_dtype))
    _refused("router_weights", nqg.moe_select_experts, _t(F32, 3, 8), _t(I32, 3, 2), _t(dtype, 3, 2),
             weight_dtype=weight_dtype, stream=0)


def test_select_refuses_64_bit_ids():
    # half of an int64 tensor would be written
    _refused("topk_ids", nqg.moe_select_experts, _t(F32, 3, 8), _t(torch.int64, 3, 2), _t(F32, 3, 2), stream=0)


def test_linear_refuses_elements_of_another_size():
    x, out = _t(BF16, 2, 128), _t(BF16, 2, 16)
    w, s, z = _t(U8, 16, 64), _t(BF16, 16, 2), _t(U8, 16, 2)
    kw = dict(w_format="int4", group_size=64)
    assert nqg.linear_w4_args(x, w, s, out, zeros=z, **kw).K == 128
    _refused("w", nqg.linear_w4_args, x, _t(I32, 16, 64), s, out, **kw)
    _refused("w_scales", nqg.linear_w4_args, x, w, _t(F32, 16, 2), out, **kw)
    _refused("zeros", nqg.linear_w4_args, x, w, s, out, zeros=_t(I32, 16, 2), **kw)
    _refused("w_scales", nqg.linear_w4_args, x, w, _t(F32, 16, 8), out)
