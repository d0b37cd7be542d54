"""The few-token operators on the GPU against 64-bit references: expert
selection, the 4-bit linear and the expert layer, at the sizes, masks, ids and
values where they can go wrong."""
import math
import os

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _canary(n, dtype, pad=512):
    buf = torch.full((n + 2 * pad,), -77, device=DEV, dtype=dtype)
    return buf, buf[pad:pad + n]


def _untouched(buf, view, pad=512):
    return bool((buf[:pad] == -77).all()) and bool((buf[pad + view.numel():] == -77).all())


# ------------------------------------------------------------------ selection

def _select(logits, k, logits_dtype, weight_dtype="fp32", **kw):
    T = logits.shape[0]
    ib, ids = _canary(T * k, torch.int32)
    wb, w = _canary(T * k, DT[weight_dtype])
    nqg.moe_select_experts(logits, ids.view(T, k), w.view(T, k), logits_dtype=logits_dtype,
                           weight_dtype=weight_dtype, **kw)
    torch.cuda.synchronize()
    assert _untouched(ib, ids) and _untouched(wb, w)
    return ids.view(T, k).cpu(), w.view(T, k).cpu()


def _check_select(logits, k, dt, scoring, renorm, scale, weight_dtype="fp32", stride=0):
    x = logits.to(DT[dt])
    T, E = x.shape
    wide = torch.full((T, E + stride), 9.0, dtype=DT[dt], device=DEV)
    wide[:, :E] = x.to(DEV)
    ids, w = _select(wide[:, :E], k, dt, weight_dtype, scoring=scoring, renormalize=renorm, scale=scale)
    want_ids, want_w = ref.select(x, k, scoring, renorm, scale)
    assert torch.equal(ids, want_ids)
    # exp, the sum over E and the divisions: a few fp32 roundings each, and one to the weight type; an exponential's
    # argument may be off by 2^-24 of the logits' span
    span = float(logits[torch.isfinite(logits)].abs().max()) * 2 if torch.isfinite(logits).any() else 0.0
    tol = (16 + math.log2(E + 1)) * 2.0 ** -24 + (min(span, 200.0) + 4) * 2.0 ** -24
    tol += {"fp32": 0, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[weight_dtype]
    floor = {"fp32": 2.0 ** -126, "bf16": 2.0 ** -126, "fp16": 2.0 ** -24}[weight_dtype]
    assert (w.double() - want_w).abs().le(tol * want_w.abs() + floor).all()


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 8, 8), (3, 33, 7), (64, 161, 6), (37, 300, 32),
                                   (2, 1024, 8), (130, 128, 2), (2, 1025, 9), (3, 8192, 32)])
def test_select_matches_definition(T, E, k, dt):
    logits = torch.randn((T, E), generator=_gen(T * E + k)) * 1.5
    for scoring, renorm, scale in (("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 1.0),
                                   ("sigmoid", False, 0.5)):
        _check_select(logits, k, dt, scoring, renorm, scale)


def test_select_ties_go_to_the_lower_index_and_zeros_are_equal():
    logits = torch.zeros((4, 70))
    logits[1, ::2] = -0.0
    logits[2] = torch.randint(0, 3, (70,), generator=_gen(1)).float()
    logits[3, 40:] = -1.0
    for dt in DT:
        _check_select(logits, 9, dt, "softmax", True, 1.0)


def test_select_closed_experts_infinities_and_nan():
    inf, nan = math.inf, math.nan
    logits = torch.randn((8, 40), generator=_gen(2))
    logits[0] = -inf                       # nothing open
    logits[1] = nan
    logits[2, 3:] = -inf                   # three open, six asked for
    logits[3, ::3] = nan
    logits[4, 7] = inf                     # takes the softmax
    logits[5, [9, 30]] = inf               # share it
    logits[6] = torch.finfo(torch.float32).min   # the lowest float is not closed
    logits[7, 1:] = nan
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check_select(logits, 6, "fp32", scoring, renorm, 1.0)


@pytest.mark.parametrize("wd", ["fp32", "bf16", "fp16"])
def test_select_strided_rows_and_weight_types(wd):
    _check_select(torch.randn((19, 50), generator=_gen(3)), 5, "bf16", "softmax", True, 1.0, wd, stride=13)


def test_select_many_tokens():
    T, E, k = 20000, 64, 4
    x = torch.randn((T, E), device=DEV)
    ids, w = _select(x, k, "fp32")
    top = x.topk(k, dim=1)  # no equal values among random floats of a row
    assert torch.equal(ids.long(), top.indices.cpu())
    assert torch.allclose(w, torch.softmax(top.values, 1).cpu(), rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
def test_select_large_batch_with_equal_values(dt):
    T, E, k = 5000, 200, 8
    x = torch.randint(0, 12, (T, E), generator=_gen(4)).float() - 6
    x[::7, ::3] = -math.inf
    ids, w = _select(x.to(DT[dt]).to(DEV), k, dt)
    top, want = torch.sort(x, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want[:, :k])
    assert torch.allclose(w, torch.softmax(top[:, :k], 1), rtol=1e-5, atol=0)


def test_select_empty_batch():
    nqg.moe_select_experts(torch.empty((0, 8), device=DEV), torch.empty((0, 2), device=DEV, dtype=torch.int32),
                           torch.empty((0, 2), device=DEV))


# --------------------------------------------------------------------- linear

FORMATS = [("nvfp4", 16, False), ("int4", 64, False), ("int4", 128, True)]


def _linear(x, W, io, stride=0, x_stride=0, **kw):
    M, K = x.shape
    N = W.codes.shape[0]
    xs = torch.full((M, K + x_stride), math.nan, dtype=ref.IO[io], device=DEV)
    xs[:, :K] = x.to(DEV)
    buf, out = _canary(M * (N + stride), ref.IO[io])
    view = out.view(M, N + stride)[:, :N]
    c = W.cuda("w")
    nqg.moe_linear_w4(xs[:, :K], c["w"], c["w_scales"], view, w_format=W.fmt, group_size=W.group,
                      zeros=c["w_zeros"], global_scale=float(W.glob[0]) if W.glob is not None else 1.0, io_dtype=io,
                      **kw)
    torch.cuda.synchronize()
    assert _untouched(buf, out)
    if stride:
        assert bool((out.view(M, N + stride)[:, N:] == -77).all())
    return view.cpu()


def _check_linear(M, N, K, fmt, group, zeros, io, **kw):
    gen = _gen(M * 7 + N * 3 + K)
    W = ref.Weights(gen, (), N, K, fmt, group, zeros, io)
    x = torch.randn((M, K), generator=gen).to(ref.IO[io])
    got = _linear(x, W, io, **kw)
    want, tol = ref.linear(x, W.value, io)
    assert (got.double() - want).abs().le(tol).all()


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 17, 1024), (2, 40, 7168), (7, 33, 896), (8, 128, 640),
                                   (9, 100, 2048), (16, 15, 384), (17, 65, 1152), (32, 50, 512), (33, 31, 256),
                                   (64, 77, 1408), (1, 700, 16384), (3, 2500, 256)])
def test_linear_matches_definition(M, N, K, fmt, group, zeros, io):
    _check_linear(M, N, K, fmt, group, zeros, io)


# bf16 and NVFP4 with a few rows and much k take a kernel of their own
@pytest.mark.parametrize("M,N,K", [(1, 1, 4096), (1, 33, 4112), (2, 4099, 4112), (3, 8193, 4096), (4, 12301, 4096),
                                   (1, 40, 32768), (2, 4100, 32752)])
def test_linear_few_rows_much_k(M, N, K):
    _check_linear(M, N, K, "nvfp4", 16, False, "bf16")


def test_linear_few_rows_much_k_non_finite_and_large():
    gen = _gen(11)
    W = ref.Weights(gen, (), 8200, 4096, "nvfp4")
    x = torch.randn((3, 4096), generator=gen).to(torch.bfloat16)
    x[0] *= 2.0 ** 100
    x[0, 5] = 2.0 ** 120
    x[2] *= 2.0 ** -100
    want, tol = ref.linear(x, W.value, "bf16")
    clean = _linear(x, W, "bf16")
    assert (clean.double() - want).abs().le(tol).all()
    x[1, 100] = math.nan
    x[2, 3] = math.inf
    W.scales[17, 5] = 0x7F
    got = _linear(x, W, "bf16")
    keep = [n for n in range(8200) if n != 17]
    assert torch.equal(got[0, keep], clean[0, keep]) and got[:, 17].isnan().all()
    assert got[1].isnan().all() and not got[2].isfinite().any()


@pytest.mark.parametrize("K,group", [(1280, 64), (1152, 64), (7168, 128), (1792, 128), (10240, 512), (16384, 1024)])
@pytest.mark.parametrize("M", [2, 12])
def test_linear_int4_panels_that_start_inside_a_scale_vector(M, K, group):
    for zeros in (False, True):
        _check_linear(M, 50, K, "int4", group, zeros, "bf16")
        _check_linear(M, 2500, K, "int4", group, zeros, "fp16")


@pytest.mark.parametrize("K", [16, 32, 48, 80, 1040, 2064])
def test_linear_nvfp4_rows_that_end_inside_a_step(K):
    for io in ("bf16", "fp16"):
        for M in (1, 9, 33):
            _check_linear(M, 35, K, "nvfp4", 16, False, io)


@pytest.mark.parametrize("group", [64, 256, 1024])
def test_linear_int4_group_sizes(group):
    _check_linear(3, 20, 2048, "int4", group, True, "fp16")


@pytest.mark.parametrize("M", [1, 5, 40])
def test_linear_strided_rows(M):
    _check_linear(M, 50, 256, "nvfp4", 16, False, "bf16", stride=7, x_stride=24)


@pytest.mark.parametrize("io", ["bf16", "fp16"])
def test_linear_nvfp4_every_code_and_scale_is_exact(io):
    # one-hot rows of x read the weights out one by one; global scale 1: the products are io numbers
    scales = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    N, K = len(scales), 32
    q = torch.arange(16).repeat(2)
    codes = (q[0::2] | (q[1::2] << 4)).to(torch.uint8).expand(N, K // 2).contiguous()
    W = ref.Weights(_gen(0), (), 1, 16, "nvfp4")
    W.codes, W.scales, W.glob = codes, scales.unsqueeze(1).expand(N, 2).contiguous(), torch.ones(1)
    want = ref.E2M1[ref.unpack(codes)] * ref.e4m3(W.scales).repeat_interleave(16, -1)
    got = _linear(torch.eye(K).to(ref.IO[io]), W, io)
    assert torch.equal(got.double(), want.t())


def test_linear_int4_every_code_and_zero_is_exact():
    N, K = 16, 64
    q = torch.arange(16).repeat(4)
    W = ref.Weights(_gen(0), (), N, K, "int4", 64, True)
    W.codes = (q[0::2] | (q[1::2] << 4)).to(torch.uint8).expand(N, K // 2).contiguous()
    W.scales = torch.full((N, 1), 0.25, dtype=torch.bfloat16)
    W.zeros = torch.arange(16, dtype=torch.uint8).view(N, 1)
    got = _linear(torch.eye(K).to(torch.bfloat16), W, "bf16")
    assert torch.equal(got.double(), ((q.view(1, K) - torch.arange(16).view(N, 1)) * 0.25).double().t())


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_linear_non_finite_rows_stay_apart(fmt, group, zeros):
    gen = _gen(5)
    W = ref.Weights(gen, (), 40, 512, fmt, group, zeros)
    x = torch.randn((6, 512), generator=gen).to(torch.bfloat16)
    clean = _linear(x, W, "bf16")
    x[2, 100] = math.nan
    x[4, 3] = math.inf
    got = _linear(x, W, "bf16")
    assert torch.equal(got[[0, 1, 3, 5]], clean[[0, 1, 3, 5]])
    assert got[2].isnan().all() and not got[4].isfinite().any()


def test_linear_nan_scale_reaches_its_row_only():
    gen = _gen(6)
    for io in ("bf16", "fp16"):
        W = ref.Weights(gen, (), 20, 256, "nvfp4")
        x = torch.randn((3, 256), generator=gen).abs().to(ref.IO[io])
        clean = _linear(x, W, io)
        W.scales[11, 5] = 0x7F
        got = _linear(x, W, io)
        keep = [n for n in range(20) if n != 11]
        assert torch.equal(got[:, keep], clean[:, keep]) and got[:, 11].isnan().all()


def test_linear_large_and_small_activations_keep_bf16_range():
    gen = _gen(7)
    W = ref.Weights(gen, (), 64, 512, "nvfp4")
    for size in (2.0 ** 100, 2.0 ** -100):
        x = (torch.randn((2, 512), generator=gen) * size).to(torch.bfloat16)
        x[1, 5] = size * 2.0 ** 20  # one value far above the rest
        got = _linear(x, W, "bf16")
        want, tol = ref.linear(x, W.value, "bf16")
        assert (got.double() - want).abs().le(tol).all()


def test_linear_results_repeat_and_empty_batch():
    gen = _gen(8)
    W = ref.Weights(gen, (), 500, 4096, "int4", 128)
    x = torch.randn((4, 4096), generator=gen).to(torch.bfloat16)
    a = _linear(x, W, "bf16")
    for _ in range(5):
        assert torch.equal(a, _linear(x, W, "bf16"))
    c = W.cuda("w")
    nqg.moe_linear_w4(torch.empty((0, 4096), device=DEV, dtype=torch.bfloat16), c["w"], c["w_scales"],
                      torch.empty((0, 500), device=DEV, dtype=torch.bfloat16), w_format="int4", group_size=128)


# ---------------------------------------------------------------------- layer

LAYER_FORMATS = [("none", 0, False), ("nvfp4", 16, False), ("int4", 64, True)]


class Problem:
    def __init__(self, T, H, I, E, k, fmt="none", group=0, zeros=False, io="bf16", seed=0, extras=True):
        gen = _gen(seed + 31 * T + H + I + E + k)
        self.T, self.H, self.I, self.E, self.k, self.fmt, self.group, self.io = T, H, I, E, k, fmt, group, io
        self.x = torch.randn((T, H), generator=gen).to(ref.IO[io])
        self.w13 = ref.Weights(gen, (E,), 2 * I, H, fmt, group, zeros, io)
        self.w2 = ref.Weights(gen, (E,), H, I, fmt, group, zeros, io)
        self.ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32) \
            if T else torch.empty((0, k), dtype=torch.int32)
        self.rw = torch.softmax(torch.randn((T, k), generator=gen), 1)
        self.shared = torch.randn((T, H), generator=gen).to(ref.IO[io]) if extras else None
        self.residual = torch.randn((T, H), generator=gen).to(ref.IO[io]) if extras else None
        self.status = None

    def run(self, activation="silu", stream=None, weight_dtype="fp32", x_pad=0):
        c = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        T, H = self.T, self.H
        xs = torch.full((T, H + x_pad), math.nan, dtype=ref.IO[self.io], device=DEV)
        xs[:, :H] = c(self.x)
        ob, out = _canary(T * H, ref.IO[self.io])
        n = nqg.moe_layer_workspace_size(T, self.k, self.I)
        wb = torch.full((n + 512,), 0xA5, device=DEV, dtype=torch.uint8)
        status = torch.zeros(1, device=DEV, dtype=torch.int32)
        kw = dict(x=xs[:, :H], topk_ids=c(self.ids), router_weights=c(self.rw.to(DT[weight_dtype])),
                  w_format=self.fmt, group_size=self.group, activation=activation, shared_out=c(self.shared),
                  residual=c(self.residual), out=out.view(T, H), workspace=wb[:n], status=status, io_dtype=self.io,
                  weight_dtype=weight_dtype, **self.w13.cuda("w13"), **self.w2.cuda("w2"))
        torch.cuda.synchronize()
        nqg.moe_layer(stream=stream, **kw)
        torch.cuda.synchronize()
        assert _untouched(ob, out) and bool((wb[n:] == 0xA5).all())
        self.status = int(status.item())
        return out.view(T, H).cpu()

    def check(self, activation="silu", weight_dtype="fp32", **kw):
        got = self.run(activation, weight_dtype=weight_dtype, **kw)
        want, tol = ref.layer(self.x, self.ids, self.rw.to(DT[weight_dtype]), self.w13.value, self.w2.value,
                              activation, self.io, self.shared, self.residual)
        bad = ~(got.double() - want).abs().le(tol)
        assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))
        return got


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group,zeros", LAYER_FORMATS)
@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 64, 1, 1), (1, 256, 128, 8, 2), (3, 320, 192, 5, 3), (8, 128, 64, 16, 8),
                                       (9, 192, 320, 6, 4), (16, 256, 128, 8, 2), (17, 128, 64, 40, 5),
                                       (32, 64, 128, 3, 2), (33, 128, 192, 4, 3), (64, 64, 64, 70, 4),
                                       (64, 128, 64, 2, 2), (2, 1024, 576, 3, 2)])
def test_layer_matches_definition(T, H, I, E, k, fmt, group, zeros, io):
    p = Problem(T, H, I, E, k, fmt, group, zeros, io)
    p.check("silu" if (T + k) % 2 else "gelu_tanh")
    assert p.status == 0


@pytest.mark.parametrize("H,I", [(8, 8), (24, 8), (40, 72), (136, 24), (1000, 104)])
def test_layer_odd_sizes_16_bit(H, I):
    for T in (1, 5, 20):
        Problem(T, H, I, 7, 3).check()


@pytest.mark.parametrize("H,I", [(16, 16), (48, 16), (80, 112), (144, 208)])
def test_layer_odd_sizes_nvfp4(H, I):
    for T in (1, 11):
        for io in ("bf16", "fp16"):
            Problem(T, H, I, 5, 2, "nvfp4", 16, io=io).check()


@pytest.mark.parametrize("wd", ["fp32", "bf16", "fp16"])
def test_layer_router_weight_types_and_strided_x(wd):
    Problem(6, 128, 64, 9, 3).check(weight_dtype=wd, x_pad=40)


def test_layer_plain_sum_without_extras():
    for fmt, group, zeros in LAYER_FORMATS:
        Problem(4, 128, 64, 6, 2, fmt, group, zeros, extras=False).check("gelu_tanh")


def test_layer_padding_repeats_and_invalid_ids():
    p = Problem(12, 128, 64, 6, 4)
    p.ids[0] = -1                      # a token without experts
    p.ids[3, 1:] = -1
    p.ids[5] = p.ids[5, 0].item()      # one expert four times
    p.ids[6, 2] = p.ids[6, 0]
    want = p.check()
    assert p.status == 0
    # weights of slots without an expert do not matter, whatever they are
    p.rw[0] = math.nan
    p.rw[3, 1:] = math.inf
    assert torch.equal(p.run(), want)
    # ids out of range are padding, and reported
    p.ids[3, 2], p.ids[0, 0] = 6, -2
    assert torch.equal(p.run(), want)
    assert p.status == nqg.MOE_ERR_INVALID_EXPERT


def test_layer_all_tokens_padded():
    for extras in (True, False):
        p = Problem(5, 64, 64, 4, 2, extras=extras)
        p.ids[:] = -1
        got = p.check()
        if not extras:
            assert bool((got == 0).all())


@pytest.mark.parametrize("T", [8, 64])
def test_layer_every_token_on_one_expert(T):
    for fmt, group, zeros in LAYER_FORMATS:
        p = Problem(T, 128, 64, 9, 1, fmt, group, zeros)
        p.ids[:] = 7
        p.check()


def test_layer_limits_of_experts_and_slots():
    p = Problem(64, 64, 64, 1024, 32)   # 2048 slots, every expert limit
    p.check()
    p = Problem(2, 64, 64, 1000, 8)
    p.ids[0, 0], p.ids[1, 3] = 999, 0
    p.check()


def test_layer_non_finite_tokens_stay_apart():
    p = Problem(7, 128, 64, 3, 2)
    clean = p.run()
    p.x[2, 5] = math.nan
    p.x[4, 0] = math.inf
    got = p.run()
    keep = [0, 1, 3, 5, 6]
    assert torch.equal(got[keep], clean[keep])
    assert got[2].isnan().all() and not got[4].isfinite().any()


def test_layer_unselected_experts_are_not_read_into_the_result():
    for T in (2, 12):
        p = Problem(T, 128, 64, 8, 2)
        p.ids = p.ids % 5
        p.ids[:, 1] = (p.ids[:, 0] + 1) % 5
        want = p.check()
        p.w13.codes[5:] = math.nan
        p.w2.codes[5:] = math.nan
        assert torch.equal(p.run(), want)


def test_layer_repeats_on_another_stream_and_in_a_graph():
    p = Problem(10, 256, 128, 12, 4, "nvfp4", 16)
    want = p.check()
    s = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(p.run(stream=s), want)
    c = lambda t: t.to(DEV)  # noqa: E731
    out = torch.zeros((10, 256), device=DEV, dtype=torch.bfloat16)
    ws = torch.empty(nqg.moe_layer_workspace_size(10, 4, 128), device=DEV, dtype=torch.uint8)
    args = nqg.layer_args(x=c(p.x), topk_ids=(ids := c(p.ids)), router_weights=(rw := c(p.rw)), w_format="nvfp4",
                          out=out, workspace=ws, shared_out=(sh := c(p.shared)), residual=(re := c(p.residual)),
                          **(a := p.w13.cuda("w13")), **(b := p.w2.cuda("w2")))
    x = c(p.x)
    args.x = x.data_ptr()
    keep = (ids, rw, sh, re, a, b, x)
    with torch.cuda.stream(s):
        nqg.moe_layer(args=args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                nqg.moe_layer(args=args)
    out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want) and keep


def test_layer_consecutive_calls_share_a_workspace():
    # calls of different sizes back to back on one stream and one workspace
    ps = [Problem(t, 128, 64, 8, 2, seed=t) for t in (1, 16, 3, 40, 8)]
    want = [p.run() for p in ps]
    ws = torch.empty(nqg.moe_layer_workspace_size(64, 2, 64), device=DEV, dtype=torch.uint8)
    c = lambda t: t.to(DEV)  # noqa: E731
    held = [dict(x=c(p.x), topk_ids=c(p.ids), router_weights=c(p.rw), shared_out=c(p.shared), residual=c(p.residual),
                 out=torch.zeros((p.T, 128), device=DEV, dtype=torch.bfloat16), workspace=ws, **p.w13.cuda("w13"),
                 **p.w2.cuda("w2")) for p in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for kw in held:
            nqg.moe_layer(**kw)
    torch.cuda.synchronize()
    for kw, w in zip(held, want):
        assert torch.equal(kw["out"].cpu(), w)


def test_select_then_layer_as_a_decode_step():
    T, H, I, E, k = 6, 256, 128, 24, 4
    p = Problem(T, H, I, E, k)
    logits = torch.randn((T, E), generator=_gen(11))
    logits[2] = -math.inf  # a padded token
    ids = torch.empty((T, k), device=DEV, dtype=torch.int32)
    rw = torch.empty((T, k), device=DEV)
    out = torch.empty((T, H), device=DEV, dtype=torch.bfloat16)
    ws = torch.empty(nqg.moe_layer_workspace_size(T, k, I), device=DEV, dtype=torch.uint8)
    c = lambda t: t.to(DEV)  # noqa: E731
    kw = dict(x=c(p.x), shared_out=c(p.shared), residual=c(p.residual), **p.w13.cuda("w13"), **p.w2.cuda("w2"))
    lg = c(logits)
    for _ in range(3):  # back to back: each kernel may start while the one before it runs
        nqg.moe_select_experts(lg, ids, rw)
        nqg.moe_layer(topk_ids=ids, router_weights=rw, out=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    p.ids, w = ref.select(logits, k, "softmax", True, 1.0)
    assert torch.equal(ids.cpu(), p.ids)
    p.rw = rw.cpu()
    want, tol = ref.layer(p.x, p.ids, p.rw, p.w13.value, p.w2.value, "silu", "bf16", p.shared, p.residual)
    assert (out.cpu().double() - want).abs().le(tol).all()


@pytest.mark.parametrize("where", ["x", "shared_out", "residual"])
def test_layer_in_place(where):
    p = Problem(7, 512, 256, 8, 2)
    want = p.run()
    c = lambda t: t.to(DEV)  # noqa: E731
    kw = dict(x=c(p.x), shared_out=c(p.shared), residual=c(p.residual), **p.w13.cuda("w13"), **p.w2.cuda("w2"))
    ws = torch.empty(nqg.moe_layer_workspace_size(7, 2, 256), device=DEV, dtype=torch.uint8)
    nqg.moe_layer(topk_ids=c(p.ids), router_weights=c(p.rw), out=kw[where], workspace=ws, **kw)
    assert torch.equal(kw[where].cpu(), want)


def test_layer_empty_batch_is_a_no_op():
    p = Problem(0, 64, 64, 4, 2)
    c = p.w13.cuda("w13") | p.w2.cuda("w2")
    nqg.moe_layer(x=p.x.to(DEV), topk_ids=p.ids.to(DEV), router_weights=p.rw.to(DEV),
                  out=torch.empty((0, 64), device=DEV, dtype=torch.bfloat16),
                  workspace=torch.empty(0, device=DEV, dtype=torch.uint8), **c)


# ---------------------------------------------------------------- bounded waits

@pytest.mark.parametrize("M,N,K,fmt,group", [(1, 3000, 4096, "nvfp4", 16), (5, 3000, 1024, "int4", 128),
                                             (40, 3000, 1024, "nvfp4", 16)])
def test_linear_wait_that_runs_out_marks_its_rows_and_the_context_survives(M, N, K, fmt, group):
    gen = _gen(3)
    W = ref.Weights(gen, (), N, K, fmt, group, False)
    x = torch.randn((M, K), generator=gen).to(torch.bfloat16)
    good = _linear(x, W, "bf16")
    try:
        nqg.moe_debug_stall(0)
        got = _linear(x, W, "bf16")
    finally:
        nqg.moe_debug_stall(-1)
    assert got[:, :16].isnan().all()
    late = got.isnan().all(0)
    assert torch.equal(got[:, ~late], good[:, ~late]) and int(late.sum()) < N // 16
    assert torch.equal(_linear(x, W, "bf16"), good)


def test_layer_wait_that_runs_out_is_reported_and_the_context_survives():
    p = Problem(4, 512, 256, 8, 2)
    p.ids[:] = torch.tensor([[0, 1], [2, 3], [0, 4], [5, 6]])
    good = p.run()
    assert p.status == 0
    try:
        nqg.moe_debug_stall(0)
        got = p.run()
    finally:
        nqg.moe_debug_stall(-1)
    assert p.status == nqg.MOE_ERR_DEVICE_TIMEOUT
    assert got[[0, 2]].isnan().all()  # the tokens of the first expert, of whose values the first block makes some
    assert torch.equal(got[[1, 3]], good[[1, 3]])
    assert torch.equal(p.run(), good) and p.status == 0


def test_example_decode_step():
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _, error, status = module.main(["--tokens", "5", "--hidden", "512", "--inner", "256", "--experts", "8",
                                    "--top-k", "2", "--steps", "3"])
    # three roundings to bf16 on the way (2^-9 each at most) and the sum's
    assert status == 0 and error < 4 * 2.0 ** -9
