"""The norms around a block on the GPU, forward and backward, against 64-bit
references: widths, gates, missing parts, outputs in place of inputs."""
import os
import subprocess
import sys

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _block_ref as ref
from test_gpu_block import gen, near, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


class Problem:
    def __init__(self, T, H, io="bf16", post=True, pre=True, gate="none", bias=0.0, residual=True, block_scale=1.0,
                 residual_scale=1.0, eps=1e-6, y_std=1.0):
        g = gen(T * H + len(gate))
        self.T, self.H, self.io = T, H, io
        self.y = normal(g, T, H, io=io, std=y_std)
        self.residual = normal(g, T, H, io=io, std=2.0) if residual else None
        self.post = (1 - bias + 0.2 * torch.randn(H, generator=g)).to(ref.IO[io]) if post else None
        self.pre = (1 - bias + 0.2 * torch.randn(H, generator=g)).to(ref.IO[io]) if pre else None
        self.kind = gate
        self.gate = {"none": None, "channel": normal(g, H, io=io), "token": torch.randn(T, generator=g)}[gate]
        self.d_res, self.d_norm = normal(g, T, H, io=io), normal(g, T, H, io=io) if pre else None
        self.options = dict(block_scale=block_scale, residual_scale=residual_scale, eps=eps, weight_bias=bias)
        self.ref = ref.Norm(self.y, self.residual, self.post, self.pre, self.gate, gate, block_scale, residual_scale, eps, bias, io)

    def dev(self, t):
        return None if t is None else t.to(DEV)

    def kw(self):
        return dict(post_gamma=self.dev(self.post), pre_gamma=self.dev(self.pre), gate=self.dev(self.gate),
                    gate_kind=self.kind, io_dtype=self.io, **self.options)

    def out(self, n=None, dtype=None):
        """A buffer inside canaries: (whole, view)."""
        shape = (self.T, self.H) if n is None else (n,)
        count = shape[0] * (shape[1] if n is None else 1)
        buf = torch.full((count + 64,), 13.0, dtype=dtype or ref.IO[self.io], device=DEV)
        return buf, buf[32:-32].view(shape)

    def check(self, pair, want):
        buf, view = pair
        assert bool((buf[:32] == 13).all()) and bool((buf[-32:] == 13).all())
        near(view, *want)

    def forward(self):
        r, n = self.out(), self.out() if self.pre is not None else None
        nqg.moe_block_norm(self.dev(self.y), self.dev(self.residual), residual_out=r[1], norm_out=n[1] if n else None, **self.kw())
        want_r, want_n = self.ref.forward()
        self.check(r, want_r)
        if n:
            self.check(n, want_n)
        return r[1], n[1] if n else None

    def backward(self, d_res=True, d_norm=True):
        d_res = self.d_res if d_res else None
        d_norm = self.d_norm if d_norm else None
        want = self.ref.backward(d_res, d_norm)
        f32 = torch.float32
        got = {"d_y": self.out()}
        if self.residual is not None:
            got["d_residual"] = self.out()
        if self.post is not None:
            got["d_post"] = self.out(self.H, f32)
        if d_norm is not None:
            got["d_pre"] = self.out(self.H, f32)
        if self.gate is not None:
            got["d_gate"] = self.out(self.gate.numel(), f32)
        at = lambda k: got[k][1] if k in got else None  # noqa: E731
        ws = torch.full((nqg.moe_block_norm_backward_workspace_size(self.T, self.H),), 255, dtype=torch.uint8, device=DEV)
        call = lambda: nqg.moe_block_norm_backward(  # noqa: E731
            self.dev(self.y), self.dev(self.residual), d_residual_out=self.dev(d_res), d_norm_out=self.dev(d_norm), d_y=at("d_y"),
            d_residual=at("d_residual"), d_post_gamma=at("d_post"), d_pre_gamma=at("d_pre"), d_gate=at("d_gate"), workspace=ws, **self.kw())
        call()
        for k, v in got.items():
            self.check(v, want[k])
        first = {k: v[1].clone() for k, v in got.items()}
        call()
        assert all(torch.equal(first[k], v[1]) for k, v in got.items())
        return first


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (5, 264), (1, 7168), (17, 2056), (200, 520), (2, 4104), (3, 8192), (2, 8200),
                                 (2, 16384), (700, 96)])
def test_forward_and_backward(T, H, gate, io):
    p = Problem(T, H, io, gate=gate, bias=float(T % 2), block_scale=0.5, residual_scale=0.75)
    p.forward()
    p.backward()


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre,residual", [(False, True, True), (True, False, True), (False, False, True), (True, True, False),
                                               (False, True, False)])
def test_missing_parts(post, pre, residual, gate):
    p = Problem(37, 328, post=post, pre=pre, residual=residual, gate=gate, residual_scale=0.5)
    p.forward()
    p.backward()
    if pre:
        p.backward(d_res=False)
    p.backward(d_norm=False)


def test_rows_of_zeros_and_small_values():
    """The epsilon holds where a row has nothing, and fp16's subnormals go through."""
    for io in ("bf16", "fp16"):
        p = Problem(9, 136, io, y_std=2.0 ** -12, eps=1e-5)
        p.y[3] = 0
        p.residual[3] = 0
        p.ref = ref.Norm(p.y, p.residual, p.post, p.pre, None, "none", 1.0, 1.0, 1e-5, 0.0, io)
        p.forward()
        p.backward()


def test_non_finite_rows_stay_alone():
    p = Problem(12, 200, gate="channel")
    y = p.y.to(DEV)
    y[4] = float("nan")
    y[9, 7] = float("inf")
    r, n = torch.empty_like(y), torch.empty_like(y)
    nqg.moe_block_norm(y, p.dev(p.residual), residual_out=r, norm_out=n, **p.kw())
    keep = [i for i in range(12) if i not in (4, 9)]
    want_r, want_n = p.ref.forward()
    near(r[keep], want_r[0][keep], want_r[1][keep])
    near(n[keep], want_n[0][keep], want_n[1][keep])
    assert bool(r[4].isnan().all()) and not bool(n[9].isfinite().all())


def test_outputs_in_place_of_inputs():
    p = Problem(150, 1032, gate="token", residual_scale=0.9)
    want_r, want_n = p.forward()
    y, r = p.dev(p.y), p.dev(p.residual)
    nqg.moe_block_norm(y, r, residual_out=r, norm_out=y, **p.kw())
    assert torch.equal(r, want_r) and torch.equal(y, want_n)
    grads = p.backward()
    for d_y, d_residual in (("y", "r"), ("dn", "dr"), ("dr", "dn")):
        t = {"y": p.dev(p.y), "r": p.dev(p.residual), "dr": p.dev(p.d_res), "dn": p.dev(p.d_norm)}
        nqg.moe_block_norm_backward(t["y"], t["r"], d_residual_out=t["dr"], d_norm_out=t["dn"], d_y=t[d_y],
                                    d_residual=t[d_residual], **p.kw())
        assert torch.equal(t[d_y], grads["d_y"]) and torch.equal(t[d_residual], grads["d_residual"])


def test_single_outputs_and_no_workspace():
    p = Problem(40, 264, gate="token")
    r, n = p.forward()
    one = torch.empty_like(n)
    nqg.moe_block_norm(p.dev(p.y), p.dev(p.residual), norm_out=one, **p.kw())
    assert torch.equal(one, n)
    nqg.moe_block_norm(p.dev(p.y), p.dev(p.residual), residual_out=one, **p.kw())
    assert torch.equal(one, r)
    grads = p.backward()
    for name in ("d_y", "d_residual", "d_gate"):  # none of them a sum over tokens
        got = torch.empty_like(grads[name])
        nqg.moe_block_norm_backward(p.dev(p.y), p.dev(p.residual), d_residual_out=p.dev(p.d_res), d_norm_out=p.dev(p.d_norm),
                                    **{name: got}, **p.kw())
        assert torch.equal(got, grads[name])


def test_no_tokens():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    gamma = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    nqg.moe_block_norm(e, e, post_gamma=gamma, residual_out=e.clone())
    sums = [torch.full((64,), 13.0, device=DEV) for _ in range(3)]
    nqg.moe_block_norm_backward(e, e, post_gamma=gamma, pre_gamma=gamma, gate=gamma, gate_kind="channel", d_norm_out=e,
                                d_post_gamma=sums[0], d_pre_gamma=sums[1], d_gate=sums[2])
    assert all(bool((s == 0).all()) for s in sums)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_gradients_against_differences(gate):
    """Along random directions: the kernels' gradients against central differences of the 64-bit forward formulas."""
    p = Problem(6, 72, gate=gate, block_scale=0.7, residual_scale=0.6, bias=1.0)
    grads = p.backward()

    def loss(v):
        n = ref.Norm(v["y"], v["residual"], v["post"], v["pre"], v.get("gate"), gate, 0.7, 0.6, 1e-6, 1.0, "bf16")
        return float((n.s * p.d_res.double()).sum() + (n.m * n.pre * p.d_norm.double()).sum())

    base = {k: getattr(p, k).double() for k in ("y", "residual", "post", "pre") + (("gate",) if p.gate is not None else ())}
    h = 1e-5
    for name in base:
        got = grads["d_" + name].cpu().double()
        for seed in range(3):
            v = torch.randn(base[name].shape, generator=gen(seed)).double()
            want = (loss({**base, name: base[name] + h * v}) - loss({**base, name: base[name] - h * v})) / (2 * h)
            # one rounding to bf16 of d_y and d_residual; the others are fp32
            assert abs(float((got * v).sum()) - want) <= 2.0 ** -8 * float((got * v).abs().sum()) + 1e-6


def test_graph_capture_and_two_graphs_with_one_workspace():
    """Graphs that share a workspace and run one after the other."""
    ps = [Problem(33, 520, gate="channel"), Problem(60, 520, gate="channel")]
    want = [p.backward() for p in ps]
    ws = torch.empty(max(nqg.moe_block_norm_backward_workspace_size(p.T, p.H) for p in ps), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for p in ps:
            o = {"d_y": p.out()[1], "d_residual": p.out()[1], "d_post_gamma": p.out(p.H, torch.float32)[1],
                 "d_pre_gamma": p.out(p.H, torch.float32)[1], "d_gate": p.out(p.H, torch.float32)[1]}
            args = [p.dev(p.y), p.dev(p.residual)]
            kw = dict(d_residual_out=p.dev(p.d_res), d_norm_out=p.dev(p.d_norm), workspace=ws, **o, **p.kw())
            side.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                nqg.moe_block_norm_backward(*args, **kw)
            outs.append((o, args, kw))
        for _ in range(2):
            for gr in graphs:
                gr.replay()
        side.synchronize()
    for (o, _, _), w in zip(outs, want):
        for k, name in (("d_y", "d_y"), ("d_residual", "d_residual"), ("d_post_gamma", "d_post"), ("d_pre_gamma", "d_pre"), ("d_gate", "d_gate")):
            assert torch.equal(o[k], w[name])


def test_large_batch():
    """More rows than CTAs hold at once, against the same rows in parts."""
    T, H = 5000, 1544
    g = gen(3)
    y, r = normal(g, T, H).to(DEV), normal(g, T, H).to(DEV)
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).to(DEV)
    whole, parts = [torch.empty_like(y) for _ in range(2)], [torch.empty_like(y) for _ in range(2)]
    nqg.moe_block_norm(y, r, post_gamma=gamma, pre_gamma=gamma, residual_out=whole[0], norm_out=whole[1])
    for at in (slice(0, 100), slice(100, 2777), slice(2777, T)):
        nqg.moe_block_norm(y[at], r[at], post_gamma=gamma, pre_gamma=gamma, residual_out=parts[0][at], norm_out=parts[1][at])
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))


def test_offsets_beyond_32_bits():
    """Matrices of more than 2^32 bytes: their last rows as a call of their own makes them, forward and backward."""
    T, H, n = 530000, 4104, 1000
    assert 2 * T * H > 2 ** 32 and T * H > 2 ** 31
    g = gen(5)
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).to(DEV)
    y, r, ds, dn = (torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(4))
    for v in (y, r, ds, dn):
        v[-n:] = normal(g, n, H).to(DEV)
    kw = dict(post_gamma=gamma, pre_gamma=gamma, eps=1e-5)
    out = [torch.full((T, H), 13.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    nqg.moe_block_norm(y, r, residual_out=out[0], norm_out=out[1], **kw)
    few = [torch.empty_like(y[-n:]) for _ in range(2)]
    nqg.moe_block_norm(y[-n:], r[-n:], residual_out=few[0], norm_out=few[1], **kw)
    assert all(torch.equal(a[-n:], b) for a, b in zip(out, few)) and all(bool((a[:-n] == 0).all()) for a in out)
    nqg.moe_block_norm_backward(y, r, d_residual_out=ds, d_norm_out=dn, d_y=out[0], d_residual=out[1], **kw)
    nqg.moe_block_norm_backward(y[-n:], r[-n:], d_residual_out=ds[-n:], d_norm_out=dn[-n:], d_y=few[0], d_residual=few[1], **kw)
    assert all(torch.equal(a[-n:], b) for a, b in zip(out, few)) and all(bool((a[:-n] == 0).all()) for a in out)


WIDE = """
import torch, norm_quant_gb300 as nqg
def run(H, io, whole):
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    v = [torch.ones((3, H), dtype=dt, device="cuda") for _ in range(6)]
    gamma, sums = torch.ones(H, dtype=dt, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(nqg.moe_block_norm_backward_workspace_size(3, H), dtype=torch.uint8, device="cuda")
    more = dict(d_residual_out=v[3], d_residual=v[5]) if whole else {}
    nqg.moe_block_norm_backward(v[0], v[1], post_gamma=gamma, pre_gamma=gamma, d_norm_out=v[2], d_y=v[4], d_post_gamma=sums,
                                workspace=ws, io_dtype=io, **more)
for io in ("bf16", "fp16"):
    for H, whole in ((16384, True), (8200, False), (16384, True), (12000, False), (8208, True), (16384, False)):
        run(H, io, whole)
torch.cuda.synchronize()
"""


def test_wide_rows_of_all_forms_in_turn():
    """The widest rows after narrower ones of another form, in a process that has made no call yet."""
    subprocess.run([sys.executable, "-c", WIDE], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   timeout=90)
