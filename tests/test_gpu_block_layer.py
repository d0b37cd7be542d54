"""The block's operators together, as they are used: a whole expert layer between
routing and combine, forward and backward, and the example of a training step."""
import os
import sys

import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _block_ref as ref
from test_gpu_block import DEV, gen, near, normal

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import block_training  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


class Layer:
    """T tokens, some of them padded, through the top k of E experts."""

    def __init__(self, T, H, I, E, k, io="bf16"):
        g = gen(T + E)
        self.T, self.H, self.I, self.E, self.k, self.io = T, H, I, E, k, io
        self.x, self.residual = normal(g, T, H, io=io), normal(g, T, H, io=io)
        self.w13, self.w2 = normal(g, E, 2 * I, H, io=io, std=H ** -0.5), normal(g, E, H, I, io=io, std=I ** -0.5)
        self.post, self.pre = ((1 + 0.1 * torch.randn(H, generator=g)).to(ref.IO[io]) for _ in range(2))
        self.logits = torch.randn((T, E), generator=g)
        self.logits[1::7] = -torch.inf  # padded tokens have no expert
        self.d_out = normal(g, T, H, io=io)
        self.dev = {n: getattr(self, n).to(DEV) for n in ("x", "residual", "w13", "w2", "post", "pre", "logits", "d_out")}

    def forward(self):
        d, T, H, I, k, R = self.dev, self.T, self.H, self.I, self.k, self.T * self.k
        dt, i32 = ref.IO[self.io], dict(dtype=torch.int32, device=DEV)
        z = lambda *s: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        ids, weights = torch.empty((T, k), **i32), torch.empty((T, k), device=DEV)
        nqg.moe_select_experts(d["logits"], ids, weights)
        counts, offsets, row_map = torch.empty(self.E, **i32), torch.empty(self.E + 1, **i32), torch.empty((T, k), **i32)
        ws = torch.empty(nqg.moe_build_row_map_workspace_size(T, k, self.E), dtype=torch.uint8, device=DEV)
        nqg.moe_build_row_map(ids, self.E, counts, offsets, row_map, None, ws)
        xg, gate_up, h, y = z(R, H), z(R, 2 * I), z(R, I), z(R, H)
        nqg.moe_dispatch_permute(d["x"], row_map, xg)
        nqg.moe_gated_linear(xg, d["w13"], h, offsets=offsets, gate_up=gate_up, io_dtype=self.io)
        nqg.moe_grouped_linear(h, d["w2"], y, offsets=offsets, io_dtype=self.io)
        combined, s, out = z(T, H), z(T, H), z(T, H)
        nqg.moe_combine(expert_out=y, row_map=row_map, router_weights=weights, combined_out=combined, io_dtype=self.io)
        nqg.moe_block_norm(combined, d["residual"], post_gamma=d["post"], pre_gamma=d["pre"], residual_out=s, norm_out=out,
                           io_dtype=self.io)
        return dict(ids=ids, weights=weights, offsets=offsets, row_map=row_map, xg=xg, gate_up=gate_up, h=h, y=y, combined=combined,
                    s=s, out=out)

    def backward(self, f):
        """From the gradient of out: d_x, d_w13, d_w2, d_residual.  The combine's own gradient (a row of d_combined times
        its weight for each slot) is torch's; that of the dispatch is a combine with weights of 1."""
        d, T, H, I, R = self.dev, self.T, self.H, self.I, self.T * self.k
        z = lambda *s: torch.zeros(s, dtype=ref.IO[self.io], device=DEV)  # noqa: E731
        d_combined, d_residual = z(T, H), z(T, H)
        nqg.moe_block_norm_backward(f["combined"], d["residual"], post_gamma=d["post"], pre_gamma=d["pre"], d_norm_out=d["d_out"],
                                    d_y=d_combined, d_residual=d_residual, io_dtype=self.io)
        d_y = z(R, H)
        taken = f["row_map"] >= 0
        slots = (d_combined.float().unsqueeze(1) * f["weights"].unsqueeze(2)).to(d_y.dtype)
        d_y[f["row_map"][taken].long()] = slots[taken]
        d_h, d_w2, d_xg, d_w13, d_x = z(R, I), torch.empty_like(d["w2"]), z(R, H), torch.empty_like(d["w13"]), z(T, H)
        nqg.moe_grouped_linear_backward(d_y, x=f["h"], w=d["w2"], d_x=d_h, d_w=d_w2, offsets=f["offsets"], io_dtype=self.io)
        ws = torch.empty(nqg.moe_gated_linear_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
        nqg.moe_gated_linear_backward(d_h, f["gate_up"], x=f["xg"], w13=d["w13"], d_x=d_xg, d_w13=d_w13, workspace=ws,
                                      offsets=f["offsets"], io_dtype=self.io)
        nqg.moe_combine(expert_out=d_xg, row_map=f["row_map"], router_weights=torch.ones_like(f["weights"]), combined_out=d_x,
                        io_dtype=self.io)
        return dict(x=d_x, w13=d_w13, w2=d_w2, residual=d_residual)

    def plain(self, ids, weights):
        """(out, gradients) of the whole layer in 64 bits; the selection is the layer's own."""
        leaf = {n: getattr(self, n).double().requires_grad_() for n in ("x", "residual", "w13", "w2")}
        y = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            t, j = (ids == e).nonzero(as_tuple=True)
            gate, up = (leaf["x"][t] @ leaf["w13"][e].t()).chunk(2, 1)
            y = y.index_add(0, t, ((ref.act(gate, "silu") * up) @ leaf["w2"][e].t()) * weights[t, j].double().unsqueeze(1))
        norm = lambda v, c: v * ((v * v).mean(1, keepdim=True) + 1e-6) ** -0.5 * c.double()  # noqa: E731
        out = norm(leaf["residual"] + norm(y, self.post), self.pre)
        return out.detach(), dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), self.d_out.double())))


@pytest.mark.parametrize("T,H,I,E,k,io", [(61, 256, 136, 8, 2, "bf16"), (300, 136, 200, 33, 4, "fp16"), (1, 64, 64, 4, 1, "bf16")])
def test_expert_layer(T, H, I, E, k, io):
    layer = Layer(T, H, I, E, k, io)
    f = layer.forward()
    c = {n: v.cpu() for n, v in f.items()}
    # each stage against its formula on what the stage before it left
    bounds = c["offsets"].tolist()
    n = bounds[-1]
    (h, hb), (gu, gb) = ref.gated(c["xg"][:n], layer.w13, bounds, "silu", io)
    near(f["h"][:n], h, hb)
    near(f["gate_up"][:n], gu, gb)
    y, yb, _ = ref.product(c["h"][:n], layer.w2, bounds, io)
    near(f["y"][:n], y, yb)
    norm = ref.Norm(c["combined"], layer.residual, layer.post, layer.pre, None, "none", 1.0, 1.0, 1e-6, 0.0, io)
    (s, sb), (out, ob) = norm.forward()
    near(f["s"], s, sb)
    near(f["out"], out, ob)
    # and the whole: five roundings on the way (h, y, combined, s's norm, out), and of the gradients eight, each of at most U of
    # its value, whose norms the products by random weights keep
    want, grads = layer.plain(c["ids"], c["weights"])
    far = lambda a, b: float((a.cpu().double() - b).norm() / b.norm().clamp(min=1e-30))  # noqa: E731
    assert far(f["out"], want) <= 5 * ref.U[io]
    got = layer.backward(f)
    for name, g in grads.items():
        assert far(got[name], g) <= 8 * ref.U[io], name


@pytest.mark.parametrize("experts", [1, 5])
def test_example_runs_and_its_gradients_are_right(experts):
    us, errors, same = block_training.main(["--rows", "300", "--hidden", "256", "--inner", "136", "--experts", str(experts), "--steps", "2"])
    assert us > 0 and all(same.values())
    # roundings to bf16 on the way to each: at most h, y, d_y, d_h, dg and du, and its own
    assert all(e <= 6 * 2.0 ** -8 for e in errors.values()), errors
