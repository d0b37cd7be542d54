"""A feed-forward block in training: norm, gated product, second product, norm, and their gradients.

    x     = N(residual; gamma1)                                     (what the block before it left)
    h     = act(x W1^T) * (x W3^T)                                  (moe_gated_linear)
    y     = h W2^T                                                  (moe_grouped_linear)
    s     = residual + gate * N(y; gamma2),  out = N(s; gamma3)     (moe_block_norm)

for a dense block (--experts 1) or for experts whose rows are grouped.  Each operator is wrapped as an autograd function;
the gradients of one step are compared with torch's, of the same formulas in fp32, and a step of plain calls is captured in
a CUDA graph and timed.

    python examples/block_training.py --rows 4096 --hidden 2048 --inner 4096 --experts 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import norm_quant_gb300 as nqg  # noqa: E402

EPS = 1e-6
BF16 = torch.bfloat16


def scratch(size, like):
    return torch.empty(size, dtype=torch.uint8, device=like.device)


class GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, offsets):
        rows, inner = x.shape[0], w13.shape[1] // 2
        gate_up, out = x.new_empty(rows, 2 * inner), x.new_zeros(rows, inner)
        nqg.moe_gated_linear(x, w13, out, offsets=offsets, gate_up=gate_up)
        ctx.save_for_backward(x, w13, offsets, gate_up)
        return out

    @staticmethod
    def backward(ctx, d_out):
        x, w13, offsets, gate_up = ctx.saved_tensors
        d_x, d_w13 = torch.zeros_like(x), torch.empty_like(w13)
        workspace = scratch(nqg.moe_gated_linear_backward_workspace_size(x.shape[0], d_out.shape[1]), x)
        nqg.moe_gated_linear_backward(d_out.contiguous(), gate_up, x=x, w13=w13, d_x=d_x, d_w13=d_w13, workspace=workspace,
                                      offsets=offsets)
        return d_x, d_w13, None


class GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        out = x.new_zeros(x.shape[0], w.shape[1])
        nqg.moe_grouped_linear(x, w, out, offsets=offsets)
        ctx.save_for_backward(x, w, offsets)
        return out

    @staticmethod
    def backward(ctx, d_out):
        x, w, offsets = ctx.saved_tensors
        d_x, d_w = torch.zeros_like(x), torch.empty_like(w)
        nqg.moe_grouped_linear_backward(d_out.contiguous(), x=x, w=w, d_x=d_x, d_w=d_w, offsets=offsets)
        return d_x, d_w, None


class BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, post, pre, gate):
        s, out = torch.empty_like(y), torch.empty_like(y)
        nqg.moe_block_norm(y, residual, post_gamma=post, pre_gamma=pre, gate=gate, gate_kind="channel", eps=EPS, residual_out=s,
                           norm_out=out)
        ctx.save_for_backward(y, residual, post, pre, gate)
        return s, out

    @staticmethod
    def backward(ctx, d_s, d_out):
        y, residual, post, pre, gate = ctx.saved_tensors
        d_y, d_residual = torch.empty_like(y), torch.empty_like(y)
        sums = [torch.empty(y.shape[1], device=y.device) for _ in range(3)]
        workspace = scratch(nqg.moe_block_norm_backward_workspace_size(*y.shape), y)
        nqg.moe_block_norm_backward(y, residual, post_gamma=post, pre_gamma=pre, gate=gate, gate_kind="channel", eps=EPS,
                                    d_residual_out=d_s.contiguous(), d_norm_out=d_out.contiguous(), d_y=d_y, d_residual=d_residual,
                                    d_post_gamma=sums[0], d_pre_gamma=sums[1], d_gate=sums[2], workspace=workspace)
        return d_y, d_residual, *(v.to(BF16) for v in sums)


class Block:
    def __init__(self, rows, hidden, inner, experts, device, seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std=1.0, mean=0.0):
            return (torch.randn(shape, generator=gen, device=device) * std + mean).to(BF16)

        self.x, self.residual = normal(rows, hidden), normal(rows, hidden)
        self.d_s, self.d_out = normal(rows, hidden), normal(rows, hidden)
        self.weights = {"w13": normal(experts, 2 * inner, hidden, std=hidden ** -0.5),
                        "w2": normal(experts, hidden, inner, std=inner ** -0.5), "post": normal(hidden, std=0.1, mean=1.0),
                        "pre": normal(hidden, std=0.1, mean=1.0), "gate": normal(hidden, std=0.3, mean=0.5)}
        cuts = torch.randint(0, rows + 1, (experts - 1,), generator=gen, device=device).sort().values
        ends = torch.tensor([0, rows], device=device)
        self.offsets = torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)

    def step(self):
        """Gradients of one step through autograd: of x, the residual and every weight."""
        leaves = {k: v.clone().requires_grad_() for k, v in {"x": self.x, "residual": self.residual, **self.weights}.items()}
        h = GatedLinear.apply(leaves["x"], leaves["w13"], self.offsets)
        y = GroupedLinear.apply(h, leaves["w2"], self.offsets)
        s, out = BlockNorm.apply(y, leaves["residual"], leaves["post"], leaves["pre"], leaves["gate"])
        grads = torch.autograd.grad([s, out], list(leaves.values()), [self.d_s, self.d_out])
        return dict(zip(leaves, grads))

    def plain(self):
        """The same from the formulas in fp32."""
        leaves = {k: v.float().requires_grad_() for k, v in {"x": self.x, "residual": self.residual, **self.weights}.items()}
        bounds, parts = self.offsets.tolist(), []
        for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
            gate, up = (leaves["x"][a:b] @ leaves["w13"][e].t()).chunk(2, 1)
            parts.append((gate * torch.sigmoid(gate) * up) @ leaves["w2"][e].t())
        y = torch.cat(parts)

        def norm(v, gamma):
            return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * gamma

        s = leaves["residual"] + leaves["gate"] * norm(y, leaves["post"])
        out = norm(s, leaves["pre"])
        grads = torch.autograd.grad([s, out], list(leaves.values()), [self.d_s.float(), self.d_out.float()])
        return dict(zip(leaves, grads))

    def calls(self):
        """A step as plain calls on buffers that are there already, for a graph."""
        w, rows = self.weights, self.x.shape[0]
        hidden, inner = w["w2"].shape[1:]
        z = lambda *shape, dtype=BF16: torch.zeros(shape, dtype=dtype, device=self.x.device)  # noqa: E731
        gate_up, h, y, s, out = z(rows, 2 * inner), z(rows, inner), z(rows, hidden), z(rows, hidden), z(rows, hidden)
        d_y, d_residual, d_h, d_x = z(rows, hidden), z(rows, hidden), z(rows, inner), z(rows, hidden)
        d_w13, d_w2 = torch.empty_like(w["w13"]), torch.empty_like(w["w2"])
        sums = [z(hidden, dtype=torch.float32) for _ in range(3)]
        norm_ws = scratch(nqg.moe_block_norm_backward_workspace_size(rows, hidden), h)
        gated_ws = scratch(nqg.moe_gated_linear_backward_workspace_size(rows, inner), h)
        norm = dict(post_gamma=w["post"], pre_gamma=w["pre"], gate=w["gate"], gate_kind="channel", eps=EPS)

        def run():
            nqg.moe_gated_linear(self.x, w["w13"], h, offsets=self.offsets, gate_up=gate_up)
            nqg.moe_grouped_linear(h, w["w2"], y, offsets=self.offsets)
            nqg.moe_block_norm(y, self.residual, residual_out=s, norm_out=out, **norm)
            nqg.moe_block_norm_backward(y, self.residual, d_residual_out=self.d_s, d_norm_out=self.d_out, d_y=d_y,
                                        d_residual=d_residual, d_post_gamma=sums[0], d_pre_gamma=sums[1], d_gate=sums[2],
                                        workspace=norm_ws, **norm)
            nqg.moe_grouped_linear_backward(d_y, x=h, w=w["w2"], d_x=d_h, d_w=d_w2, offsets=self.offsets)
            nqg.moe_gated_linear_backward(d_h, gate_up, x=self.x, w13=w["w13"], d_x=d_x, d_w13=d_w13, workspace=gated_ws,
                                          offsets=self.offsets)
            return {"x": d_x, "residual": d_residual, "w13": d_w13, "w2": d_w2}
        return run


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    block = Block(a.rows, a.hidden, a.inner, a.experts, "cuda")
    got, want = block.step(), block.plain()
    errors = {k: float((got[k].float() - want[k]).norm() / want[k].norm()) for k in want}
    run = block.calls()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        same = {k: torch.equal(v, got[k]) for k, v in run().items()}
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            graph.replay()
        start.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
        end.synchronize()
    us = start.elapsed_time(end) / a.steps * 1e3
    flops = 3 * 6 * a.rows * a.hidden * a.inner
    print(f"{a.rows} rows, {a.experts} experts of {a.hidden} x {a.inner}: {us:.1f} us a step, {flops / us / 1e6:.0f} TFLOP/s; "
          f"relative errors of the gradients " + ", ".join(f"{k} {v:.1e}" for k, v in errors.items()))
    return us, errors, same


if __name__ == "__main__":
    main()
