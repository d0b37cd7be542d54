"""A decode step of one mixture-of-experts layer with 4-bit weights.

For up to 64 tokens x [T, H] and a residual:

    logits  = gate x                                   (torch)
    ids, w  = the top_k experts of each token          (moe_select_experts)
    shared  = W2s (silu(W1s x) * (W3s x))              (moe_linear_w4, twice)
    out     = sum_j w_j W2_j (silu(W1_j x) * (W3_j x)) + shared + residual   (moe_layer)

The step is captured in a CUDA graph, replayed and timed, and its result is
compared with the same formulas in fp32 on the dequantised weights.

    python examples/decode_step.py --tokens 8 --experts 64 --top-k 6
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import norm_quant_gb300 as nqg  # noqa: E402

GROUP = 128


def quantise(w):
    """Asymmetric 4-bit integers of w [..., K] with a scale and a zero point per GROUP elements:
    packed codes, bf16 scales, uint8 zero points."""
    g = w.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=2.0 ** -40).to(torch.bfloat16)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    q = ((g / scale.float().unsqueeze(-1)).round() + zero.unsqueeze(-1)).clamp(0, 15).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), scale, zero.to(torch.uint8)


def dequantise(codes, scale, zero):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return ((q - zero.float().unsqueeze(-1)) * scale.float().unsqueeze(-1)).flatten(-2)


class Layer:
    """The weights of one layer and the buffers of a batch of `tokens` rows."""

    def __init__(self, tokens, hidden, inner, experts, top_k, device, seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def weights(*shape):
            return torch.randn(shape, generator=gen, device=device) * shape[-1] ** -0.5

        self.gate = weights(experts, hidden).to(torch.bfloat16)
        self.w13, self.w2 = quantise(weights(experts, 2 * inner, hidden)), quantise(weights(experts, hidden, inner))
        self.s13, self.s2 = quantise(weights(2 * inner, hidden)), quantise(weights(hidden, inner))
        self.x = torch.randn((tokens, hidden), generator=gen, device=device).to(torch.bfloat16)
        self.residual = torch.randn((tokens, hidden), generator=gen, device=device).to(torch.bfloat16)
        self.ids = torch.empty((tokens, top_k), dtype=torch.int32, device=device)
        self.router_weights = torch.empty((tokens, top_k), dtype=torch.float32, device=device)
        self.gate_up = torch.empty((tokens, 2 * inner), dtype=torch.bfloat16, device=device)
        self.shared, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        size = nqg.moe_layer_workspace_size(tokens, top_k, inner)
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def linear(self, x, weights, out):
        codes, scale, zero = weights
        nqg.moe_linear_w4(x, codes, scale, out, w_format="int4", group_size=GROUP, zeros=zero)

    def step(self):
        nqg.moe_select_experts(self.x @ self.gate.t(), self.ids, self.router_weights, logits_dtype="bf16")
        self.linear(self.x, self.s13, self.gate_up)
        gate, up = self.gate_up.chunk(2, 1)
        self.linear(F.silu(gate) * up, self.s2, self.shared)
        nqg.moe_layer(x=self.x, topk_ids=self.ids, router_weights=self.router_weights,
                      w13=self.w13[0], w13_scales=self.w13[1], w13_zeros=self.w13[2],
                      w2=self.w2[0], w2_scales=self.w2[1], w2_zeros=self.w2[2],
                      w_format="int4", group_size=GROUP, shared_out=self.shared, residual=self.residual,
                      out=self.out, workspace=self.workspace, status=self.status)

    def plain(self):
        """The step's formulas on dequantised weights; the selection is the step's own."""
        x = self.x.float()

        def expert(rows, w13, w2):
            gate, up = (rows @ w13.t()).chunk(2, 1)
            return (F.silu(gate) * up) @ w2.t()

        out = expert(x, dequantise(*self.s13), dequantise(*self.s2)) + self.residual.float()
        for e in self.ids.unique().tolist():
            token, slot = (self.ids == e).nonzero(as_tuple=True)
            y = expert(x[token], dequantise(*(p[e] for p in self.w13)), dequantise(*(p[e] for p in self.w2)))
            out.index_add_(0, token, self.router_weights[token, slot].unsqueeze(1) * y)
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=6)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args(argv)
    layer = Layer(a.tokens, a.hidden, a.inner, a.experts, a.top_k, "cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        layer.step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            graph.replay()
        start.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
        end.synchronize()
    want = layer.plain()
    error = float((layer.out.float() - want).norm() / want.norm())
    us = start.elapsed_time(end) / a.steps * 1e3
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.top_k}: "
          f"{us:.1f} us a step, relative error {error:.2e}, status {int(layer.status)}")
    return us, error, int(layer.status)


if __name__ == "__main__":
    main()
