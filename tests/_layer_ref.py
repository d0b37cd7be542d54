"""Plain 64-bit references of the few-token operators, with bounds on the
error of a kernel that keeps its sums in fp32, for the parity tests.

Bounds.  u is the unit roundoff of the output type (2^-8 bf16, 2^-11 fp16).
A sum of K products held in fp32 and added 16 at a time, then over at most 64
partial sums, has an error of at most (K / 16 + 96) 2^-23 times the sum of the
products' magnitudes (2^-23: an addition that truncates).  The activation adds
its own fp32 error, its derivative (at most 1.13 for both) carries the error of
the gate, and the gated product is rounded once to the 16-bit type."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
IO = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24}  # spacing of the subnormals


def sum_eps(K):
    return (K / 16 + 96) * 2.0 ** -23


def e4m3(codes):
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def unpack(codes):
    lo, hi = (codes & 15).to(torch.int64), (codes >> 4).to(torch.int64)
    return torch.stack((lo, hi), -1).flatten(-2)


class Weights:
    """Random weights [*lead, N, K] in a format, with their 64-bit values."""

    def __init__(self, gen, lead, N, K, fmt, group=64, zeros=False, io="bf16", std=None):
        std = std or K ** -0.5
        shape = (*lead, N, K)
        self.fmt, self.group = fmt, group
        self.scales = self.zeros = self.glob = None
        if fmt == "none":
            self.codes = (torch.randn(shape, generator=gen) * std).to(IO[io])
            self.value = self.codes.double()
            return
        self.codes = torch.randint(0, 256, (*lead, N, K // 2), generator=gen, dtype=torch.uint8)
        q = unpack(self.codes)
        if fmt == "nvfp4":
            self.scales = torch.randint(0x20, 0x7F, (*lead, N, K // 16), generator=gen, dtype=torch.uint8)
            self.glob = (torch.rand(lead or (1,), generator=gen) + 0.5) * (500 / std)
            g = self.glob.double().view(*lead, 1, 1) if lead else self.glob.double()
            self.value = E2M1[q] * e4m3(self.scales).repeat_interleave(16, -1) / g
        else:
            self.scales = ((torch.rand((*lead, N, K // group), generator=gen) + 0.5) * std / 4.8).to(IO[io])
            z = torch.full(self.scales.shape, 8, dtype=torch.uint8)
            if zeros:
                z = torch.randint(0, 16, self.scales.shape, generator=gen, dtype=torch.uint8)
                self.zeros = z
            self.value = (q.double() - z.double().repeat_interleave(group, -1)) * \
                self.scales.double().repeat_interleave(group, -1)

    def cuda(self, name):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return {name: c(self.codes), f"{name}_scales": c(self.scales), f"{name}_zeros": c(self.zeros),
                f"{name}_global": c(self.glob)}


def linear(x, W, io):
    """(result, bound) of x W^T in 64 bits; x is of the io type."""
    y = x.double() @ W.t()
    mag = x.double().abs() @ W.abs().t()
    err = sum_eps(x.shape[1]) * mag
    return y, err + U[io] * (y.abs() + err) + TINY[io]


def act(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def layer(x, ids, rw, w13, w2, kind, io, shared=None, residual=None):
    """(result, bound) of the expert layer in 64 bits."""
    T, H = x.shape
    E, _, I = w2.shape
    out = torch.zeros(T, H, dtype=torch.float64)
    err = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    for t in range(T):
        for e in sorted({int(v) for v in ids[t] if 0 <= v < E}):
            w = float(sum(rw[t, j].double() for j in range(ids.shape[1]) if int(ids[t, j]) == e))
            xt, m = x[t].double(), w13[e]
            h, hm = m @ xt, sum_eps(H) * (m.abs() @ xt.abs())
            g, up, dg, du = h[:I], h[I:], hm[:I], hm[I:]
            ag = act(g, kind)
            a = w * ag * up
            da = abs(w) * (1.13 * dg * (up.abs() + du) + ag.abs() * du
                           + 2.0 ** -21 * (g.abs() + ag.abs()) * up.abs()) + 2.0 ** -22 * a.abs()
            da = da + U[io] * (a.abs() + da) + TINY[io]
            out[t] += w2[e] @ a
            err[t] += w2[e].abs() @ da
            mag[t] += w2[e].abs() @ a.abs()
    for extra in (shared, residual):
        if extra is not None:
            out += extra.double()
            mag += extra.double().abs()
    err = err + sum_eps(I * ids.shape[1]) * mag
    return out, err + U[io] * (out.abs() + err) + TINY[io]


def select(logits, k, scoring, renorm, scale):
    """(ids, weights) by the definition, in 64 bits."""
    T, E = logits.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    big = torch.finfo(torch.float32).max
    for t in range(T):
        row = [float(v) for v in logits[t].double()]
        open_ = [e for e in range(E) if row[e] > -math.inf]  # drops NaN too
        order = sorted(open_, key=lambda e: (-row[e], e))[:k]
        if not order:
            continue
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        if scoring == "softmax":
            top = max(-big, min(big, row[order[0]]))
            ex = {e: math.exp(max(-800.0, min(big, row[e]) - top)) for e in open_}
            s = [ex[e] for e in order]
            total = sum(s) if renorm else sum(ex.values())
        else:
            s = [1 / (1 + math.exp(min(700.0, -row[e]))) for e in order]
            total = sum(s) if renorm else 1.0
        w[t, :len(order)] = torch.tensor([v / total * scale for v in s], dtype=torch.float64)
    return ids, w
