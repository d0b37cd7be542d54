"""Plain 64-bit references of the block's operators for many tokens, with bounds
on the error of kernels that hold sums and norms in fp32.

u is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16: half a step
of a value at the lower end of its binade), and a sum of K products has the error
that _layer_ref.sum_eps states.  The activations and their slopes are off by at most
2^-20 (|g| + 1): their exponential by (|z| + 4) 2^-23 of itself, with z times its
slope at most 0.5 + |g|, and a handful of roundings."""
from __future__ import annotations

import math

import torch

from _layer_ref import IO, TINY, U, act, sum_eps  # noqa: F401  (used by the tests)


def slope(g, kind):
    if kind == "silu":
        p = torch.sigmoid(g)
        return p * (1 + g * (1 - p))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def ranges(bounds):
    return [slice(a, b) for a, b in zip(bounds[:-1], bounds[1:])]


def rounded(v, err, io):
    """The bound after one rounding of a value that is off by err."""
    return err + U[io] * (v.abs() + err) + TINY[io]


def product(x, w, bounds, io):
    """(result, bound) of out[r] = W[e] x[r]; rows of no expert are 0."""
    x = x.double()
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64)
    err = torch.zeros_like(y)
    for e, at in enumerate(ranges(bounds)):
        m = w[e].double()
        y[at] = x[at] @ m.t()
        err[at] = sum_eps(x.shape[1]) * (x[at].abs() @ m.abs().t())
    return y, rounded(y, err, io), err


def gated(x, w13, bounds, kind, io):
    """((out, bound), (gate_up, bound))."""
    gu, gu_bound, err = product(x, w13, bounds, io)
    I = w13.shape[1] // 2
    g, u, dg, du = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
    a = act(g, kind)
    out = a * u
    e = 1.13 * dg * (u.abs() + du) + a.abs() * du + 2.0 ** -20 * (g.abs() + a.abs()) * u.abs() + 2.0 ** -22 * out.abs()
    return (out, rounded(out, e, io)), (gu, gu_bound)


def input_grad(dy, dy_err, w, bounds, io):
    """(d_x, bound) for rows dy that are off by dy_err."""
    dx = torch.zeros((dy.shape[0], w.shape[2]), dtype=torch.float64)
    err = torch.zeros_like(dx)
    for e, at in enumerate(ranges(bounds)):
        m = w[e].double()
        dx[at] = dy[at] @ m
        err[at] = dy_err[at] @ m.abs() + sum_eps(dy.shape[1]) * ((dy[at].abs() + dy_err[at]) @ m.abs())
    return dx, rounded(dx, err, io)


def weight_grad(dy, dy_err, x, bounds, io, grad):
    """(d_w, bound); grad: the type of d_w."""
    dw = torch.zeros((len(bounds) - 1, dy.shape[1], x.shape[1]), dtype=torch.float64)
    err = torch.zeros_like(dw)
    x = x.double()
    for e, at in enumerate(ranges(bounds)):
        rows = at.stop - at.start
        dw[e] = dy[at].t() @ x[at]
        err[e] = dy_err[at].t() @ x[at].abs() + sum_eps(rows) * ((dy[at].abs() + dy_err[at]).t() @ x[at].abs())
    return dw, err + 2.0 ** -126 if grad == "fp32" else rounded(dw, err, io)


def few(rows, I):
    """Whether dg and du are held as sums of two 16-bit values."""
    return rows <= 64 and rows * (I + 56) <= 4096


def gate_grad(d_out, gate_up, kind, io):
    """([dg, du], bound) as the kernel holds them: rounded to the 16-bit type, or, where there are few, what is left rounded
    once more."""
    d, gu = d_out.double(), gate_up.double()
    I = d.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    a, s = act(g, kind), slope(g, kind)
    v = torch.cat((d * u * s, d * a), 1)
    err = 2.0 ** -20 * torch.cat(((d * u).abs() * (1 + g.abs()), d.abs() * (g.abs() + a.abs())), 1)
    if few(d.shape[0], I):
        return v, err + U[io] ** 2 * (v.abs() + err) + 2 * TINY[io]
    return v, rounded(v, err, io)


class Norm:
    """The block norm's forward values and gradients in 64 bits, with bounds.  c covers the fp32 roundings of a value that
    goes through a row's sums: a sum over H <= 16384 columns adds up at most 32 values a thread, then 5 + 4 levels, and
    a sum that comes out of cancellation is measured by the magnitudes that go into it."""

    c = 128 * 2.0 ** -24

    def __init__(self, y, residual, post, pre, gate, kind, block_scale, residual_scale, eps, bias, io):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        self.y, self.io, self.bias, self.bs, self.rs = d(y), io, bias, block_scale, residual_scale
        self.post = None if post is None else d(post) + bias
        self.pre = None if pre is None else d(pre) + bias
        self.kind = kind
        self.gate = torch.ones(1, 1).double() if gate is None else d(gate).view((-1, 1) if kind == "token" else (1, -1))
        self.ry = ((self.y ** 2).mean(1, keepdim=True) + eps) ** -0.5
        self.n = self.y * self.ry
        self.a = self.n * self.post if post is not None else self.y
        from_residual = 0 if residual is None else residual_scale * d(residual)
        block = block_scale * self.gate * self.a
        self.s = from_residual + block
        self.s_mag = torch.as_tensor(from_residual).abs() + block.abs()
        self.rr = ((self.s ** 2).mean(1, keepdim=True) + eps) ** -0.5
        self.m, self.m_mag = self.s * self.rr, self.s_mag * self.rr

    def forward(self):
        """((residual_out, bound), (norm_out, bound) or None)."""
        out = (self.s, rounded(self.s, self.c * self.s_mag, self.io))
        if self.pre is None:
            return out, None
        # the second norm's scale is off by what s is off by, in the root of the mean square
        rel = self.c * (1 + (self.s_mag ** 2).mean(1, keepdim=True).sqrt() * self.rr)
        x = self.m * self.pre
        return out, (x, rounded(x, rel * self.m_mag * self.pre.abs(), self.io))

    def backward(self, d_res, d_norm):
        """{name: (gradient, bound)}; the gradients of gammas and gates in fp32."""
        zero = torch.zeros_like(self.y)
        dr = zero if d_res is None else d_res.double()
        ds, mag = dr, dr.abs()
        out = {}
        T = self.y.shape[0]
        # a bound on how much larger the magnitudes behind s are than s itself
        grow = 1 + (self.s_mag ** 2).mean(1, keepdim=True).sqrt() * self.rr
        c = 4 * self.c * grow
        add = (T + 512) * 2.0 ** -24

        def total(v, m, err):
            return v.sum(0), (err * m).sum(0) + add * m.sum(0) + 2.0 ** -126

        if d_norm is not None:
            dx = d_norm.double()
            v = dx * self.pre
            ds = ds + self.rr * (v - self.m * (v * self.m).mean(1, keepdim=True))
            mag = mag + self.rr * (v.abs() + self.m_mag * (v.abs() * self.m_mag).mean(1, keepdim=True))
            out["d_pre"] = total(dx * self.m, dx.abs() * self.m_mag, c)
        dres = self.rs * ds
        out["d_residual"] = (dres, rounded(dres, c * abs(self.rs) * mag, self.io))
        w, wm = self.bs * self.a * ds, (self.bs * self.a).abs() * mag
        if self.kind == "token":
            out["d_gate"] = (w.sum(1), (c * wm).sum(1) + 2.0 ** -126)
        elif self.kind == "channel":
            out["d_gate"] = total(w, wm, c)
        da, dm = self.bs * self.gate * ds, (self.bs * self.gate).abs() * mag
        if self.post is None:
            dy, ym = da, dm
        else:
            out["d_post"] = total(da * self.n, dm * self.n.abs(), c)
            p, pm = da * self.post, dm * self.post.abs()
            dy = self.ry * (p - self.n * (p * self.n).mean(1, keepdim=True))
            ym = self.ry * (pm + self.n.abs() * (pm * self.n.abs()).mean(1, keepdim=True))
        out["d_y"] = (dy, rounded(dy, c * ym, self.io))
        return out
