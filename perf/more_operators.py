"""The feed-forward block for many tokens, forward and backward, as cases that can be timed.

Three operators and their gradients, which a layer runs one after the other between moe_dispatch_permute and
moe_combine (rows grouped by expert) or over all tokens (one expert: a dense block, a shared expert):

  gated    h = act(x W1^T) * (x W3^T)            rows of x [R, H], w13 = W1's I rows and then W3's for each expert
  linear   y = x W^T                             rows of x [R, K], w [E, N, K] (the block's second product)
  norm     s = rs * residual + bs * gate * N(y; post_gamma),  x = N(s; pre_gamma)
           the norms after one block and before the next, N(v; c) = v / sqrt(mean(v^2) + eps) * (c + weight_bias)

Row r belongs to expert e where offsets[e] <= r < offsets[e + 1]; rows from offsets[E] on belong to none and are left
as they were.  ``run`` computes them in plain torch operations, or (``own``) through norm_quant_gb300's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6

# What the largest listed cases take; a drawn case takes no more.
MOST_PRODUCTS = 32768 * 2 * 2048 * 7168
MOST_HELD = 256 * 2 * 2048 * 7168
MOST_ELEMENTS = 4096 * 7168


def _gated(name, R, H, inner, E, io="bf16", act="silu", save=False, behind=0.0, grad=False):
    return dict(name=name, op="gated_grad" if grad else "gated", R=R, H=H, I=inner, E=E, io=io, act=act, save=save,
                behind=behind)


def _linear(name, R, K, N, E, io="bf16", behind=0.0, grad=False):
    return dict(name=name, op="linear_grad" if grad else "linear", R=R, K=K, N=N, E=E, io=io, behind=behind)


def _norm(name, T, H, io="bf16", post=True, pre=True, gate="none", bias=0.0, block_scale=1.0, residual_scale=1.0,
          grad=False):
    return dict(name=name, op="norm_grad" if grad else "norm", T=T, H=H, io=io, post=post, pre=pre, gate=gate, bias=bias,
                block_scale=block_scale, residual_scale=residual_scale)


def listed():
    return [
        # the smallest layer of a few tokens over 8 experts, hidden 256: launch latency
        _gated("gated_R32_H256_I128_E8", 32, 256, 128, 8),
        # 4096 tokens of a prompt at top 8 of 256 experts: 128 rows an expert, so the weights' stream counts
        _gated("gated_R32768_H7168_I2048_E256", 32768, 7168, 2048, 256),
        # a training batch through a dense block: arithmetic alone
        _gated("gated_grad_R4096_H4096_I8192", 4096, 4096, 8192, 1, grad=True),
        # a training batch over small experts, odd rows, some experts empty, rows behind the last; GELU gates, fp16
        _gated("gated_grad_R8191_H2048_I1408_E64", 8191, 2048, 1408, 64, io="fp16", act="gelu_tanh", behind=0.05,
               grad=True),
        # a decode batch over more experts than it has rows for: the second product's weights are read once
        _linear("linear_R61_K1024_N4096_E128", 61, 1024, 4096, 128),
        # a prompt's second product, 256 rows an expert
        _linear("linear_R32768_K1024_N4096_E128", 32768, 1024, 4096, 128, io="fp16"),
        # a dense block's second product in training
        _linear("linear_grad_R8192_K8192_N4096", 8192, 8192, 4096, 1, grad=True),
        # few odd rows, odd widths
        _linear("linear_grad_R1021_K1400_N2056_E8", 1021, 1400, 2056, 8, io="fp16", grad=True),
        # one token's norms between two blocks: latency
        _norm("norm_T1_H7168", 1, 7168),
        # a prompt's, in the (1 + gamma) form
        _norm("norm_T8192_H4096", 8192, 4096, bias=1.0),
        # a training batch with a gate for each channel and a scaled residual
        _norm("norm_grad_T4096_H7168", 4096, 7168, gate="channel", residual_scale=0.75, grad=True),
        # odd rows and width, a gate for each token (a shared expert's)
        _norm("norm_grad_T1021_H2056", 1021, 2056, io="fp16", gate="token", block_scale=0.5, bias=1.0, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "linear", "linear_grad", "norm", "norm_grad"])
    io = rng.choice(["bf16", "fp16"])
    if op.startswith("norm"):
        H = max(1, _log(rng, 64, 16384) // 8) * 8
        post = rng.random() < 0.75
        c = _norm("", min(_log(rng, 1, 16384), MOST_ELEMENTS // H), H, io=io, post=post, pre=not post or rng.random() < 0.75,
                  gate=rng.choice(["none", "channel", "token"]), bias=rng.choice([0.0, 1.0]),
                  block_scale=rng.choice([1.0, 0.5]), residual_scale=rng.choice([1.0, 0.75]), grad=op == "norm_grad")
    else:
        grad = op.endswith("grad")
        while True:
            R = _log(rng, 1, 32768)
            E = rng.choice([1, 1, _log(rng, 2, 256), _log(rng, 2, 256)])
            a, b = (max(1, _log(rng, 64, hi) // 8) * 8 for hi in (7168, 8192))
            # rows of the fullest expert, times experts: what the plain form multiplies
            if E * (2 * R / E + 32) * a * b * 2 * (2 if grad else 1) <= MOST_PRODUCTS and \
                    E * a * b * 2 * (2 if grad else 1) <= MOST_HELD:
                break
        behind = rng.choice([0.0, 0.1])
        if op.startswith("gated"):
            c = _gated("", R, a, b, E, io=io, act=rng.choice(["silu", "gelu_tanh"]), save=not grad and rng.random() < 0.5,
                       behind=behind, grad=grad)
        else:
            c = _linear("", R, a, b, E, io=io, behind=behind, grad=grad)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------- inputs


def _counts(c, seed):
    """Rows of each expert: shares between 1 and 3 to each other, and of 8 experts or more a tenth has none."""
    rng = np.random.default_rng(int(seed))
    share = 0.5 + rng.random(c["E"])
    if c["E"] >= 8:
        share[rng.permutation(c["E"])[:c["E"] // 10]] = 0.0
    return rng.multinomial(c["R"] - int(c["R"] * c["behind"]), share / share.sum())


def prepare(case, seed):
    c = case
    dev, io = "cuda", DTYPE[c["io"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=c)

    def normal(*shape, std=1.0, dtype=io):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype).mul_(std)

    def empty(*shape, dtype=io):
        return torch.zeros(shape, device=dev, dtype=dtype)

    if c["op"].startswith("norm"):
        T, H = c["T"], c["H"]
        s["y"], s["residual"] = normal(T, H), normal(T, H, std=2.0)
        about = 1.0 - c["bias"]  # gamma + weight_bias is about 1
        for name in ("post", "pre"):
            s[name] = (about + 0.2 * torch.randn(H, generator=g, device=dev)).to(io) if c[name] else None
        s["gate"] = None
        if c["gate"] == "channel":
            s["gate"] = (0.5 + 0.3 * torch.randn(H, generator=g, device=dev)).to(io)
        elif c["gate"] == "token":
            s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device=dev))
        if c["op"] == "norm":
            s["residual_out"] = empty(T, H)
            s["norm_out"] = empty(T, H) if c["pre"] else None
        else:
            s["d_residual_out"] = normal(T, H)
            s["d_norm_out"] = normal(T, H) if c["pre"] else None
            s["d_y"], s["d_residual"] = empty(T, H), empty(T, H)
            for name in ("post", "pre"):
                s["d_" + name] = empty(H, dtype=torch.float32) if c[name] else None
            s["d_gate"] = None if s["gate"] is None else empty(*s["gate"].shape, dtype=torch.float32)
            # scratch for the column sums, as large as the library's size function asks at most
            s["workspace"] = torch.empty(12 * 1024 * H + 65536, device=dev, dtype=torch.uint8)
        return s

    R, E = c["R"], c["E"]
    counts = _counts(c, seed)
    bounds = np.concatenate([[0], np.cumsum(counts)])
    s["most"] = int(counts.max())
    s["bounds"] = [int(v) for v in bounds]
    s["offsets"] = torch.from_numpy(bounds.astype(np.int32)).to(dev)
    if c["op"].startswith("gated"):
        H, inner = c["H"], c["I"]
        s["x"], s["w"] = normal(R, H), normal(E, 2 * inner, H, std=H ** -0.5)
        if c["op"] == "gated":
            s["out"] = empty(R, inner)
            s["gate_up"] = empty(R, 2 * inner) if c["save"] else None
        else:
            # what the forward pass left: of the spread of x W^T
            s["gate_up"] = normal(R, 2 * inner)
            s["d_out"] = normal(R, inner)
            s["d_x"], s["d_w"] = empty(R, H), empty(E, 2 * inner, H)
            s["workspace"] = torch.empty(4 * R * inner + 65536, device=dev, dtype=torch.uint8)
    else:
        K, N = c["K"], c["N"]
        s["x"], s["w"] = normal(R, K), normal(E, N, K, std=K ** -0.5)
        if c["op"] == "linear":
            s["out"] = empty(R, N)
        else:
            s["d_out"] = normal(R, N)
            s["d_x"], s["d_w"] = empty(R, K), empty(E, N, K)
    return s


# ------------------------------------------------------------------------------------- the plain forms


class _Groups:
    """Rows [R, C] as [E, most, C], each expert's rows from its first on and zeros after them, and back."""

    def __init__(self, s, c):
        first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
        self.R, self.most = c["R"], max(1, s["most"])
        at = first[:, None] + torch.arange(self.most, device=first.device)
        self.inside = (at < last[:, None])[:, :, None]
        self.at = at.clamp(max=c["R"] - 1).reshape(-1)
        r = torch.arange(c["R"], device=first.device)
        e = torch.searchsorted(last, r, right=True).clamp(max=c["E"] - 1)
        self.back = (e * self.most + (r - first[e])).clamp(max=c["E"] * self.most - 1)
        self.taken = (r < last[-1])[:, None]

    def split(self, rows):
        return torch.where(self.inside, rows.float().index_select(0, self.at).view(-1, self.most, rows.shape[1]), 0.0)

    def join(self, groups, dtype):
        rows = groups.reshape(-1, groups.shape[2]).index_select(0, self.back)
        return torch.where(self.taken, rows, 0.0).to(dtype)


def _act(v, kind):
    """(act(v), its derivative) in elementary operations."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-v))
        return v * p, p * (1 + v * (1 - p))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def _plain_gated(s, c):
    groups, io, inner = _Groups(s, c), DTYPE[c["io"]], c["I"]
    gu = torch.bmm(groups.split(s["x"]), s["w"].float().transpose(1, 2))
    out = {"out": groups.join(_act(gu[:, :, :inner], c["act"])[0] * gu[:, :, inner:], io)}
    if c["save"]:
        out["gate_up"] = groups.join(gu, io)
    return out


def _plain_gated_grad(s, c):
    groups, io, inner = _Groups(s, c), DTYPE[c["io"]], c["I"]
    gu, dh = groups.split(s["gate_up"]), groups.split(s["d_out"])
    a, da = _act(gu[:, :, :inner], c["act"])
    dgu = torch.cat((dh * gu[:, :, inner:] * da, dh * a), 2)
    dx = torch.bmm(dgu, s["w"].float())
    dw = torch.bmm(dgu.transpose(1, 2), groups.split(s["x"]))
    return {"d_x": groups.join(dx, io), "d_w": dw.to(io)}


def _plain_linear(s, c):
    groups = _Groups(s, c)
    y = torch.bmm(groups.split(s["x"]), s["w"].float().transpose(1, 2))
    return {"out": groups.join(y, DTYPE[c["io"]])}


def _plain_linear_grad(s, c):
    groups, io = _Groups(s, c), DTYPE[c["io"]]
    dy = groups.split(s["d_out"])
    dx = torch.bmm(dy, s["w"].float())
    dw = torch.bmm(dy.transpose(1, 2), groups.split(s["x"]))
    return {"d_x": groups.join(dx, io), "d_w": dw.to(io)}


def _norm_parts(s, c, real):
    """The forward pass's values in the type `real`: y's normalised row and scale, the block's row before its gate,
    the gate, the new residual, its normalised row and scale."""
    y = s["y"].to(real)
    ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    n = y * ry
    a = n * (s["post"].to(real) + c["bias"]) if c["post"] else y
    gate = 1.0 if s["gate"] is None else s["gate"].to(real).view((-1, 1) if c["gate"] == "token" else (1, -1))
    r = c["residual_scale"] * s["residual"].to(real) + c["block_scale"] * gate * a
    rr = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
    return n, ry, a, gate, r, r * rr, rr


def _plain_norm(s, c):
    io = DTYPE[c["io"]]
    _, _, _, _, r, m, _ = _norm_parts(s, c, torch.float32)
    out = {"residual_out": r.to(io)}
    if c["pre"]:
        out["norm_out"] = (m * (s["pre"].float() + c["bias"])).to(io)
    return out


def _plain_norm_grad(s, c):
    io = DTYPE[c["io"]]
    n, ry, a, gate, _, m, rr = _norm_parts(s, c, torch.float32)
    out = {}
    dr = s["d_residual_out"].float()
    if c["pre"]:
        dx = s["d_norm_out"].float()
        u = dx * (s["pre"].float() + c["bias"])
        dr = dr + rr * (u - m * (u * m).mean(1, keepdim=True))
        out["d_pre"] = (dx * m).sum(0)
    out["d_residual"] = (c["residual_scale"] * dr).to(io)
    if s["gate"] is not None:
        out["d_gate"] = (c["block_scale"] * a * dr).sum(1 if c["gate"] == "token" else 0)
    dy = c["block_scale"] * gate * dr
    if c["post"]:
        out["d_post"] = (dy * n).sum(0)
        v = dy * (s["post"].float() + c["bias"])
        dy = ry * (v - n * (v * n).mean(1, keepdim=True))
    out["d_y"] = dy.to(io)
    return out


# ---------------------------------------------------------------------------------------- the library


def _own_gated(nqg, s, c):
    nqg.moe_gated_linear(s["x"], s["w"], s["out"], offsets=s["offsets"], gate_up=s["gate_up"], activation=c["act"],
                         io_dtype=c["io"])
    return {k: s[k] for k in ("out", "gate_up") if s[k] is not None}


def _own_gated_grad(nqg, s, c):
    nqg.moe_gated_linear_backward(s["d_out"], s["gate_up"], x=s["x"], w13=s["w"], d_x=s["d_x"], d_w13=s["d_w"],
                                  workspace=s["workspace"], offsets=s["offsets"], activation=c["act"], io_dtype=c["io"],
                                  grad_dtype=c["io"])
    return {"d_x": s["d_x"], "d_w": s["d_w"]}


def _own_linear(nqg, s, c):
    nqg.moe_grouped_linear(s["x"], s["w"], s["out"], offsets=s["offsets"], io_dtype=c["io"])
    return {"out": s["out"]}


def _own_linear_grad(nqg, s, c):
    nqg.moe_grouped_linear_backward(s["d_out"], x=s["x"], w=s["w"], d_x=s["d_x"], d_w=s["d_w"], offsets=s["offsets"],
                                    io_dtype=c["io"], grad_dtype=c["io"])
    return {"d_x": s["d_x"], "d_w": s["d_w"]}


def _norm_options(s, c):
    return dict(post_gamma=s["post"], pre_gamma=s["pre"], gate=s["gate"], gate_kind=c["gate"],
                block_scale=c["block_scale"], residual_scale=c["residual_scale"], eps=EPS, weight_bias=c["bias"],
                io_dtype=c["io"])


def _own_norm(nqg, s, c):
    nqg.moe_block_norm(s["y"], s["residual"], residual_out=s["residual_out"], norm_out=s["norm_out"], **_norm_options(s, c))
    return {k: s[k] for k in ("residual_out", "norm_out") if s[k] is not None}


def _own_norm_grad(nqg, s, c):
    nqg.moe_block_norm_backward(s["y"], s["residual"], d_residual_out=s["d_residual_out"], d_norm_out=s["d_norm_out"],
                                d_y=s["d_y"], d_residual=s["d_residual"], d_post_gamma=s["d_post"],
                                d_pre_gamma=s["d_pre"], d_gate=s["d_gate"], workspace=s["workspace"],
                                **_norm_options(s, c))
    return {k: s[k] for k in ("d_y", "d_residual", "d_post", "d_pre", "d_gate") if s[k] is not None}


def run(state):
    c = state["case"]
    if own:
        import norm_quant_gb300 as nqg
        call = {"gated": _own_gated, "gated_grad": _own_gated_grad, "linear": _own_linear, "linear_grad": _own_linear_grad,
                "norm": _own_norm, "norm_grad": _own_norm_grad}[c["op"]]
        return call(nqg, state, c)
    return {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "linear": _plain_linear,
            "linear_grad": _plain_linear_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[c["op"]](state, c)


# -------------------------------------------------------------------------------------- work and oracle


def work(case):
    c = case
    if c["op"].startswith("norm"):
        n, H = c["T"] * c["H"], c["H"]
        if c["op"] == "norm":
            return {"bytes": 2 * n * (3 + c["pre"]) + 4 * H, "flops": 12 * n}
        return {"bytes": 2 * n * (5 + c["pre"]) + 12 * H, "flops": 40 * n}
    R, E = c["R"] - int(c["R"] * c["behind"]), c["E"]
    open_ = E - (E // 10 if E >= 8 else 0)
    used = open_ * (1 - (1 - 1 / open_) ** R)  # experts that have rows
    if c["op"].startswith("gated"):
        a, b, products = c["H"], c["I"], 2
        rows = a + b + (2 * b if c["save"] else 0)
        grad_rows = 2 * a + b + 2 * b
    else:
        a, b, products = c["K"], c["N"], 1
        rows = a + b
        grad_rows = 2 * a + b
    if c["op"].endswith("grad"):
        # every expert's gradient is written, zeros where it has no rows
        return {"bytes": 2 * (products * a * b * (used + E) + R * grad_rows), "flops": 4 * products * R * a * b}
    return {"bytes": 2 * (products * a * b * used + R * rows), "flops": 2 * products * R * a * b}


def _exact_norm(s, c):
    """The two norms row by row from their definition, and the gradients by differentiation of them."""
    leaf = {k: s[k].double().requires_grad_(c["op"] == "norm_grad") for k in ("y", "residual", "post", "pre", "gate")
            if s[k] is not None}

    def norm(v, gamma):
        mean = torch.linalg.vector_norm(v, dim=1).square() / c["H"]
        return torch.einsum("th,t,h->th", v, (mean + EPS) ** -0.5, gamma + c["bias"])

    block = norm(leaf["y"], leaf["post"]) if c["post"] else leaf["y"]
    if c["gate"] != "none":
        block = torch.einsum("th,t->th" if c["gate"] == "token" else "th,h->th", block, leaf["gate"])
    out = {"residual_out": block * c["block_scale"] + leaf["residual"] * c["residual_scale"]}
    if c["pre"]:
        out["norm_out"] = norm(out["residual_out"], leaf["pre"])
    if c["op"] == "norm":
        return out
    d = torch.autograd.grad([out[k] for k in sorted(out)], list(leaf.values()), [s["d_" + k].double() for k in sorted(out)])
    return {"d_" + k: v for k, v in zip(leaf, d)}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(s, c)
    x = s["x"].double()
    out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("out", "gate_up", "d_x")
           if k in s and s[k] is not None and not (k == "gate_up" and c["op"] == "gated_grad")}
    grads = []
    for e in range(c["E"]):
        at = slice(s["bounds"][e], s["bounds"][e + 1])
        w = s["w"][e].double()
        if c["op"] == "linear":
            out["out"][at] = x[at] @ w.t()
            continue
        if c["op"] == "gated":
            gate, up = x[at] @ w[:c["I"]].t(), x[at] @ w[c["I"]:].t()
            if c["act"] == "silu":
                a = gate * torch.sigmoid(gate)
            else:
                a = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))
            out["out"][at] = a * up
            if c["save"]:
                out["gate_up"][at] = torch.cat((gate, up), 1)
            continue
        d = s["d_out"][at].double()
        if c["op"] == "gated_grad":
            gu = s["gate_up"][at].double().requires_grad_()
            gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
            if c["act"] == "silu":
                a = gate * torch.sigmoid(gate)
            else:
                a = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))
            d, = torch.autograd.grad((a * up * d).sum(), gu)
        out["d_x"][at] = d @ w
        # values of 16-bit results: 32 bits hold them far beyond what they are held to
        grads.append((d.t() @ x[at]).float())
    if grads:
        out["d_w"] = torch.stack(grads)
    return out
