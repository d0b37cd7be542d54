"""The serving operators of a mixture-of-experts layer for a few tokens, as cases that can be timed.

Three operators that a decode step runs one after the other:

  select   router logits [T, E] -> the top_k experts of each token and their weights
  linear   y = x W^T for a few rows x and a weight matrix held in 4 bits with group scales
           (a shared expert's or an attention projection's product)
  layer    out[t] = sum_j w[t, j] * W2[e] act(W1[e] x[t], W3[e] x[t]) over the token's experts
           e = ids[t, j], plus the shared expert's row and the residual

``run`` computes them in plain torch operations, or (``own``) through norm_quant_gb300's entry points.

4-bit weights hold element 2i of a row in the low nibble of byte i:
  nvfp4   e2m1 code times an e4m3 scale for every 16 elements, divided by one global scale
  int4    (code - zero) times a scale for every group_size elements; zero is 8 where none is given
"""
import math

import torch

own = False

DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)

# A drawn layer gathers at most this many fp32 weight elements in its plain form, and holds at most this
# many weight elements over all experts: the sizes of the largest listed layers.
MOST_GATHERED = 512 * 3 * 4096 * 1024
MOST_HELD = 256 * 3 * 7168 * 2048


def _select(name, T, E, k, logits="fp32", scoring="softmax", renormalize=True, scale=1.0, masked=0.0):
    return dict(name=name, op="select", T=T, E=E, k=k, logits=logits, scoring=scoring, renormalize=renormalize,
                scale=scale, masked=masked)


def _linear(name, M, N, K, fmt="nvfp4", group=16, zeros=False, io="bf16"):
    return dict(name=name, op="linear", M=M, N=N, K=K, fmt=fmt, group=group, zeros=zeros, io=io)


def _layer(name, T, H, inner, E, k, fmt="none", group=0, io="bf16", act="silu", zipf=0.0, pad=0.0, shared=True,
           residual=True):
    return dict(name=name, op="layer", T=T, H=H, I=inner, E=E, k=k, fmt=fmt, group=group, io=io, act=act, zipf=zipf,
                pad=pad, shared=shared, residual=residual)


def listed():
    return [
        # one token's routing among 256 experts: a launch and a chain of comparisons, latency alone
        _select("select_T1_E256_k8", 1, 256, 8),
        # a prefill batch's routing from 16-bit logits (many equal values), with padded tokens
        _select("select_T16384_E256_k8", 16384, 256, 8, logits="bf16", masked=0.1),
        # sigmoid scores of a batch of odd length over an odd number of experts
        _select("select_T1021_E161_k6", 1021, 161, 6, scoring="sigmoid", scale=2.5, masked=0.02),
        # one token through a shared expert's up projection
        _linear("linear_M1_N2048_K7168", 1, 2048, 7168),
        # one token through a wide projection: the whole of it is the weights' stream
        _linear("linear_M1_N16384_K7168", 1, 16384, 7168),
        # a small batch of odd length, odd rows, 4-bit integers with zero points, fp16
        _linear("linear_M5_N7001_K4096_int4", 5, 7001, 4096, fmt="int4", group=128, zeros=True, io="fp16"),
        # the largest batch that these products take
        _linear("linear_M64_N7168_K7168_int4", 64, 7168, 7168, fmt="int4", group=64),
        # the smallest layer: 16 tokens over 8 experts of hidden 256, launch latency
        _layer("layer_T16_H256_E8_k2", 16, 256, 128, 8, 2, shared=False, residual=False),
        # one token of a large model in bf16: eight experts' weights are read once
        _layer("layer_T1_H7168_E256_k8", 1, 7168, 2048, 256, 8),
        # a decode batch over the same experts held in 4 bits, skewed routing, some tokens padded
        _layer("layer_T16_H7168_E256_k8_nvfp4", 16, 7168, 2048, 256, 8, fmt="nvfp4", group=16, zipf=1.1, pad=0.1),
        # a decode batch that reads almost every expert; GELU gates, fp16
        _layer("layer_T64_H4096_E128_k8_fp16", 64, 4096, 1024, 128, 8, io="fp16", act="gelu_tanh"),
        # few large experts, so that several tokens share each, in 4-bit integers
        _layer("layer_T8_H4096_E8_k2_int4", 8, 4096, 8192, 8, 2, fmt="int4", group=128, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "linear", "linear", "layer", "layer"])
    if op == "select":
        E = _log(rng, 4, 512)
        c = _select("", _log(rng, 1, 16384), E, rng.randint(1, min(8, E)), logits=rng.choice(["fp32", "bf16", "fp16"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]))
    elif op == "linear":
        fmt = rng.choice(["nvfp4", "int4"])
        group = 16 if fmt == "nvfp4" else rng.choice([64, 128])
        K = max(1, _log(rng, 256, 16384) // group) * group
        c = _linear("", _log(rng, 1, 64), min(_log(rng, 64, 16384), 16384 * 7168 // K), K, fmt=fmt, group=group,
                    zeros=fmt == "int4" and rng.random() < 0.5, io=rng.choice(["bf16", "fp16"]))
    else:
        while True:
            fmt = rng.choice(["none", "nvfp4", "int4"])
            group = {"none": 0, "nvfp4": 16, "int4": rng.choice([64, 128])}[fmt]
            unit = group or 8
            T, E = _log(rng, 1, 64), _log(rng, 4, 256)
            H, inner = (max(1, _log(rng, 256, hi) // unit) * unit for hi in (7168, 8192))
            k = rng.randint(1, min(8, E))
            if T * k * 3 * H * inner <= MOST_GATHERED and E * 3 * H * inner <= MOST_HELD:
                break
        c = _layer("", T, H, inner, E, k, fmt=fmt, group=group, io=rng.choice(["bf16", "fp16"]),
                   act=rng.choice(["silu", "gelu_tanh"]), zipf=rng.choice([0.0, 1.1]), pad=rng.choice([0.0, 0.1]),
                   shared=rng.random() < 0.5, residual=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------- inputs


def _weights(g, s, name, shape, c, std):
    """A weight matrix [.., N, K] of standard deviation about `std`, in the case's format, as state entries."""
    dev = "cuda"
    io = DTYPE[c["io"]]
    if c["fmt"] == "none":
        s[name] = torch.randn(shape, generator=g, device=dev, dtype=io).mul_(std)
        return
    packed = (*shape[:-1], shape[-1] // 2)
    groups = (*shape[:-1], shape[-1] // c["group"])
    s[name] = torch.randint(0, 256, packed, generator=g, device=dev, dtype=torch.uint8)
    if c["fmt"] == "nvfp4":
        # e4m3 codes 0x68..0x7e: scales 64 to 448, the upper end as quantisers that use a global scale give them;
        # the root of the mean square of the 16 codes is 3.0, that of the scales about 221
        s[name + "_scales"] = torch.randint(0x68, 0x7F, groups, generator=g, device=dev, dtype=torch.uint8)
        s[name + "_global"] = (3.0 * 221 / std) * (0.75 + 0.5 * torch.rand(shape[:-2] or (1,), generator=g, device=dev))
    else:
        # the root of the mean square of (code - 8) is 4.6
        s[name + "_scales"] = (torch.rand(groups, generator=g, device=dev).add_(0.5) * (std / 4.8)).to(io)
        if c.get("zeros"):
            s[name + "_zeros"] = torch.randint(6, 11, groups, generator=g, device=dev, dtype=torch.uint8)


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "select":
        T, E, k = c["T"], c["E"], c["k"]
        logits = torch.randn((T, E), generator=g, device=dev) * 1.5
        # padded tokens have no expert open to them: every logit -inf
        pad = torch.rand((T, 1), generator=g, device=dev) < c["masked"]
        s["logits"] = logits.masked_fill_(pad, -math.inf).to(DTYPE[c["logits"]])
        s["ids"] = torch.empty((T, k), device=dev, dtype=torch.int32)
        s["weights"] = torch.empty((T, k), device=dev, dtype=torch.float32)
    elif c["op"] == "linear":
        M, N, K, io = c["M"], c["N"], c["K"], DTYPE[c["io"]]
        s["x"] = torch.randn((M, K), generator=g, device=dev).to(io)
        _weights(g, s, "w", (N, K), c, K ** -0.5)
        if c["fmt"] == "nvfp4":
            s["global_scale"] = float(s["w_global"].item())
        s["out"] = torch.empty((M, N), device=dev, dtype=io)
    else:
        T, H, inner, E, k, io = c["T"], c["H"], c["I"], c["E"], c["k"], DTYPE[c["io"]]
        s["x"] = torch.randn((T, H), generator=g, device=dev).to(io)
        _weights(g, s, "w13", (E, 2 * inner, H), c, H ** -0.5)
        _weights(g, s, "w2", (E, H, inner), c, inner ** -0.5)
        # k distinct experts for each token, p(e) ~ (e + 1)^-zipf, by the largest Gumbel-perturbed logits
        u = torch.rand((T, E), generator=g, device=dev).clamp_(1e-9, 1 - 1e-7)
        key = -torch.log(-torch.log(u)) - c["zipf"] * torch.log(torch.arange(1, E + 1, device=dev).float())
        ids = key.topk(k, dim=1).indices.to(torch.int32)
        w = torch.softmax(torch.randn((T, k), generator=g, device=dev), dim=1)
        pad = torch.rand((T, 1), generator=g, device=dev) < c["pad"]
        s["ids"] = ids.masked_fill_(pad, -1).contiguous()
        s["weights"] = w.masked_fill_(pad, 0.0).contiguous()
        s["shared"] = torch.randn((T, H), generator=g, device=dev).mul_(0.5).to(io) if c["shared"] else None
        s["residual"] = torch.randn((T, H), generator=g, device=dev).to(io) if c["residual"] else None
        s["out"] = torch.empty((T, H), device=dev, dtype=io)
        # scratch for the gated products of every (token, slot), as large as the library's size function asks at most
        s["workspace"] = torch.empty(4 * T * k * inner + 65536, device=dev, dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------------------- the plain forms


def _plain_select(s, c):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    # the largest first; equal logits keep the order of their index
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    taken = top > -math.inf
    if c["scoring"] == "softmax":
        most = top[:, :1].clamp(-3e38, 3e38)
        w = torch.exp(top - most)
        total = w.sum(1, keepdim=True) if c["renormalize"] else torch.exp(x - most).sum(1, keepdim=True)
        w = w / total
    else:
        w = 1 / (1 + torch.exp(-top))
        if c["renormalize"]:
            w = w / w.sum(1, keepdim=True)
    w = torch.where(taken, w * c["scale"], 0.0)
    return {"ids": torch.where(taken, ids, -1).to(torch.int32), "weights": w}


def _widen(s, name, c, at=None):
    """The fp32 values of a weight matrix, or of the experts `at` of a stack of them."""
    pick = (lambda t: t) if at is None else (lambda t: t.index_select(0, at))
    w = pick(s[name])
    if c["fmt"] == "none":
        return w.float()
    if c["fmt"] == "nvfp4":
        one = torch.tensor(E2M1, device=w.device)
    else:
        one = torch.arange(16, device=w.device, dtype=torch.float32)
    byte = torch.stack((one.repeat(16), one.repeat_interleave(16)), 1)  # the two elements of a byte
    v = byte.index_select(0, w.reshape(-1).int()).view(*w.shape[:-1], -1, c["group"])
    if c["fmt"] == "nvfp4":
        scale = pick(s[name + "_scales"]).view(torch.float8_e4m3fn).float()
        g = pick(s[name + "_global"])
        v.mul_(scale.unsqueeze(-1)).div_(g.view(-1, *[1] * (v.dim() - 1)) if at is not None else g)
    else:
        zeros = s.get(name + "_zeros")
        v.sub_(8.0 if zeros is None else pick(zeros).float().unsqueeze(-1))
        v.mul_(pick(s[name + "_scales"]).float().unsqueeze(-1))
    return v.flatten(-2)


def _plain_linear(s, c):
    return (s["x"].float() @ _widen(s, "w", c).t()).to(DTYPE[c["io"]])


def _plain_layer(s, c):
    T, H, inner, k = c["T"], c["H"], c["I"], c["k"]
    taken = s["ids"] >= 0
    at = s["ids"].clamp(min=0).reshape(-1)
    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
    gu = torch.bmm(_widen(s, "w13", c, at), x)
    gate, up = gu[:, :inner], gu[:, inner:]
    if c["act"] == "silu":
        a = gate / (1 + torch.exp(-gate))
    else:
        a = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)))
    y = torch.bmm(_widen(s, "w2", c, at), a * up).view(T, k, H)
    y = torch.where(taken.unsqueeze(2), y * s["weights"].unsqueeze(2), 0.0).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPE[c["io"]])


# ---------------------------------------------------------------------------------------- the library


def _own_select(nqg, s, c):
    nqg.moe_select_experts(s["logits"], s["ids"], s["weights"], scoring=c["scoring"], renormalize=c["renormalize"],
                           scale=c["scale"], logits_dtype=c["logits"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _own_linear(nqg, s, c):
    nqg.moe_linear_w4(s["x"], s["w"], s["w_scales"], s["out"], w_format=c["fmt"], group_size=c["group"],
                      zeros=s.get("w_zeros"), global_scale=s.get("global_scale", 1.0), io_dtype=c["io"])
    return s["out"]


def _own_layer(nqg, s, c):
    nqg.moe_layer(x=s["x"], topk_ids=s["ids"], router_weights=s["weights"], w13=s["w13"], w2=s["w2"],
                  w13_scales=s.get("w13_scales"), w2_scales=s.get("w2_scales"), w13_global=s.get("w13_global"),
                  w2_global=s.get("w2_global"), w_format=c["fmt"], group_size=c["group"], activation=c["act"],
                  shared_out=s["shared"], residual=s["residual"], out=s["out"], workspace=s["workspace"],
                  io_dtype=c["io"])
    return s["out"]


def run(state):
    c = state["case"]
    if own:
        import norm_quant_gb300 as nqg
        call = {"select": _own_select, "linear": _own_linear, "layer": _own_layer}[c["op"]]
        return call(nqg, state, c)
    return {"select": _plain_select, "linear": _plain_linear, "layer": _plain_layer}[c["op"]](state, c)


# -------------------------------------------------------------------------------------- work and oracle


def _bytes_per_weight(c):
    if c["fmt"] == "none":
        return 2.0
    if c["fmt"] == "nvfp4":
        return 0.5 + 1 / 16
    return 0.5 + (3 if c.get("zeros") else 2) / c["group"]


def work(case):
    c = case
    if c["op"] == "select":
        size = {"fp32": 4, "bf16": 2, "fp16": 2}[c["logits"]]
        return {"bytes": c["T"] * (c["E"] * size + c["k"] * 8), "flops": c["T"] * c["E"] * 2}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * _bytes_per_weight(c) + 2 * M * (N + K), "flops": 2 * M * N * K}
    T, H, inner, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    tokens = T * (1 - c["pad"])
    # experts that at least one token takes: with p(e) the chance that one of k draws is e
    p = [(e + 1.0) ** -c["zipf"] for e in range(E)]
    total = sum(p)
    used = sum(1 - (1 - min(1.0, k * v / total)) ** tokens for v in p)
    used = min(used, tokens * k, E)
    rows = 2 + (1 if c["shared"] else 0) + (1 if c["residual"] else 0)
    return {"bytes": used * 3 * H * inner * _bytes_per_weight(c) + 2 * T * H * rows + T * k * 8,
            "flops": 6 * tokens * k * H * inner}


def _exact_matrix(s, name, c, e=None):
    """One weight matrix in float64 from the format's definition."""
    one = (lambda t: t) if e is None else (lambda t: t[e])
    w = one(s[name])
    if c["fmt"] == "none":
        return w.double()
    code = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.int32, device=w.device)
    code[:, 0::2] = w % 16
    code[:, 1::2] = w // 16
    scale = one(s[name + "_scales"])
    if c["fmt"] == "int4":
        z = one(s[name + "_zeros"]).double().repeat_interleave(c["group"], 1) if name + "_zeros" in s else 8.0
        return (code.double() - z) * scale.double().repeat_interleave(c["group"], 1)
    mag, neg = code % 8, code >= 8
    field, man = mag // 2, (mag % 2).double()
    v = torch.where(field == 0, 0.5 * man, (1 + 0.5 * man) * torch.pow(2.0, field.double() - 1))
    v = torch.where(neg, -v, v)
    sc = scale.int()
    f, m = (sc // 8) % 16, (sc % 8).double()
    sv = torch.where(f == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, f.double() - 7))
    g = float(s[name + "_global"].reshape(-1)[0 if e is None else e])
    return v * sv.repeat_interleave(16, 1) / g


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "select":
        x = s["logits"].double().cpu()
        w = torch.zeros((c["T"], c["k"]), dtype=torch.float64)
        left = x.clone()
        rows = torch.arange(c["T"])
        score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
        for j in range(c["k"]):
            i = left.argmax(1)
            open_ = left[rows, i] > -math.inf
            w[:, j] = torch.where(open_, score[rows, i], 0.0)
            left[rows, i] = -math.inf
        if c["renormalize"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0.0)
        return {"ids": None, "weights": w * c["scale"]}
    if c["op"] == "linear":
        return s["x"].double() @ _exact_matrix(s, "w", c).t()
    x, ids, rw = s["x"].double(), s["ids"].cpu(), s["weights"].double()
    out = torch.zeros_like(x)
    for extra in (s["shared"], s["residual"]):
        if extra is not None:
            out += extra.double()
    for e in sorted(set(ids.reshape(-1).tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        t, j = t.cuda(), j.cuda()
        h = x[t] @ _exact_matrix(s, "w13", c, e).t()
        a, b = h[:, :c["I"]], h[:, c["I"]:]
        a = a * torch.sigmoid(a) if c["act"] == "silu" else 0.5 * a * (
            1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
        y = (a * b) @ _exact_matrix(s, "w2", c, e).t()
        out.index_add_(0, t, rw[t, j].unsqueeze(1) * y)
    return out
