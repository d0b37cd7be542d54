"""The block's operators for many tokens on the GPU against 64-bit references:
grouped rows with empty and ragged experts, strides, rows of no expert, odd
widths, non-finite neighbours, bad offsets, graphs and streams."""
import pytest
import torch

import norm_quant_gb300 as nqg
from norm_quant_gb300.build import build

import _block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
CANARY = 13.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    nqg.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, io="bf16", std=1.0):
    return (torch.randn(shape, generator=g) * std).to(ref.IO[io])


def strided(t, extra):
    """t on the GPU, its rows `extra` elements apart from each other, with canaries between them."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), CANARY, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t.to(DEV)
    return wide[:, :t.shape[1]]


class Out:
    """A matrix of rows to be written, inside canaries."""

    def __init__(self, rows, width, io, extra=0, dtype=None):
        self.buf = torch.full((rows + 4, width + extra), CANARY, dtype=dtype or ref.IO[io], device=DEV)
        self.view = self.buf[2:rows + 2, :width]
        self.width = width

    def check(self, want, bound, bounds):
        got = self.buf.cpu()
        edge = [*got[:2].flatten(), *got[-2:].flatten(), *got[:, self.width:].flatten()]
        assert all(v == CANARY for v in edge), "written outside the rows"
        got = got[2:-2, :self.width]
        assert bool((got[:bounds[0]] == CANARY).all()) and bool((got[bounds[-1]:] == CANARY).all()), "rows of no expert"
        at = slice(bounds[0], bounds[-1])
        near(got[at], want[at], bound[at])


def near(got, want, bound):
    """|got - want| <= bound; a value beyond the type's range rounds to an infinity."""
    most = torch.finfo(got.dtype).max if got.dtype != torch.float64 else torch.inf
    got = got.cpu().double()
    beyond = (want.abs() + bound > most) & got.isinf() & (got.sign() == want.sign())
    got = torch.where(beyond, want, got)
    over = (got - want).abs() - bound
    assert bool((over <= 0).all()), (float(over.max()), int((~(over <= 0)).sum()), got.shape)


def dev_offsets(bounds):
    return torch.tensor(bounds, dtype=torch.int32, device=DEV)


# rows of each expert, as offsets; the last are rows of no expert behind (and before) the others
GROUPS = {
    "one": ([0, 1], 1),
    "dense": ([0, 130], 130),
    "tile": ([0, 256, 512], 512),
    "over": ([0, 257, 300, 301], 301),
    "ragged": ([0, 0, 7, 7, 140, 269, 270, 270], 281),
    "before": ([5, 69, 100], 117),
    "none": ([0, 0, 0], 9),
    "few": ([2, 5, 5, 20], 22),
    "many": ([0] + [3 * (i // 2) + (i % 7) * 0 for i in range(1, 41)], 64),
}
SIZES = [(8, 8), (64, 64), (72, 40), (136, 200), (256, 128), (520, 264), (200, 1000)]


def groups_of(name):
    bounds, rows = GROUPS[name]
    return bounds, rows, len(bounds) - 1


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("H,I", SIZES)
def test_gated_linear(H, I, name, io):
    bounds, rows, E = groups_of(name)
    g = gen(H * I + rows)
    x, w = normal(g, rows, H, io=io), normal(g, E, 2 * I, H, io=io, std=H ** -0.5)
    kind = "silu" if (H + rows) % 16 else "gelu_tanh"
    (out, bound), (gu, gu_bound) = ref.gated(x, w, bounds, kind, io)
    extra = 8 * (rows % 3)
    for save in (False, True):
        o, s = Out(rows, I, io, extra), Out(rows, 2 * I, io, extra) if save else None
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        nqg.moe_gated_linear(strided(x, extra), w.to(DEV), o.view, offsets=dev_offsets(bounds),
                             gate_up=s.view if save else None, activation=kind, status=status, io_dtype=io)
        o.check(out, bound, bounds)
        if save:
            s.check(gu, gu_bound, bounds)
        assert int(status) == 0


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("K,N", SIZES)
def test_grouped_linear(K, N, name, io):
    bounds, rows, E = groups_of(name)
    g = gen(K * N + rows + 1)
    x, w = normal(g, rows, K, io=io), normal(g, E, N, K, io=io, std=K ** -0.5)
    y, bound, _ = ref.product(x, w, bounds, io)
    o = Out(rows, N, io, 16)
    nqg.moe_grouped_linear(strided(x, 8), w.to(DEV), o.view, offsets=dev_offsets(bounds), io_dtype=io)
    o.check(y, bound, bounds)


def check_linear_backward(bounds, rows, K, N, io, grad, extra=8):
    E = len(bounds) - 1
    g = gen(K * N + rows + 2)
    x, w, dy = normal(g, rows, K, io=io), normal(g, E, N, K, io=io, std=K ** -0.5), normal(g, rows, N, io=io)
    zero = torch.zeros(rows, N, dtype=torch.float64)
    dx, dx_bound = ref.input_grad(dy.double(), zero, w, bounds, io)
    dw, dw_bound = ref.weight_grad(dy.double(), zero, x, bounds, io, grad)
    o = Out(rows, K, io, extra)
    dt = torch.float32 if grad == "fp32" else ref.IO[io]
    gw = Out(E * N, K, io, dtype=dt)
    got_w = gw.buf[2:-2].view(E, N, K)
    nqg.moe_grouped_linear_backward(strided(dy, extra), x=strided(x, extra), w=w.to(DEV), d_x=o.view, d_w=got_w,
                                    offsets=dev_offsets(bounds), io_dtype=io, grad_dtype=grad)
    o.check(dx, dx_bound, bounds)
    gw.check(dw.flatten(0, 1), dw_bound.flatten(0, 1), [0, E * N])
    return g, x, w, dy, o, got_w


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("K,N", SIZES)
def test_grouped_linear_backward(K, N, name, io):
    bounds, rows, E = groups_of(name)
    grad = io if (K + rows) % 3 else "fp32"
    g, x, w, dy, o, got_w = check_linear_backward(bounds, rows, K, N, io, grad)
    # each gradient alone
    one = torch.full((rows, K), CANARY, dtype=ref.IO[io], device=DEV)
    nqg.moe_grouped_linear_backward(dy.to(DEV), w=w.to(DEV), d_x=one, offsets=dev_offsets(bounds), io_dtype=io)
    assert torch.equal(one, o.view)
    two = torch.full_like(got_w, CANARY)
    nqg.moe_grouped_linear_backward(dy.to(DEV), x=x.to(DEV), d_w=two, offsets=dev_offsets(bounds), io_dtype=io, grad_dtype=grad)
    assert torch.equal(two, got_w)


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("name,H,I", [("one", 64, 72), ("ragged", 136, 200), ("before", 72, 40), ("over", 256, 128),
                                      ("none", 64, 64), ("many", 200, 96), ("few", 136, 72),
                                      ("few", 520, 128), ("few", 64, 8), ("over", 72, 8)])
def test_gated_linear_backward(name, H, I, kind, io):
    bounds, rows, E = groups_of(name)
    g = gen(H + I + rows)
    x, w = normal(g, rows, H, io=io), normal(g, E, 2 * I, H, io=io, std=H ** -0.5)
    gu, d = normal(g, rows, 2 * I, io=io, std=2.0), normal(g, rows, I, io=io)
    dgu, err = ref.gate_grad(d, gu, kind, io)
    dx, dx_bound = ref.input_grad(dgu, err, w, bounds, io)
    for grad in (io, "fp32"):
        dw, dw_bound = ref.weight_grad(dgu, err, x, bounds, io, grad)
        o = Out(rows, H, io, 8)
        gw = torch.full((E, 2 * I, H), CANARY, dtype=torch.float32 if grad == "fp32" else ref.IO[io], device=DEV)
        ws = torch.full((nqg.moe_gated_linear_backward_workspace_size(rows, I),), 255, dtype=torch.uint8, device=DEV)
        nqg.moe_gated_linear_backward(strided(d, 8), strided(gu, 16), x=strided(x, 8), w13=w.to(DEV), d_x=o.view, d_w13=gw,
                                      workspace=ws, offsets=dev_offsets(bounds), activation=kind, io_dtype=io, grad_dtype=grad)
        o.check(dx, dx_bound, bounds)
        near(gw, dw, dw_bound)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_gradients_against_differences(kind):
    """Along random directions: the kernels' gradients against central differences of the 64-bit forward formulas."""
    bounds, rows, H, I = [0, 3, 20], 20, 40, 24
    g = gen(7)
    x, w, d = normal(g, rows, H), normal(g, 2, 2 * I, H, std=H ** -0.5), normal(g, rows, I)
    gu = torch.empty((rows, 2 * I), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((rows, I), dtype=torch.bfloat16, device=DEV)
    off = dev_offsets(bounds)
    nqg.moe_gated_linear(x.to(DEV), w.to(DEV), out, offsets=off, gate_up=gu, activation=kind)
    dx, dw = torch.empty_like(x, device=DEV), torch.empty((2, 2 * I, H), dtype=torch.float32, device=DEV)
    ws = torch.empty(nqg.moe_gated_linear_backward_workspace_size(rows, I), dtype=torch.uint8, device=DEV)
    nqg.moe_gated_linear_backward(d.to(DEV), gu, x=x.to(DEV), w13=w.to(DEV), d_x=dx, d_w13=dw, workspace=ws, offsets=off,
                                  activation=kind, grad_dtype="fp32")

    def loss(x, w):
        return sum(float((d[at].double() * ref.act(x[at] @ w[e][:I].t(), kind) * (x[at] @ w[e][I:].t())).sum())
                   for e, at in enumerate(ref.ranges(bounds)))

    h = 1e-5
    for seed in range(4):
        vx, vw = torch.randn(x.shape, generator=gen(seed)).double(), torch.randn(w.shape, generator=gen(seed + 9)).double()
        for a, b, got in ((vx, 0 * vw, (dx.cpu().double() * vx)), (0 * vx, vw, (dw.cpu().double() * vw))):
            want = (loss(x.double() + h * a, w.double() + h * b) - loss(x.double() - h * a, w.double() - h * b)) / (2 * h)
            # gate_up, dg, du and d_x are rounded to bf16: four relative errors of at most 2^-8 in each of the terms,
            # whose signs are independent, so the sum is off by far less than by 4 2^-8 of the sum of their magnitudes
            assert abs(float(got.sum()) - want) <= 4 * 2.0 ** -8 * float(got.abs().sum())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_with_their_rows_and_experts(bad):
    """Rows of no expert, neighbouring experts' rows and weights, and what lies behind the tensors' last column."""
    bounds, rows, K, N = [3, 40, 40, 111, 130], 140, 72, 144
    E = len(bounds) - 1
    g = gen(11)
    x, w, dy = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5), normal(g, rows, N)
    xs, ds = (torch.full((rows, n + 8), bad, dtype=torch.bfloat16, device=DEV) for n in (K, N))
    xs[:, :K], ds[:, :N] = x.to(DEV), dy.to(DEV)
    for t in (xs, ds):
        t[:3] = t[130:] = bad
        t[40:111] = bad      # the rows of expert 2, and expert 2's weights
    wd = w.to(DEV)
    wd[1:3] = bad            # expert 1 has no rows
    off = dev_offsets(bounds)
    out, dx = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV), torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((E, N, K), dtype=torch.float32, device=DEV)
    nqg.moe_grouped_linear(xs[:, :K], wd, out, offsets=off)
    nqg.moe_grouped_linear_backward(ds[:, :N], x=xs[:, :K], w=wd, d_x=dx, d_w=dw, offsets=off, grad_dtype="fp32")
    gated = torch.zeros((rows, N // 2), dtype=torch.bfloat16, device=DEV)
    nqg.moe_gated_linear(xs[:, :K], wd, gated, offsets=off)
    for at in (slice(3, 40), slice(111, 130)):
        for t in (out, dx, gated):
            assert bool(t[at].isfinite().all())
    assert not bool(out[40:111].isfinite().any()) and not bool(dx[40:111].isfinite().any())
    assert bool(dw[[0, 1, 3]].isfinite().all()) and not bool(dw[2].isfinite().any())
    assert bool((dw[1] == 0).all())
    for t in (out, dx, gated):
        assert bool((t[:3] == 0).all()) and bool((t[130:] == 0).all())


@pytest.mark.parametrize("bad,meant", [([0, 50, 40, 80], [0, 50, 50, 80]), ([0, 50, 60, 200], [0, 50, 60, 80]),
                                       ([-5, 50, 60, 70], [0, 50, 60, 70]), ([90, 95, 99, 100], [80, 80, 80, 80])])
def test_offsets_out_of_order_or_range(bad, meant):
    """Each one that lies below an earlier one counts as that, each outside the rows as the nearer end, and *status says so."""
    rows, K, N = 80, 64, 72
    g = gen(5)
    x, w, dy = normal(g, rows, K), normal(g, 3, N, K, std=K ** -0.5), normal(g, rows, N)
    y, bound, _ = ref.product(x, w, meant, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = Out(rows, N, "bf16")
    nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bad), status=status)
    o.check(y, bound, meant)
    assert int(status) == nqg.MOE_ERR_ROW_OUT_OF_RANGE
    zero = torch.zeros(rows, N, dtype=torch.float64)
    dx, dx_bound = ref.input_grad(dy.double(), zero, w, meant, "bf16")
    dw, dw_bound = ref.weight_grad(dy.double(), zero, x, meant, "bf16", "bf16")
    d = Out(rows, K, "bf16")
    gw = torch.full((3, N, K), CANARY, dtype=torch.bfloat16, device=DEV)
    status.zero_()
    nqg.moe_grouped_linear_backward(dy.to(DEV), x=x.to(DEV), w=w.to(DEV), d_x=d.view, d_w=gw, offsets=dev_offsets(bad), status=status)
    d.check(dx, dx_bound, meant)
    near(gw, dw, dw_bound)
    assert int(status) == nqg.MOE_ERR_ROW_OUT_OF_RANGE


@pytest.mark.parametrize("E", [31, 32, 287, 288, 700])
def test_offsets_of_many_experts_out_of_order(E):
    """The same, where a lane reads several offsets and there are several turns of them."""
    rows, K, N = 90, 64, 72
    g = gen(E)
    bad = torch.randint(0, rows + 1, (E + 1,), generator=g).sort().values
    wrong = torch.randint(0, E + 1, (E // 10,), generator=g)
    bad[wrong] = torch.randint(-20, rows + 20, (E // 10,), generator=g)
    meant = bad.clamp(0, rows).cummax(0).values.tolist()
    x, w, dy = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5), normal(g, rows, N)
    for given, code in ((bad.tolist(), nqg.MOE_ERR_ROW_OUT_OF_RANGE if meant != bad.tolist() else 0), (meant, 0)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, dw = Out(rows, N, "bf16"), torch.full((E, N, K), CANARY, dtype=torch.float32, device=DEV)
        nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(given), status=status)
        assert int(status) == code
        y, bound, _ = ref.product(x, w, meant, "bf16")
        o.check(y, bound, meant)
        status.zero_()
        nqg.moe_grouped_linear_backward(dy.to(DEV), x=x.to(DEV), d_w=dw, offsets=dev_offsets(given), status=status, grad_dtype="fp32")
        assert int(status) == code
        want, bound = ref.weight_grad(dy.double(), torch.zeros(rows, N, dtype=torch.float64), x, meant, "bf16", "fp32")
        near(dw, want, bound)


def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    off = dev_offsets([0, 0, 0])
    nqg.moe_gated_linear(e(0, 64), e(2, 32, 64), e(0, 16), offsets=off)
    nqg.moe_grouped_linear(e(0, 64), e(2, 32, 64), e(0, 32), offsets=off)
    for grad, dt in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        dw = torch.full((2, 32, 64), CANARY, dtype=dt, device=DEV)
        nqg.moe_grouped_linear_backward(e(0, 32), x=e(0, 64), w=e(2, 32, 64), d_x=e(0, 64), d_w=dw, offsets=off, grad_dtype=grad)
        assert bool((dw == 0).all())
        dw.fill_(CANARY)
        nqg.moe_gated_linear_backward(e(0, 16), e(0, 32), x=e(0, 64), d_w13=dw, offsets=off, grad_dtype=grad)
        assert bool((dw == 0).all())


# larger sizes, where tiles, pipelines and waves wrap; only what 64 bits take little time for
@pytest.mark.parametrize("rows,K,N,E", [(1000, 1024, 2048, 1), (777, 2056, 1392, 3), (1500, 520, 4096, 24), (3, 7168, 2048, 2),
                                        (40, 4096, 1040, 1)])
def test_larger_products(rows, K, N, E):
    cuts = torch.randint(0, rows + 1, (E - 1,), generator=gen(rows)).sort().values.tolist()
    bounds = [0, *cuts, rows - rows // 50]
    bounds = [min(b, bounds[-1]) for b in bounds]
    g = gen(K)
    x, w = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5)
    y, bound, _ = ref.product(x, w, bounds, "bf16")
    o = Out(rows, N, "bf16")
    nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds))
    o.check(y, bound, bounds)
    (out, ob), (gu, gb) = ref.gated(x, w, bounds, "silu", "bf16")
    o, s = Out(rows, N // 2, "bf16"), Out(rows, N, "bf16")
    nqg.moe_gated_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds), gate_up=s.view)
    o.check(out, ob, bounds)
    s.check(gu, gb, bounds)
    check_linear_backward(bounds, rows, K, N, "bf16", "fp32")


# few tiles with a long contraction, which several pairs share: 4 of them, 3, 2, an odd number of steps, columns in several chunks
@pytest.mark.parametrize("rows,K,N,E", [(1, 4096, 272, 1), (130, 3080, 512, 1), (256, 2600, 208, 1), (250, 3000, 64, 2),
                                        (700, 4104, 1040, 1), (33, 8192, 1040, 1), (40, 4104, 2048, 2), (16, 2568, 4112, 1), (120, 4096, 5136, 1)])
def test_shared_contractions(rows, K, N, E):
    bounds = [0, rows] if E == 1 else [0, rows // 3, rows - 1]
    g = gen(K + rows)
    x, w = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5)
    y, bound, _ = ref.product(x, w, bounds, "bf16")
    (out, ob), (gu, gb) = ref.gated(x, w, bounds, "gelu_tanh", "bf16")
    for _ in range(2):
        o = Out(rows, N, "bf16")
        nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds))
        o.check(y, bound, bounds)
        o, s = Out(rows, N // 2, "bf16"), Out(rows, N, "bf16")
        nqg.moe_gated_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds), gate_up=s.view, activation="gelu_tanh")
        o.check(out, ob, bounds)
        s.check(gu, gb, bounds)
    check_linear_backward(bounds, rows, K, N, "bf16", "bf16")
    check_linear_backward(bounds, rows, N, K, "bf16", "fp32")


# the weights' gradient of many rows with few columns
@pytest.mark.parametrize("rows,K,N,E,grad", [(3001, 72, 64, 1, "bf16"), (5000, 264, 520, 1, "fp32"), (9000, 40, 1000, 2, "bf16"),
                                             (12000, 136, 200, 3, "fp32"), (2600, 64, 256, 1, "bf16"), (4200, 1288, 1032, 1, "bf16"),
                                             (4104, 1200, 1024, 1, "bf16"), (4104, 1200, 1024, 1, "fp32"), (4130, 1344, 1536, 1, "bf16"),
                                             (6000, 512, 1288, 1, "bf16"), (5300, 640, 1032, 1, "fp32")])
def test_shared_rows(rows, K, N, E, grad):
    bounds = {1: [0, rows], 2: [5, 100, rows], 3: [0, rows - 7, rows - 7, rows]}[E]
    check_linear_backward(bounds, rows, K, N, "bf16", grad)


# tiles of 224, 192, 160 and 128 columns: of rows and, in the weights' gradient, of the other matrix
@pytest.mark.parametrize("rows,K,N,E", [(450, 136, 1040, 1), (900, 264, 2064, 1), (1100, 136, 4112, 1), (640, 72, 4112, 1),
                                        (130, 1400, 2064, 1), (70, 4000, 1040, 1), (203, 3304, 1040, 1), (190, 2000, 1040, 2)])
def test_tiles_of_other_widths(rows, K, N, E):
    bounds = [0, rows] if E == 1 else [3, 100, rows - 5]
    g = gen(K + rows)
    x, w = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5)
    y, bound, _ = ref.product(x, w, bounds, "bf16")
    o = Out(rows, N, "bf16", 8)
    nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds))
    o.check(y, bound, bounds)
    (out, ob), (gu, gb) = ref.gated(x, w, bounds, "silu", "bf16")
    o, s = Out(rows, N // 2, "bf16"), Out(rows, N, "bf16", 8)
    nqg.moe_gated_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds), gate_up=s.view)
    o.check(out, ob, bounds)
    s.check(gu, gb, bounds)
    check_linear_backward(bounds, rows, K, N, "bf16", "bf16")
    check_linear_backward(bounds, rows, N, K, "bf16", "fp32")


def test_matrices_of_more_than_2_to_the_32_bytes():
    """Rows far beyond 2^31 elements from the first, of a matrix and of a gradient."""
    rows, K, N = 600_000, 4096, 64
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    tail = normal(gen(3), 200, K)
    x[-200:] = tail.to(DEV)
    w = normal(gen(4), 1, N, K, std=K ** -0.5)
    out = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    nqg.moe_grouped_linear(x, w.to(DEV), out)
    y, bound, _ = ref.product(tail, w, [0, 200], "bf16")
    near(out[-200:], y, bound)
    assert bool((out[:-200] == 0).all())
    dy = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    dt = normal(gen(5), 200, N)
    dy[-200:] = dt.to(DEV)
    dx, dw = torch.empty_like(x), torch.empty((1, N, K), dtype=torch.float32, device=DEV)
    nqg.moe_grouped_linear_backward(dy, x=x, w=w.to(DEV), d_x=dx, d_w=dw, grad_dtype="fp32")
    zero = torch.zeros(200, N, dtype=torch.float64)
    want, bound = ref.input_grad(dt.double(), zero, w, [0, 200], "bf16")
    near(dx[-200:], want, bound)
    want, _ = ref.weight_grad(dt.double(), zero, tail, [0, 200], "bf16", "fp32")
    # rows of zeros add nothing, but each of their additions may round
    mag = dt.double().abs().t() @ tail.double().abs()
    near(dw[0], want[0], (rows / 16 + 96) * 2.0 ** -23 * mag)


def test_repeated_calls_streams_and_graphs():
    """The same result from call to call, on another stream, and from a graph that is replayed with other inputs and
    offsets than it was captured with."""
    rows, H, I, E = 300, 136, 72, 5
    g = gen(21)
    w = normal(g, E, 2 * I, H, std=H ** -0.5).to(DEV)
    w2 = normal(g, E, H, I, std=I ** -0.5).to(DEV)
    x = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV)
    d = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    inputs = [(normal(gen(s), rows, H), normal(gen(s + 50), rows, H), b) for s, b in
              ((1, [0, 10, 10, 200, 300, 300]), (2, [0, 0, 150, 160, 170, 290]), (3, [7, 100, 200, 201, 202, 203]))]

    def load(i):
        x.copy_(inputs[i][0])
        d.copy_(inputs[i][1])
        off.copy_(torch.tensor(inputs[i][2], dtype=torch.int32))

    class Step:
        def __init__(self):
            z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
            self.gu, self.h, self.y = z(rows, 2 * I), z(rows, I), z(rows, H)
            self.dh, self.dx, self.dw2, self.dw = z(rows, I), z(rows, H), z(E, H, I), z(E, 2 * I, H)
            self.ws = torch.empty(nqg.moe_gated_linear_backward_workspace_size(rows, I), dtype=torch.uint8, device=DEV)

        def run(self):
            for t in (self.gu, self.h, self.y, self.dh, self.dx):
                t.zero_()
            nqg.moe_gated_linear(x, w, self.h, offsets=off, gate_up=self.gu)
            nqg.moe_grouped_linear(self.h, w2, self.y, offsets=off)
            nqg.moe_grouped_linear_backward(d, x=self.h, w=w2, d_x=self.dh, d_w=self.dw2, offsets=off)
            nqg.moe_gated_linear_backward(self.dh, self.gu, x=x, w13=w, d_x=self.dx, d_w13=self.dw, workspace=self.ws, offsets=off)
            return [self.h, self.gu, self.y, self.dh, self.dx, self.dw2, self.dw]

    eager, want = Step(), []
    for i in range(3):
        load(i)
        want.append([t.clone() for t in eager.run()])
        again = eager.run()
        assert all(torch.equal(a, b) for a, b in zip(again, want[i]))
    side = torch.cuda.Stream()
    steps, graphs = [Step(), Step()], []
    load(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(steps[0].run(), want[0]))
        side.synchronize()
        for s in steps:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                s.run()
    torch.cuda.synchronize()
    for i in (2, 1, 0):
        load(i)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s in steps:
            assert all(torch.equal(a, b) for a, b in zip([s.h, s.gu, s.y, s.dh, s.dx, s.dw2, s.dw], want[i])), i


def test_calls_on_two_streams_at_once():
    rows, K, N = 400, 264, 520
    g = gen(8)
    xs = [normal(g, rows, K).to(DEV) for _ in range(2)]
    w = normal(g, 1, N, K, std=K ** -0.5).to(DEV)
    want = []
    for x in xs:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
        nqg.moe_grouped_linear(x, w, out)
        want.append(out)
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, s in zip(xs, outs, streams):
            nqg.moe_grouped_linear(x, w, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("E,rows", [(1024, 700), (1024, 5), (300, 2000), (915, 64)])
def test_many_experts(E, rows):
    """Most experts empty, and tables of the largest size."""
    H, I = 72, 40
    g = gen(E + rows)
    counts = torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E)
    bounds = [0, *counts.cumsum(0).tolist()]
    x, w = normal(g, rows, H), normal(g, E, 2 * I, H, std=H ** -0.5)
    (out, ob), (gu, gb) = ref.gated(x, w, bounds, "silu", "bf16")
    o, s = Out(rows, I, "bf16"), Out(rows, 2 * I, "bf16")
    nqg.moe_gated_linear(x.to(DEV), w.to(DEV), o.view, offsets=dev_offsets(bounds), gate_up=s.view)
    o.check(out, ob, bounds)
    s.check(gu, gb, bounds)
    check_linear_backward(bounds, rows, H, 2 * I, "bf16", "bf16")


@pytest.mark.parametrize("rows,K,N", [(3, 65536, 16), (5, 16, 65536)])
def test_widest_matrices(rows, K, N):
    bounds = [0, rows]
    g = gen(K)
    x, w = normal(g, rows, K), normal(g, 1, N, K, std=K ** -0.5)
    y, bound, _ = ref.product(x, w, bounds, "bf16")
    o = Out(rows, N, "bf16")
    nqg.moe_grouped_linear(x.to(DEV), w.to(DEV), o.view)
    o.check(y, bound, bounds)
    check_linear_backward(bounds, rows, K, N, "bf16", "fp32")


def test_weights_beyond_2_to_the_31_elements():
    """The last of experts that hold more than 2^31 elements together, forward and backward."""
    E, N, K, rows = 70, 4096, 8192, 40
    g = gen(9)
    tail = normal(g, 1, N, K, std=K ** -0.5)
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    w[-1] = tail[0].to(DEV)
    x, dy = normal(g, rows, K), normal(g, rows, N)
    bounds = [0] * E + [rows]
    out = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    nqg.moe_grouped_linear(x.to(DEV), w, out, offsets=dev_offsets(bounds))
    y, bound, _ = ref.product(x, tail, [0, rows], "bf16")
    near(out, y, bound)
    dx, dw = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV), torch.full_like(w, CANARY)
    nqg.moe_grouped_linear_backward(dy.to(DEV), x=x.to(DEV), w=w, d_x=dx, d_w=dw, offsets=dev_offsets(bounds))
    zero = torch.zeros(rows, N, dtype=torch.float64)
    near(dx, *ref.input_grad(dy.double(), zero, tail, [0, rows], "bf16"))
    want, bound = ref.weight_grad(dy.double(), zero, x, [0, rows], "bf16", "bf16")
    near(dw[-1], want[0], bound[0])
    assert bool((dw[:-1] == 0).all())
