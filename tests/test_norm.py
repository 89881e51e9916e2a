"""Layer norm and its gradients against the formulas in 64 bits.

Tolerances from the arithmetic (e = 2^-24, half a float32 step): a row sum is at most 40 additions deep
(16 columns of a thread, the shuffles and the warps), so it is off by 40 e times the sum of magnitudes; the
rest are a few roundings each, and one to the output's type (h = 2^-8 for bf16, 2^-24 for float32).  The column
sums of the gradients run over at most `rows` rows, then 64 additions."""
import pytest
import torch

from tests.gpu_helpers import require_gpu

E = 2.0 ** -24
DEEP = 40
EPS = 1e-6


def half_step(t):
    return torch.finfo(t).eps / 2


def make(seed, rows, width, dtype, affine=True, offset=0.3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    X = (r(rows, width) * (0.5 + torch.rand(width, device="cuda", generator=g)) + offset * r(width)).to(dtype)
    dY = (0.1 * r(rows, width)).to(dtype)
    return X, dY, (1 + 0.1 * r(width) if affine else None), (0.1 * r(width) if affine else None)


def forward_ref(X, gamma, beta, eps=EPS):
    x = X.double()
    w = x.shape[1]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xhat = c * rstd
    ga = torch.ones(w, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    be = torch.zeros(w, device="cuda", dtype=torch.float64) if beta is None else beta.double()
    y = xhat * ga + be
    e_mean = (DEEP + 2) * E * x.abs().mean(1, keepdim=True)
    e_c = e_mean + E * c.abs()
    e_var = (DEEP + 4) * E * var + 2 * (c.abs() * e_c).mean(1, keepdim=True) + (e_c ** 2).mean(1, keepdim=True)
    rel = (0.5 * e_var / (var + eps) + 6 * E) * 1.1  # rsqrtf: 2 units in the last place = 4 E
    e_y = (rstd * e_c + xhat.abs() * rel) * ga.abs() + 3 * E * (xhat * ga).abs() + 2 * E * y.abs()
    return (y, e_y * 1.1 + half_step(X.dtype) * y.abs() + 1e-37), (mean[:, 0], e_mean[:, 0] + 1e-37), (rstd[:, 0], (rel * rstd)[:, 0])


def backward_ref(X, dY, gamma, mean, rstd):
    x, dy, m, r = X.double(), dY.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, w = x.shape
    ga = torch.ones(w, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    xhat, g = (x - m) * r, dy * ga
    c1, c2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = r * (g - c1 - xhat * c2)
    e_c1 = (DEEP + 3) * E * g.abs().mean(1, keepdim=True)
    e_c2 = (DEEP + 6) * E * (g * xhat).abs().mean(1, keepdim=True)
    e_dx = r * (6 * E * (g.abs() + c1.abs() + (xhat * c2).abs()) + e_c1 + xhat.abs() * e_c2)
    dg, db = (dy * xhat).sum(0), dy.sum(0)
    n = (rows + 64) * E
    return ((dx, e_dx * 1.1 + half_step(X.dtype) * dx.abs() + 1e-37), (dg, (n + 3 * E) * (dy * xhat).abs().sum(0) * 1.1 + 1e-37),
            (db, n * dy.abs().sum(0) * 1.1 + 1e-37))


def check(got, ref, what):
    over = (got.double() - ref[0]).abs() - ref[1]
    assert not torch.isnan(over).any() and over.max().item() <= 0, (what, over.max().item())


def both(svg2, X, dY, gamma, beta, eps=EPS):
    rows, width = X.shape
    Y, dX = torch.full_like(X, torch.nan), torch.full_like(X, torch.nan)
    f = lambda n: torch.full((n,), torch.nan, device="cuda")  # noqa: E731
    mean, rstd, dgamma, dbeta = f(rows), f(rows), f(width), f(width)
    svg2.svg2_layer_norm(X, gamma, beta, eps, Y, mean, rstd)
    ws = svg2.layer_norm_bwd_workspace(rows, width)
    svg2.svg2_layer_norm_bwd(X, dY, gamma, mean, rstd, dX, dgamma, dbeta, ws)
    svg2.raise_on_device_error(ws)
    return Y, mean, rstd, dX, dgamma, dbeta


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width,affine", [
    (1, 1, True), (3, 2, False), (1, 8, True), (5, 7, True), (33, 32, True), (1000, 64, True), (1, 128, True),
    (4099, 128, True), (517, 77, True), (100, 129, False), (77, 256, True), (50, 264, True), (300, 520, True),
    (19, 1000, True), (31, 1025, True), (40, 2048, False), (200, 2056, True), (700, 5120, True), (3, 8191, True),
    (17, 8192, True),
])
def test_norm_and_gradients(rows, width, affine, dtype):
    svg2 = require_gpu()
    X, dY, gamma, beta = make(rows * 31 + width, rows, width, dtype, affine)
    Y, mean, rstd, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)
    ry, rm, rr = forward_ref(X, gamma, beta)
    check(mean, rm, "mean")
    check(rstd, rr, "rstd")
    check(Y, ry, "Y")
    rx, rg, rb = backward_ref(X, dY, gamma, mean, rstd)
    check(dX, rx, "dX")
    check(dgamma, rg, "dgamma")
    check(dbeta, rb, "dbeta")


@pytest.mark.gpu
def test_long_reduction():
    """More rows than the CTAs take at once: every thread sums over many rows."""
    svg2 = require_gpu()
    X, dY, gamma, beta = make(3, 200003, 64, torch.bfloat16)
    Y, mean, rstd, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)
    check(Y, forward_ref(X, gamma, beta)[0], "Y")
    rx, rg, rb = backward_ref(X, dY, gamma, mean, rstd)
    check(dX, rx, "dX")
    for got, ref in ((dgamma, rg), (dbeta, rb)):  # the sums of 200003 terms, float32: far inside the worst case
        assert torch.linalg.norm(got.double() - ref[0]) <= 1e-5 * torch.linalg.norm(ref[0])
    again = both(svg2, X, dY, gamma, beta)
    assert all(torch.equal(a, b) for a, b in zip((Y, mean, rstd, dX, dgamma, dbeta), again))


@pytest.mark.gpu
def test_unaligned_and_in_place():
    """Contiguous views that start off a 16-byte boundary, and Y written over X."""
    svg2 = require_gpu()
    for dtype in (torch.bfloat16, torch.float32):
        X, dY, gamma, beta = make(9, 40, 128, dtype)
        Y, mean, rstd, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)
        shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
        Xs, dYs, gs, bs = shift(X), shift(dY), shift(gamma), shift(beta)
        assert Xs.data_ptr() % 16 and Xs.is_contiguous()
        Y2, mean2, rstd2, dX2, dgamma2, dbeta2 = both(svg2, Xs, dYs, gs, bs)
        check(Y2, forward_ref(X, gamma, beta)[0], "Y")
        check(dX2, backward_ref(X, dY, gamma, mean2, rstd2)[0], "dX")
        buf = X.clone()
        svg2.svg2_layer_norm(buf, gamma, beta, EPS, buf)
        assert torch.equal(buf, Y)
        g = dY.clone()
        svg2.svg2_layer_norm_bwd(X, g, gamma, mean, rstd, g, None, dbeta, svg2.layer_norm_bwd_workspace(40, 128))
        assert torch.equal(g, dX)


@pytest.mark.gpu
def test_hard_rows():
    """A constant row, a row far from zero, and a row that holds an infinity (only its own outputs suffer)."""
    svg2 = require_gpu()
    X, dY, gamma, beta = make(4, 64, 96, torch.float32)
    X[3] = 2.5
    X[5] = 1e4 + X[5]
    X[7, 11] = torch.inf
    Y, mean, rstd, dX, _, _ = both(svg2, X, dY, gamma, beta)
    fine = [i for i in range(64) if i != 7]
    ry, rm, rr = forward_ref(X[fine], gamma, beta)
    check(Y[fine], ry, "Y")
    check(mean[fine], rm, "mean")
    assert torch.isnan(Y[7]).any()
    check(dX[fine], backward_ref(X[fine], dY[fine], gamma, mean[fine], rstd[fine])[0], "dX")


@pytest.mark.gpu
def test_gradients_against_differences():
    """dX and the parameters' gradients against central differences of the 64-bit forward."""
    svg2 = require_gpu()
    X, dY, gamma, beta = make(6, 6, 24, torch.float32)
    _, _, _, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)

    def loss(x, ga, be):
        x = x.double()
        c = x - x.mean(1, keepdim=True)
        return ((c * ((c * c).mean(1, keepdim=True) + EPS) ** -0.5 * ga.double() + be.double()) * dY.double()).sum()
    args = [X.double(), gamma.double(), beta.double()]
    h = 1e-5
    for a, got in ((0, dX), (1, dgamma), (2, dbeta)):
        flat = args[a].view(-1)
        for i in range(0, flat.numel(), 7):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(*args)
            flat[i] = keep - h
            down = loss(*args)
            flat[i] = keep
            # differences: h^2 times a third derivative of order 1, and 1e-15 / h of rounding
            assert abs((up - down).item() / (2 * h) - got.flatten()[i].item()) <= 1e-6


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """17 million rows of 128: 2.2e9 elements, a block of 1000 rows repeated, so its results are too."""
    svg2 = require_gpu()
    X, dY, gamma, beta = make(31, 1000, 128, torch.bfloat16)
    ref = both(svg2, X, dY, gamma, beta)
    times = 17000
    got = both(svg2, X.repeat(times, 1), dY.repeat(times, 1), gamma, beta)
    assert got[0].numel() > 2 ** 31
    for i in range(4):  # Y, mean, rstd, dX
        parts = got[i].view(times, *ref[i].shape)
        for t in range(0, times, 1000):
            assert (parts[t:t + 1000] == ref[i]).all(), (i, t)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_all_kinds():
    """Few rows (the last CTA adds the partial rows) and many (another kernel does), in turn, and replayed."""
    svg2 = require_gpu()
    sizes = [(300, 64), (40000, 64), (37, 77), (5, 8192), (2000, 1000), (1, 8)]
    ws = svg2.layer_norm_bwd_workspace(40000, 8192)
    calls = []
    for i, (rows, width) in enumerate(sizes):
        X, dY, gamma, beta = make(40 + i, rows, width, torch.bfloat16)
        _, mean, rstd, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)
        out = [torch.empty_like(t) for t in (dX, dgamma, dbeta)]
        calls.append((lambda X=X, dY=dY, gamma=gamma, mean=mean, rstd=rstd, out=out:
                      svg2.svg2_layer_norm_bwd(X, dY, gamma, mean, rstd, *out, ws), out, (dX, dgamma, dbeta)))
    def compare():
        torch.cuda.synchronize()
        for (_, out, ref), size in zip(calls, sizes):
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), size
            for t in out:
                t.fill_(torch.nan)
    for _ in range(2):
        for call, _, _ in calls:
            call()
        compare()
    graphs = []
    for part in (calls[:3], calls[3:]):  # two graphs share the workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call, _, _ in part:
                call()
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        compare()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width,affine", [
    (4736, 1, True), (4739, 3, True), (5001, 31, False), (4999, 33, True), (6007, 77, True), (5003, 97, True),
    (9001, 129, True), (4741, 255, False), (5005, 257, True), (4800, 333, True), (4743, 511, True), (4737, 513, True),
])
def test_many_rows_of_odd_width(rows, width, affine, dtype):
    """Enough rows for the kernel that copies 16-byte multiples of rows (and one width past it), the last few alone."""
    svg2 = require_gpu()
    X, dY, gamma, beta = make(rows + width, rows, width, dtype, affine)
    Y, mean, rstd, dX, dgamma, dbeta = both(svg2, X, dY, gamma, beta)
    ry, rm, rr = forward_ref(X, gamma, beta)
    check(Y, ry, "Y"), check(mean, rm, "mean"), check(rstd, rr, "rstd")
    rx, rg, rb = backward_ref(X, dY, gamma, mean, rstd)
    check(dX, rx, "dX"), check(dgamma, rg, "dgamma"), check(dbeta, rb, "dbeta")
    again = both(svg2, X, dY, gamma, beta)
    assert all(torch.equal(p, q) for p, q in zip(again, (Y, mean, rstd, dX, dgamma, dbeta)))
    buf = X.clone()  # in place, both ways
    svg2.svg2_layer_norm(buf, gamma, beta, EPS, buf, torch.empty_like(mean), torch.empty_like(rstd))
    assert torch.equal(buf, Y)
    ws = svg2.layer_norm_bwd_workspace(rows, width)
    for into_x in (True, False):
        x, dy = X.clone(), dY.clone()
        svg2.svg2_layer_norm_bwd(x, dy, gamma, mean, rstd, x if into_x else dy, torch.empty_like(dgamma), None, ws)
        assert torch.equal(x if into_x else dy, dX), into_x
