"""The attentions' log-sum-exp and gradients against the formulas in 64 bits.

Tolerances, elementwise, from the formulas (u = 2^-8, half a bf16 step).  A probability carries a relative
error of at most EP: the cubic exponential's 7.5e-5, twice (once in P, once in lse), and the error of
a float32 score, at most (d + 2) 2^-24 scale sum |q k|, twice.  P and dS are rounded to bf16, O too
(it enters delta = dO.O), and the outputs.  dQ is summed as scale sum_j dS_ij (k_j - c) with c the mean of up to
512 evenly spaced keys, or of the keys that the row's cluster keeps in the sparse call (the same in exact arithmetic,
where a row of dS sums to zero; formulas() takes the first for both, which for keys of one distribution is as far
from them), so an error e_ij of dS enters as e_ij (k_j - c), and the float32 sums over N keys add N 2^-24 times their terms' magnitudes (which the
bf16 terms cover everywhere else).  With |.| taken inside every sum this bounds each entry; for
errors of independent sign the relative 2-norm stays below 2 u, which is checked where the sums do not cancel."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu

U = 2.0 ** -8


def mean_key(k):
    S = min(512, k.shape[0])
    x = k[torch.arange(S, device=k.device) * k.shape[0] // S].double()
    return torch.where(x.isfinite(), x, 0.0).mean(0)


def formulas(q, k, v, do, scale, keep=None, c=None):
    """Float64 outputs and their error bounds for one plane [N, d]; keep [N, N]: the kept pairs."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    d = q.shape[1]
    s = q @ k.T * scale
    if keep is not None:
        s = s.masked_fill(~keep, -torch.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.where(lse[:, None] > -torch.inf, torch.exp(s - lse.clamp(min=-1e300)[:, None]), 0.0)
    o, dp = p @ v, do @ v.T
    delta = (do * o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    out = {"O": o, "dV": p.T @ do, "dQ": ds @ k * scale, "dK": ds.T @ q * scale}
    es = (d + 2) * 2.0 ** -24 * scale * (q.abs() @ k.abs().T)
    if keep is not None:
        es = es * keep
    ep = (2 * 7.5e-5 + es + es.amax(1, keepdim=True)) * 1.01
    pv = p @ v.abs()
    e_o = (U + ep.amax(1, keepdim=True)) * pv + U * o.abs()
    e_delta = (do.abs() * e_o).sum(1, keepdim=True) + d * 2.0 ** -23 * (do.abs() * o.abs()).sum(1, keepdim=True)
    c = mean_key(k) if c is None else c
    e_dp = d * 2.0 ** -23 * (do.abs() @ v.abs().T)
    e_ds = (U + 2 * ep) * ds.abs() + p * (e_delta + e_dp) * (1 + U)
    tol = {"O": e_o, "dV": ((U + ep) * p).T @ do.abs() + U * out["dV"].abs(),
           "dQ": (e_ds @ (k - c).abs() + (len(k) + 8) * 2.0 ** -24 * (ds.abs() @ (k.abs() + c.abs()))) * scale + U * out["dQ"].abs(), "dK": e_ds.T @ q.abs() * scale + U * out["dK"].abs()}
    out["lse"] = lse
    tol["lse"] = 7.5e-5 * 1.01 + es.amax(1) + 2.0 ** -22 * lse.abs().clamp(max=1e30)
    return out, {n: 1.02 * t + 1e-30 for n, t in tol.items()}


def check(got, ref, tol, what, norm=True):
    got = got.double()
    empty = torch.isinf(ref)
    assert torch.equal(got[empty], ref[empty]), what
    err = (got - ref).abs()[~empty]
    over = err - tol[~empty]
    assert not torch.isnan(err).any() and (err.numel() == 0 or over.max().item() <= 0), (what, over.max().item(), err.max().item())
    if norm and err.numel():
        rel = (torch.linalg.norm((got - ref)[~empty]) / torch.linalg.norm(ref[~empty]).clamp(min=1e-30)).item()
        assert rel <= 2 * U, (what, rel)


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dense_step(svg2, Q, K, V, dO, scale, ws=None):
    B, H, N, d = Q.shape
    O, dQ, dK, dV = (torch.full_like(Q, torch.nan) for _ in range(4))
    lse = torch.full((B, H, N), torch.nan, device="cuda")
    ws = svg2.dense_bwd_workspace(B, H, N, d) if ws is None else ws
    svg2.svg2_dense_attn_lse(Q, K, V, scale, O, lse, ws)
    svg2.svg2_dense_attn_bwd(Q, K, V, O, lse, dO, scale, dQ, dK, dV, ws)
    svg2.raise_on_device_error(ws)
    return {"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,d", [
    (1, 1, 1, 128), (2, 1, 1, 64),       # one token: P = 1, dS = 0
    (1, 2, 2, 128), (1, 1, 31, 64),
    (1, 1, 127, 64), (1, 1, 128, 128),   # one tile
    (2, 2, 129, 128),                     # one row past it
    (1, 3, 257, 64), (1, 1, 384, 128),   # three tiles: every stage is reused
    (2, 1, 640, 64), (1, 2, 1000, 128), (1, 1, 2111, 128),
])
def test_dense_gradients(B, H, N, d):
    svg2 = require_gpu()
    g = gen(N * 131 + d + H)
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    scale = d ** -0.5
    got = dense_step(svg2, Q, K, V, dO, scale)
    for b in range(B):
        for h in range(H):
            ref, tol = formulas(Q[b, h], K[b, h], V[b, h], dO[b, h], scale)
            for n in ref:
                check(got[n][b, h], ref[n], tol[n], (n, b, h), norm=N > 1 and n != "lse")


@pytest.mark.gpu
@pytest.mark.parametrize("scale,mag", [(0.5, 1.0), (1e-30, 1.0), (0.125, 4.0), (1e-3, 30.0)])
def test_dense_gradients_scales(scale, mag):
    """P from one-hot to uniform (a scale of zero or below is refused)."""
    svg2 = require_gpu()
    g = gen(5)
    Q, K = (randn(g, 1, 1, 300, 64, scale=mag) for _ in range(2))
    V, dO = (randn(g, 1, 1, 300, 64) for _ in range(2))
    got = dense_step(svg2, Q, K, V, dO, scale)
    ref, tol = formulas(Q[0, 0], K[0, 0], V[0, 0], dO[0, 0], scale)
    for n in ref:
        check(got[n][0, 0], ref[n], tol[n], n, norm=False)


def plan(seed, B, H, N, nQ, nK, density, empty_q=(), unkept_k=(), empty_clusters=False):
    """Random clusters and kept pairs: offsets, permutations (token of each permuted row), kept lists, mask."""
    rng = np.random.default_rng(seed)
    q_off, k_off = np.zeros((B, H, nQ + 1), np.int32), np.zeros((B, H, nK + 1), np.int32)
    perm_q, perm_k = np.zeros((B, H, N), np.int32), np.zeros((B, H, N), np.int32)
    keep = rng.random((B, H, nQ, nK)) < density
    keep[:, :, list(empty_q)] = False
    keep[:, :, :, list(unkept_k)] = False
    for b in range(B):
        for h in range(H):
            for n, off, perm in ((nQ, q_off, perm_q), (nK, k_off, perm_k)):
                w = rng.random(n) ** 2 + 0.01
                if empty_clusters and n > 3:
                    w[[1, n - 1]] = 0
                off[b, h, 1:] = np.cumsum(rng.multinomial(N, w / w.sum()))
                perm[b, h] = rng.permutation(N)
    count = keep.sum(3).astype(np.int32)
    idx = np.argsort(~keep, axis=3, kind="stable").astype(np.int32)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(q_off=c(q_off), k_off=c(k_off), perm_q=c(perm_q), perm_k=c(perm_k), sel_count=c(count), sel_idx=c(idx),
                keep=c(keep))


def rows_kept(pl, b, h, N):
    """The plan's kept pairs by permuted rows [N, N]."""
    of = lambda off: torch.repeat_interleave(torch.arange(off.numel() - 1, device="cuda"), off.long().diff())  # noqa: E731
    return pl["keep"][b, h][of(pl["q_off"][b, h])][:, of(pl["k_off"][b, h])]


def sparse_step(svg2, pl, Q, K, V, dO, scale, perms=True, ws=None):
    """Q, K, V by permuted row; O, dO and the gradients by token when perms is set."""
    B, H, N, d = Q.shape
    nQ, nK = pl["q_off"].shape[2] - 1, pl["k_off"].shape[2] - 1
    O, dQ, dK, dV = (torch.full_like(Q, torch.nan) for _ in range(4))
    lse = torch.full((B, H, N), torch.nan, device="cuda")
    ws = svg2.sparse_bwd_workspace(B, H, N, d, nQ, nK) if ws is None else ws
    pq, pk = (pl["perm_q"], pl["perm_k"]) if perms else (None, None)
    args = [pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")]
    svg2.svg2_sparse_attn_lse(Q, K, V, *args, scale, O, lse, ws, perm_q=pq)
    svg2.svg2_sparse_attn_bwd(Q, K, V, O, lse, dO, *args, scale, dQ, dK, dV, ws, perm_q=pq, perm_k=pk)
    svg2.raise_on_device_error(ws)
    return {"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}


def by_row(x, perm, b, h):
    return x[b, h] if perm is None else x[b, h][perm[b, h].long()]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,d,nQ,nK,density,kw,perms", [
    (1, 1, 1, 128, 1, 1, 1.0, {}, True),                                      # one token
    (1, 1, 5, 64, 5, 5, 0.5, {}, True),                                       # clusters of about a row
    (1, 2, 300, 128, 3, 4, 0.6, {}, False),
    (2, 1, 700, 64, 7, 11, 0.5, dict(empty_q=(2,), unkept_k=(3, 5)), True),  # rows without keys, keys without rows
    (1, 1, 1000, 128, 40, 65, 0.3, dict(empty_clusters=True, empty_q=(0, 39)), True),
    (1, 1, 513, 64, 2, 300, 0.7, dict(empty_clusters=True), False),           # tiles of many short pieces
    (1, 1, 1500, 128, 100, 2, 0.5, {}, True),
    (1, 1, 1300, 128, 33, 32, 1.0, {}, True),                                 # every pair: the dense sums
    (1, 1, 1200, 64, 1024, 1024, 0.1, {}, True),                              # the most clusters
    (1, 1, 400, 128, 6, 6, 0.0, {}, True),                                    # nothing kept at all
])
def test_sparse_gradients(B, H, N, d, nQ, nK, density, kw, perms):
    svg2 = require_gpu()
    if nQ > N or nK > N:
        pytest.skip("clusters are at most tokens")
    pl = plan(N + nQ, B, H, N, nQ, nK, density, **kw)
    g = gen(N * 7 + d)
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    scale = d ** -0.5
    got = sparse_step(svg2, pl, Q, K, V, dO, scale, perms)
    pq, pk = (pl["perm_q"], pl["perm_k"]) if perms else (None, None)
    for b in range(B):
        for h in range(H):
            ref, tol = formulas(Q[b, h], K[b, h], V[b, h], by_row(dO, pq, b, h), scale, rows_kept(pl, b, h, N))
            for n in ref:
                x = got[n][b, h] if n == "lse" else by_row(got[n], pk if n in ("dK", "dV") else pq, b, h)
                check(x, ref[n], tol[n], (n, b, h), norm=n != "lse" and N >= 300)


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.gpu
def test_forward_is_the_plain_call_bit_for_bit_and_runs_repeat():
    svg2 = require_gpu()
    g = gen(8)
    Q, K, V, dO = (randn(g, 1, 3, 901, 128) for _ in range(4))
    got = dense_step(svg2, Q, K, V, dO, 0.1)
    O = torch.empty_like(Q)
    svg2.svg2_dense_attn(Q, K, V, 0.1, O, svg2.dense_workspace(1, 3, 901, 128))
    assert torch.equal(O, got["O"])
    pl = plan(3, 1, 3, 901, 9, 30, 0.5)
    one = sparse_step(svg2, pl, Q, K, V, dO, 0.1)
    svg2.svg2_sparse_attn(Q, K, V, *(pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")), 0.1, O,
                          svg2.workspace(1, 3, 901, 128, 9, 30), perm_q=pl["perm_q"])
    assert torch.equal(O, one["O"])
    for _ in range(3):
        assert same(dense_step(svg2, Q, K, V, dO, 0.1), got)
        assert same(sparse_step(svg2, pl, Q, K, V, dO, 0.1), one)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_planes_do_not_leak(d):
    """Rows past a plane's end belong to the next plane: NaN and infinity there reach nothing."""
    svg2 = require_gpu()
    g = gen(d)
    Q, K, V, dO = (randn(g, 1, 3, 321, d) for _ in range(4))
    ref = dense_step(svg2, Q, K, V, dO, 0.1)
    pl = plan(4, 1, 3, 321, 5, 9, 0.5)
    sref = sparse_step(svg2, pl, Q, K, V, dO, 0.1)
    for t, bad in ((Q, torch.nan), (K, torch.inf), (V, torch.nan), (dO, -torch.inf)):
        t[:, 2] = bad
    got = dense_step(svg2, Q, K, V, dO, 0.1)
    sgot = sparse_step(svg2, pl, Q, K, V, dO, 0.1)
    for n in ref:
        assert torch.equal(got[n][:, :2], ref[n][:, :2]) and torch.equal(sgot[n][:, :2], sref[n][:, :2]), n


@pytest.mark.gpu
def test_keys_nobody_keeps_reach_nothing():
    """NaN in a K cluster that no Q cluster keeps: nothing else changes, but for the constant that dQ subtracts."""
    svg2 = require_gpu()
    N = 600
    g = gen(11)
    Q, K, V, dO = (randn(g, 1, 1, N, 64) for _ in range(4))
    pl = plan(6, 1, 1, N, 6, 12, 0.6, unkept_k=(4,))
    ref = sparse_step(svg2, pl, Q, K, V, dO, 0.125, perms=False)
    lo, hi = pl["k_off"][0, 0, 4].item(), pl["k_off"][0, 0, 5].item()
    assert hi > lo
    K[:, :, lo:hi] = torch.nan
    V[:, :, lo:hi] = torch.inf
    got = sparse_step(svg2, pl, Q, K, V, dO, 0.125, perms=False)
    for n in ("O", "lse"):
        assert torch.equal(got[n], ref[n]), n
    exact, tol = formulas(Q[0, 0], torch.where(K.isfinite(), K, 0.0)[0, 0], torch.where(V.isfinite(), V, 0.0)[0, 0],
                          dO[0, 0], 0.125, rows_kept(pl, 0, 0, N), mean_key(K[0, 0]))
    check(got["dQ"][0, 0], exact["dQ"], tol["dQ"], "dQ")
    inside = torch.zeros(N, dtype=torch.bool, device="cuda")
    inside[lo:hi] = True
    for n in ("dK", "dV"):
        assert torch.equal(got[n][0, 0, ~inside], ref[n][0, 0, ~inside]), n


@pytest.mark.gpu
def test_rows_outside_every_cluster_are_left_alone():
    svg2 = require_gpu()
    N = 500
    g = gen(12)
    Q, K, V, dO = (randn(g, 1, 1, N, 128) for _ in range(4))
    pl = plan(7, 1, 1, N, 4, 4, 0.7)
    pl["q_off"][0, 0, 4] = pl["k_off"][0, 0, 4] = N - 70  # the last clusters end early
    pl["q_off"][0, 0, :4].clamp_(max=N - 70)
    pl["k_off"][0, 0, :4].clamp_(max=N - 70)
    got = sparse_step(svg2, pl, Q, K, V, dO, 0.1, perms=False)
    for n in ("dQ", "dK", "dV"):
        assert torch.isnan(got[n][0, 0, N - 70:]).all() and not torch.isnan(got[n][0, 0, :N - 70]).any(), n


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["twice", "past", "negative", "count"])
def test_bad_plans_are_reported_and_write_nothing(what):
    svg2 = require_gpu()
    g = gen(13)
    Q, K, V, dO = (randn(g, 1, 2, 400, 64) for _ in range(4))
    pl = plan(8, 1, 2, 400, 5, 7, 0.8)
    O, lse = torch.empty_like(Q), torch.empty(1, 2, 400, device="cuda")
    args = [pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")]
    ws = svg2.sparse_bwd_workspace(1, 2, 400, 64, 5, 7)
    svg2.svg2_sparse_attn_lse(Q, K, V, *args, 0.1, O, lse, ws)
    row = int(pl["sel_count"][0, 1].argmax())
    assert pl["sel_count"][0, 1, row] >= 2
    if what == "twice":
        pl["sel_idx"][0, 1, row, 1] = pl["sel_idx"][0, 1, row, 0]
    elif what == "count":
        pl["sel_count"][0, 1, row] = 8
    else:
        pl["sel_idx"][0, 1, row, 0] = 7 if what == "past" else -1
    grads = [torch.full_like(Q, 3.0) for _ in range(3)]
    svg2.svg2_sparse_attn_bwd(Q, K, V, O, lse, dO, *args, 0.1, *grads, ws)
    with pytest.raises(svg2.Svg2Error) as e:
        svg2.raise_on_device_error(ws)
    assert e.value.code == 6
    assert all((x == 3.0).all() for x in grads)
    svg2.raise_on_device_error(ws)  # reading cleared it


@pytest.mark.gpu
def test_other_stream_and_captured_graph():
    """The same bits on a side stream and from a replayed CUDA graph (after new inputs were copied in)."""
    svg2 = require_gpu()
    g = gen(14)
    sets = [[randn(g, 1, 2, 700, 128) for _ in range(4)] for _ in range(2)]
    pl = plan(9, 1, 2, 700, 6, 20, 0.6)
    want = [(dense_step(svg2, *s, 0.09), sparse_step(svg2, pl, *s, 0.09)) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dense_step(svg2, *sets[0], 0.09), sparse_step(svg2, pl, *sets[0], 0.09)
    torch.cuda.synchronize()
    assert same(got[0], want[0][0]) and same(got[1], want[0][1])
    Q, K, V, dO = (x.clone() for x in sets[0])
    O, dQ, dK, dV = (torch.empty_like(Q) for _ in range(4))
    lse = torch.empty(1, 2, 700, device="cuda")
    ws_d, ws_s = svg2.dense_bwd_workspace(1, 2, 700, 128), svg2.sparse_bwd_workspace(1, 2, 700, 128, 6, 20)
    out2 = [torch.empty_like(Q) for _ in range(4)]
    lse2 = torch.empty_like(lse)
    args = [pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")]

    def step():
        svg2.svg2_dense_attn_lse(Q, K, V, 0.09, O, lse, ws_d)
        svg2.svg2_dense_attn_bwd(Q, K, V, O, lse, dO, 0.09, dQ, dK, dV, ws_d)
        svg2.svg2_sparse_attn_lse(Q, K, V, *args, 0.09, out2[0], lse2, ws_s, perm_q=pl["perm_q"])
        svg2.svg2_sparse_attn_bwd(Q, K, V, out2[0], lse2, dO, *args, 0.09, *out2[1:], ws_s, perm_q=pl["perm_q"],
                                  perm_k=pl["perm_k"])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0):
        for t, s in zip((Q, K, V, dO), sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert same({"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}, want[i][0])
        assert same({"O": out2[0], "lse": lse2, "dQ": out2[1], "dK": out2[2], "dV": out2[3]}, want[i][1])


@pytest.mark.gpu
def test_two_calls_at_once_on_their_own_workspaces():
    svg2 = require_gpu()
    g = gen(15)
    sets = [[randn(g, 1, 4, 1500, 64) for _ in range(4)] for _ in range(2)]
    want = [dense_step(svg2, *s, 0.1) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, ws = [], []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            O, dQ, dK, dV = (torch.empty_like(s[0]) for _ in range(4))
            lse = torch.empty(1, 4, 1500, device="cuda")
            ws.append(svg2.dense_bwd_workspace(1, 4, 1500, 64))
            for _ in range(5):
                svg2.svg2_dense_attn_lse(*s[:3], 0.1, O, lse, ws[-1])
                svg2.svg2_dense_attn_bwd(*s[:3], O, lse, s[3], 0.1, dQ, dK, dV, ws[-1])
            got.append({"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV})
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_gradients_against_differences():
    """Entries of dQ, dK, dV against central differences of the 64-bit loss sum(O o dO)."""
    svg2 = require_gpu()
    g = gen(16)
    Q, K, V, dO = (randn(g, 1, 1, 40, 64) for _ in range(4))
    got = dense_step(svg2, Q, K, V, dO, 0.125)
    ref, tol = formulas(Q[0, 0], K[0, 0], V[0, 0], dO[0, 0], 0.125)
    x = [t[0, 0].double() for t in (Q, K, V)]
    h = 1e-5
    for a, n in enumerate(("dQ", "dK", "dV")):
        for i in range(0, 40 * 64, 331):
            at = divmod(i, 64)
            v = []
            for sgn in (h, -h):
                y = [t.clone() for t in x]
                y[a][at] += sgn
                v.append(((torch.softmax(y[0] @ y[1].T * 0.125, 1) @ y[2]) * dO[0, 0].double()).sum().item())
            # differences: 1e-14 / h of rounding, h^2 times a third derivative of order 1
            assert abs((v[0] - v[1]) / (2 * h) - got[n][0, 0][at].item()) <= tol[n][at].item() + 1e-8


@pytest.mark.gpu
def test_wait_that_runs_out_is_reported_and_leaves_the_workspace_usable():
    svg2 = require_gpu()
    g = gen(17)
    Q, K, V, dO = (randn(g, 1, 2, 1000, 128) for _ in range(4))
    want = dense_step(svg2, Q, K, V, dO, 0.1)
    ws = svg2.dense_bwd_workspace(1, 2, 1000, 128)
    O, dQ, dK, dV = (torch.empty_like(Q) for _ in range(4))
    svg2.svg2_set_wait_budget(ws, 1)
    svg2.svg2_dense_attn_bwd(Q, K, V, want["O"], want["lse"], dO, 0.1, dQ, dK, dV, ws)
    code = svg2.svg2_check_status(ws)[0]
    assert code == 5
    svg2.svg2_set_wait_budget(ws, 0)
    assert same(dense_step(svg2, Q, K, V, dO, 0.1, ws), want)


def _chain64(layer, Q, K, V, dO, params, keep):
    """The whole training layer in float64 with autograd: norm, attention over the kept pairs, loss sum(O o dO)."""
    leaves = {n: t.detach().double().requires_grad_() for n, t in dict(Q=Q, K=K, V=V, **params).items()}

    def norm(x, ga, be):
        c = x - x.mean(-1, keepdim=True)
        return c * ((c * c).mean(-1, keepdim=True) + layer.norm_eps) ** -0.5 * ga + be
    q = norm(leaves["Q"], leaves["gamma_q"], leaves["beta_q"])
    k = norm(leaves["K"], leaves["gamma_k"], leaves["beta_k"])
    s = q @ k.mT * layer.scale
    if keep is not None:
        s = s.masked_fill(~keep, -torch.inf)
    O = torch.softmax(s, -1) @ leaves["V"]
    (O * dO.double()).sum().backward()
    return O.detach(), {("d" + n): t.grad for n, t in leaves.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("sparse", [False, True])
def test_training_layer(sparse):
    """Norm, attention and both gradients as one layer, against the chain in 64 bits.  Seven roundings to bf16 lie on
    the way (Qn, Kn, P, O, dS, the attention's gradient, dX), each at most U of its value; a change of U in q
    and k moves a score by at most 2 U scale |q||k| ~ 2 U sqrt(d) for normed rows, and P by that factor: the
    relative 2-norm stays below (7 + 2 sqrt(d)) U.  The parameters' gradients are sums over rows whose terms cancel
    (dbeta_k is zero: adding one vector to all keys moves no probability), so the sums of the terms' magnitudes
    take their place there: |dY| for beta, at most sqrt(d) |dY| for gamma (a normed row's entries)."""
    svg2 = require_gpu()
    B, H, N, d = 1, 2, 900, 64
    g = gen(18)
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    r = lambda c: c + 0.1 * torch.randn(d, device="cuda", generator=g)  # noqa: E731
    params = dict(gamma_q=r(1), beta_q=r(0), gamma_k=r(1), beta_k=r(0))
    prm = svg2.LayerParams(6, 12, 2, svg2.SVG2_INIT_KMEANSPP, 0.6, d ** -0.5, 1) if sparse else None
    layer = svg2.TrainingLayer(B, H, N, d, prm, norm_eps=1e-5)
    u = dict(uq=torch.rand(B, H, 6, dtype=torch.float64, device="cuda", generator=g),
             uk=torch.rand(B, H, 12, dtype=torch.float64, device="cuda", generator=g)) if sparse else {}
    with pytest.raises(ValueError):
        layer.backward(dO)
    O = layer.forward(Q, K, V, **params, **u)
    grads = layer.backward(dO)
    svg2.raise_on_device_error(layer.ws)
    keep = None
    if sparse:
        m = layer.plan["mask"].bool()
        lq, lk = layer.plan["labels_q"].long(), layer.plan["labels_k"].long()
        keep = torch.stack([m[0, h][lq[0, h]][:, lk[0, h]] for h in range(H)])[None]
        assert 0 < keep.float().mean() < 1
    ref_O, ref = _chain64(layer, Q, K, V, dO, params, keep)
    bound = (7 + 2 * d ** 0.5) * U
    for n, x in dict(grads, O=O).items():
        y = ref_O if n == "O" else ref[n]
        size = torch.linalg.norm(y)
        if n.startswith(("dbeta", "dgamma")):
            terms = (layer.dQ if n.endswith("q") else layer.dK).double().abs().sum((0, 1, 2))
            size = torch.linalg.norm(terms) * (d ** 0.5 if n.startswith("dgamma") else 1.0)
        rel = (torch.linalg.norm(x.double() - y) / size).item()
        assert rel <= bound, (n, rel)
    if sparse:  # a second step from the cached centroids
        layer.forward(Q, K, V, **params, init=svg2.SVG2_INIT_GIVEN)
        layer.backward(dO)
        svg2.raise_on_device_error(layer.ws)


@pytest.mark.gpu
@pytest.mark.parametrize("sparse", [False, True])
def test_offsets_past_32_bits(sparse):
    """18000 planes of 1000 x 128: 2.3e9 elements per tensor.  They repeat three planes, so every result does."""
    svg2 = require_gpu()
    g = gen(21)
    N, d, times = 1000, 128, 6000
    base = [randn(g, 1, 3, N, d) for _ in range(4)]
    big = [x.repeat(1, times, 1, 1) for x in base]
    assert big[0].numel() > 2 ** 31
    if sparse:
        pl = plan(22, 1, 3, N, 6, 9, 0.5)
        ref = sparse_step(svg2, pl, *base, 0.1)
        many = {n: x.repeat(1, times, *[1] * (x.dim() - 2)) if torch.is_tensor(x) and x.dim() > 2 else x for n, x in pl.items()}
        got = sparse_step(svg2, many, *big, 0.1)
    else:
        ref = dense_step(svg2, *base, 0.1)
        got = dense_step(svg2, *big, 0.1)
    del big
    for n in ref:
        parts = got[n].view(times, 3, *ref[n].shape[2:])
        for i in range(0, times, 500):
            assert (parts[i:i + 500] == ref[n]).all(), (n, i)


@pytest.mark.gpu
def test_as_many_planes_as_allowed():
    """65535 planes of one token: P = 1 within EP, so O = V, dV = dO within EP and a rounding, and dS = P dP (1 - P)."""
    svg2 = require_gpu()
    g = gen(23)
    Q, K, V, dO = (randn(g, 5, 13107, 1, 64) for _ in range(4))
    got = {n: x.double() for n, x in dense_step(svg2, Q, K, V, dO, 0.125).items()}
    q, k, v, do = (x.double() for x in (Q, K, V, dO))
    es = 66 * 2.0 ** -24 * 0.125 * (q * k).abs().sum(3, keepdim=True)
    ep = (2 * 7.5e-5 + 2 * es) * 1.01
    assert ((got["O"] - v).abs() <= (ep + U) * 1.02 * v.abs()).all()
    assert ((got["dV"] - do).abs() <= (ep + U) * 1.02 * do.abs()).all()
    assert ((got["lse"] - 0.125 * (q * k).sum(3)).abs() <= (7.5e-5 + 2 * es[..., 0]) * 1.02 + 2.0 ** -22 * got["lse"].abs()).all()
    ds = ep * (do * v).abs().sum(3, keepdim=True) * (1 + 2 * U)
    assert (got["dK"].abs() <= 0.125 * ds * q.abs() * 1.02).all()
    assert (got["dQ"].abs() <= 0.125 * ds * 2 * k.abs() * 1.02).all()  # dS k - (its sum) times the mean key


@pytest.mark.gpu
def test_debug_build_of_the_gradients():
    """The library with its bounds checks: nothing is reported on good plans; offsets that do not ascend or
    reach past the plane, and a permutation entry out of range, are."""
    from sparse_attention_video_head_b200 import build
    svg2 = require_gpu()
    g = gen(24)
    B, H, N, d, nQ, nK = 1, 2, 1500, 64, 40, 70
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    pl = plan(25, B, H, N, nQ, nK, 0.5)
    ref = sparse_step(svg2, pl, Q, K, V, dO, 0.125)
    dref = dense_step(svg2, Q, K, V, dO, 0.125)
    build.build(debug=True)
    svg2.use_debug_library(True)
    try:
        got, dgot = sparse_step(svg2, pl, Q, K, V, dO, 0.125), dense_step(svg2, Q, K, V, dO, 0.125)
        for n in ref:
            assert torch.equal(got[n], ref[n]) and torch.equal(dgot[n], dref[n]), n
        ws = svg2.sparse_bwd_workspace(B, H, N, d, nQ, nK)
        for name, at, value in (("k_off", 3, N + 5), ("q_off", 20, -7), ("k_off", 40, 0), ("perm_q", 11, N), ("perm_k", 12, -1)):
            bad = {n: x.clone() if torch.is_tensor(x) else x for n, x in pl.items()}
            bad[name][0, 1, at] = value
            grads = [torch.zeros_like(Q) for _ in range(3)]
            svg2.svg2_sparse_attn_bwd(Q, K, V, ref["O"], ref["lse"], dO, *(bad[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")),
                                      0.125, *grads, ws, perm_q=bad["perm_q"], perm_k=bad["perm_k"])
            with pytest.raises(svg2.Svg2Error) as e:
                svg2.raise_on_device_error(ws)
            assert e.value.code == 6, name
    finally:
        svg2.use_debug_library(False)


@pytest.mark.gpu
def test_malformed_offsets_stay_in_their_planes():
    """Offsets of one plane that do not ascend: the other plane's gradients are what they were."""
    svg2 = require_gpu()
    g = gen(26)
    B, H, N, d, nQ, nK = 1, 2, 1500, 64, 70, 90
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    pl = plan(27, B, H, N, nQ, nK, 0.5)
    ref = sparse_step(svg2, pl, Q, K, V, dO, 0.125, perms=False)
    for name, n in (("q_off", nQ), ("k_off", nK)):
        pl[name][0, 1] = torch.randint(-50, N + 50, (n + 1,), device="cuda", generator=g, dtype=torch.int32)
    ws = svg2.sparse_bwd_workspace(B, H, N, d, nQ, nK)
    grads = [torch.full_like(Q, 3.0) for _ in range(3)]
    svg2.svg2_sparse_attn_bwd(Q, K, V, ref["O"], ref["lse"], dO, *(pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")),
                              0.125, *grads, ws)
    svg2.raise_on_device_error(ws)
    for n, x in zip(("dQ", "dK", "dV"), grads):
        assert torch.equal(x[0, 0], ref[n][0, 0]), n


def even_plan(seed, B, H, N, nQ, nK, keep):
    """Clusters of about equal size, keep [nQ, nK] for every plane, no permutations."""
    edges = lambda n: torch.tensor([N * i // n for i in range(n + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    keep = keep.to("cuda").expand(B, H, nQ, nK).contiguous()
    return dict(q_off=edges(nQ).expand(B, H, nQ + 1).contiguous(), k_off=edges(nK).expand(B, H, nK + 1).contiguous(),
                keep=keep, sel_count=keep.sum(3, dtype=torch.int32),
                sel_idx=torch.sort(keep.to(torch.uint8), dim=3, descending=True, stable=True).indices.int().contiguous())


def rel_norm(x, ref):
    return (torch.linalg.norm(x.double() - ref) / torch.linalg.norm(ref)).item()


@pytest.mark.gpu
@pytest.mark.parametrize("N,nQ,nK,d", [(5000, 100, 40, 64), (5000, 5, 40, 128), (1000, 20, 40, 64), (400, 2, 40, 128),
                                        (3000, 900, 900, 128)])
def test_large_keys_cost_nothing_to_rows_that_do_not_keep_them(N, nQ, nK, d):
    """K clusters 7 and 30 hold finite keys 300 past the others in every column; the odd Q clusters keep neither (30
    is kept by none), and the last rows of the plane, in no cluster, are larger still.  The dS that is handed over sums to
    some r_i, so what dQ subtracts has to come from the keys that the row keeps: the limit is the one of
    the other tests, 2 U for roundings of independent sign, and does not know the large keys.  Units hold rows of one
    cluster (nQ small) and of odd and even ones."""
    svg2 = require_gpu()
    g = gen(N + nQ)
    Q, K, V, dO = (randn(g, 1, 1, N, d) for _ in range(4))
    keep = torch.ones(nQ, nK, dtype=torch.bool)
    keep[:, 30] = False
    keep[1::2, 7] = False
    pl = even_plan(0, 1, 1, N, nQ, nK, keep)
    end = N - N // 50  # rows past the last cluster
    pl["k_off"].clamp_(max=end)
    for c, x in ((7, 300.0), (30, 300.0)):
        K[0, 0, pl["k_off"][0, 0, c]:pl["k_off"][0, 0, c + 1]] += x
    K[0, 0, end:] = 1e4
    got = sparse_step(svg2, pl, Q, K, V, dO, d ** -0.5, perms=False)
    rows = torch.cat([torch.arange(pl["q_off"][0, 0, c].item(), pl["q_off"][0, 0, c + 1].item(), device="cuda") for c in range(1, nQ, 2)])
    cols = torch.cat([torch.arange(pl["k_off"][0, 0, c].item(), pl["k_off"][0, 0, c + 1].item(), device="cuda") for c in range(nK) if c not in (7, 30)])
    ref, _ = formulas(Q[0, 0, rows], K[0, 0, cols], V[0, 0, cols], dO[0, 0, rows], d ** -0.5)
    for n in ("O", "dQ"):
        assert rel_norm(got[n][0, 0, rows], ref[n]) <= 2 * U, (n, rel_norm(got[n][0, 0, rows], ref[n]))


@pytest.mark.gpu
@pytest.mark.parametrize("N,nQ,nK,mean", [(5000, 100, 40, 4.0), (5000, 5, 3, 4.0), (2000, 40, 2, 30.0)])
def test_what_the_kept_keys_have_in_common_costs_little(N, nQ, nK, mean):
    """Keys with a large mean of their own in every K cluster: dQ subtracts the kept keys' mean.  With c that mean, an
    error e_ij of dS enters as e_ij (k_j - c): the keys' spread counts, their mean does not; the limit is 2 U.  K clusters
    of up to 512 rows have their exact mean, longer ones that of 512 evenly spaced rows."""
    svg2 = require_gpu()
    g = gen(N + nK)
    Q, K, V, dO = (randn(g, 1, 1, N, 64) for _ in range(4))
    K = (K.float() + mean).bfloat16()
    keep = torch.ones(nQ, nK, dtype=torch.bool)
    keep[1, 0] = False
    pl = even_plan(0, 1, 1, N, nQ, nK, keep)
    scale = 0.125 / mean
    got = sparse_step(svg2, pl, Q, K, V, dO, scale, perms=False)
    ref, _ = formulas(Q[0, 0], K[0, 0], V[0, 0], dO[0, 0], scale, rows_kept(pl, 0, 0, N))
    assert rel_norm(got["dQ"][0, 0], ref["dQ"]) <= 2 * U, rel_norm(got["dQ"][0, 0], ref["dQ"])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [600, 5000])
def test_what_an_empty_cluster_keeps_changes_nothing(N):
    """Empty Q clusters between small ones, and empty K clusters: their part of the selection has no rows.  With all of
    it listed and with none the gradients have the same bits, and NaN that only empty clusters keep reaches nothing."""
    svg2 = require_gpu()
    B, H, d, n = 1, 2, 64, 41
    g = gen(N + 1)
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    rng = np.random.default_rng(N)
    keep = torch.from_numpy(rng.random((n, n)) < 0.3)
    empty = torch.arange(n) % 2 == 1
    at = [0]  # the odd clusters are empty
    for i in range(n):
        at.append(at[-1] if i % 2 else N * (i // 2 + 1) // 21)
    got = []
    for listed in (False, True):
        k = keep.clone()
        k[empty], k[:, empty] = listed, listed
        k[~empty, 6] = False  # the rows of K cluster 6 and of Q cluster 8: kept by empty clusters alone
        k[8, ~empty] = False
        pl = even_plan(0, B, H, N, n, n, k)
        pl["q_off"] = pl["k_off"] = torch.tensor(at, dtype=torch.int32, device="cuda").expand(B, H, n + 1).contiguous()
        got.append(sparse_step(svg2, pl, Q, K, V, dO, 0.125, perms=False))
    assert same(*got)
    K[:, :, at[6]:at[7]] = torch.nan
    V[:, :, at[6]:at[7]] = torch.inf
    Q[:, :, at[8]:at[9]] = torch.nan
    dO[:, :, at[8]:at[9]] = torch.nan
    bad = sparse_step(svg2, pl, Q, K, V, dO, 0.125, perms=False)
    rows = torch.ones(N, dtype=torch.bool, device="cuda")
    rows[at[8]:at[9]] = False
    assert torch.equal(bad["dQ"][:, :, rows], got[1]["dQ"][:, :, rows])
    rows[:] = True
    rows[at[6]:at[7]] = False
    for m in ("dK", "dV"):
        assert torch.equal(bad[m][:, :, rows], got[1][m][:, :, rows]), m


@pytest.mark.gpu
@pytest.mark.parametrize("N", [300, 700, 4200])
@pytest.mark.parametrize("at", [5, 20])
def test_dense_nan_reaches_every_row_it_shares_a_pair_with(N, at):
    """A NaN query, key, value or gradient row, at places that each way of taking 2^x has: every gradient whose formula
    has it is NaN, in all its entries; the other queries' dQ keep their bits where only a query's row is NaN."""
    svg2 = require_gpu()
    g = gen(N)
    x = {n: randn(g, 1, 1, N, 64) for n in ("Q", "K", "V", "dO")}
    ref = dense_step(svg2, *x.values(), 0.125)
    others = torch.arange(N, device="cuda") != at
    for n, reached in (("Q", ("dK", "dV")), ("dO", ("dK", "dV")), ("K", ("dQ",)), ("V", ("dQ", "dK"))):
        bad = {m: t.clone() for m, t in x.items()}
        bad[n][0, 0, at] = torch.nan
        got = dense_step(svg2, *bad.values(), 0.125)
        for m in reached:
            assert torch.isnan(got[m]).all(), (n, m, torch.isnan(got[m]).float().mean().item())
        if n in ("Q", "dO"):
            assert torch.isnan(got["dQ"][0, 0, at]).all()
            assert torch.equal(got["dQ"][0, 0, others], ref["dQ"][0, 0, others]), n
        if n == "K":
            assert torch.isnan(got["dK"][0, 0, at]).all() and torch.isnan(got["dV"][0, 0, at]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H,N,nQ", [(17, 1100, 1024), (3, 3000, 200), (2, 20000, 40)])
def test_forward_plans_of_overlapping_clusters_stay_in_their_room(H, N, nQ):
    """Offsets of one plane that go up and down between 0 and N hold many more units than the plan has room for: what
    stands behind its part of the workspace and behind the workspace stays, and the other planes' rows are what they
    were (17 planes of 1024 clusters are planned by the kernels of large plans, with log-sum-exp too)."""
    svg2 = require_gpu()
    g = gen(33)
    d, nK = 64, 30
    Q, K, V = (randn(g, 1, H, N, d) for _ in range(3))
    pl = plan(34, 1, H, N, nQ, nK, 0.5)
    args = [pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")]
    bad = [args[0].clone(), *args[1:]]
    bad[0][0, H - 1] = torch.arange(nQ + 1, device="cuda", dtype=torch.int32) % 2 * N
    for lse in (None, torch.full((1, H, N), torch.nan, device="cuda")):
        size = (svg2.svg2_workspace_size if lse is None else svg2.svg2_sparse_attn_bwd_workspace_size)(1, H, N, d, nQ, nK)
        out = []
        for a in (args, bad):
            room = torch.full((size + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
            room[:256] = 0
            O = torch.zeros_like(Q)
            if lse is None:
                svg2.svg2_sparse_attn(Q, K, V, *a, 0.1, O, room[:size])
            else:
                svg2.svg2_sparse_attn_lse(Q, K, V, *a, 0.1, O, lse, room[:size])
            svg2.raise_on_device_error(room[:size])
            assert (room[size:] == 0x5a).all()
            out.append((O[:, :H - 1], None if lse is None else lse[:, :H - 1].clone()))
        assert torch.equal(out[0][0], out[1][0]) and (lse is None or torch.equal(out[0][1], out[1][1]))


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,d", [(1, 2, 4096, 64), (1, 1, 4097, 128), (1, 1, 4097, 64), (2, 1, 4500, 128), (1, 1, 5003, 64)])
def test_dense_gradients_of_long_rows(B, H, N, d):
    """The last length whose query units hand half of dS over as two numbers, and longer ones, which have a kernel of
    their own; 33 tiles and more, so every stage is reused many times."""
    test_dense_gradients(B, H, N, d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nQ,nK", [(2, 3), (100, 90), (100, 3), (2, 90)])
def test_sparse_gradients_of_long_streams(nQ, nK, d):
    """Streams of more than 4096 rows, for units inside one cluster (few clusters) and over several (many), for
    queries and keys each: the variants without split hand-over."""
    test_sparse_gradients(1, 1, 5500, d, nQ, nK, 0.97, {}, True)


@pytest.mark.gpu
def test_sparse_wait_that_runs_out_is_reported_and_leaves_the_workspace_usable():
    """The same as for the dense call, through the gathering producers: tiles of one piece and of many."""
    svg2 = require_gpu()
    g = gen(31)
    B, H, N, d = 1, 2, 1000, 128
    Q, K, V, dO = (randn(g, B, H, N, d) for _ in range(4))
    for nQ, nK in ((3, 4), (60, 50)):
        pl = plan(32 + nQ, B, H, N, nQ, nK, 0.7)
        want = sparse_step(svg2, pl, Q, K, V, dO, 0.1)
        ws = svg2.sparse_bwd_workspace(B, H, N, d, nQ, nK)
        grads = [torch.empty_like(Q) for _ in range(3)]
        svg2.svg2_set_wait_budget(ws, 1)
        svg2.svg2_sparse_attn_bwd(Q, K, V, want["O"], want["lse"], dO, *(pl[n] for n in ("q_off", "k_off", "sel_count", "sel_idx")),
                                  0.1, *grads, ws, perm_q=pl["perm_q"], perm_k=pl["perm_k"])
        assert svg2.svg2_check_status(ws)[0] == 5
        svg2.svg2_set_wait_budget(ws, 0)
        assert same(sparse_step(svg2, pl, Q, K, V, dO, 0.1, ws=ws), want)


@pytest.mark.gpu
@pytest.mark.parametrize("N,d", [(300, 64), (1000, 128), (4600, 64)])
@pytest.mark.parametrize("part,far", [(0.02, 1e4), (0.04, 100.0), (0.1, 300.0), (0.2, 30.0)])
def test_far_keys_of_no_weight_cost_dq_nothing(N, d, part, far):
    """Some keys lie far from the others in every column, on the side that the queries turn away from: their P is 0, so
    no product holds them, and what dQ subtracts must not either.  Dense with the far keys anywhere, and sparse with every
    cluster kept, the far ones in clusters of their own and anywhere; also with what all keys have in common added.
    The limit is 2 U."""
    svg2 = require_gpu()
    g = gen(N + d)
    Q, K, V, dO = (randn(g, 1, 1, N, d) for _ in range(4))
    Q = (Q.float() - 0.5).bfloat16()
    away = torch.randperm(N, device="cuda", generator=g)
    n = int(N * part)
    for common in (0.0, 4.0):
        x = K.float() + common
        x[0, 0, away[:n]] += far
        x = x.bfloat16()
        ref, _ = formulas(Q[0, 0], x[0, 0], V[0, 0], dO[0, 0], d ** -0.5)
        got = dense_step(svg2, Q, x, V, dO, d ** -0.5)
        assert rel_norm(got["dQ"][0, 0], ref["dQ"]) <= 2 * U, (common, rel_norm(got["dQ"][0, 0], ref["dQ"]))
        for nK in (3, 20):
            pl = even_plan(0, 1, 1, N, 4, nK, torch.ones(4, nK, dtype=torch.bool))
            for order in (away, torch.arange(N, device="cuda")):  # the far keys first, and where they are
                got = sparse_step(svg2, pl, Q, x[:, :, order].contiguous(), V[:, :, order].contiguous(), dO, d ** -0.5, perms=False)
                assert rel_norm(got["dQ"][0, 0], ref["dQ"]) <= 2 * U, (common, nK, rel_norm(got["dQ"][0, 0], ref["dQ"]))
