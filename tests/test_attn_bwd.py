"""The attentions' log-sum-exp and gradients against the formulas in 64 bits.

Tolerances, elementwise, from the formulas (u = 2^-8, half a bf16 step).  A probability carries a relative
error of at most EP: the cubic exponential's 7.5e-5, twice (once in P, once in lse), and the error of
a float32 score, at most (d + 2) 2^-24 scale sum |q k|, twice.  P and dS are rounded to bf16, O too
(it enters delta = dO.O), and the outputs.  dQ is summed as scale sum_j dS_ij (k_j - c) with c the mean of up to
512 evenly spaced keys (the same in exact arithmetic, where a row of dS sums to zero), so an error e_ij of dS
enters as e_ij (k_j - c), and the float32 sums over N keys add N 2^-24 times their terms' magnitudes (which the
bf16 terms cover everywhere else).  With |.| taken inside every sum this bounds each entry; for
errors of independent sign the relative 2-norm stays below 2 u, which is checked where the sums do not cancel."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu

U = 2.0 ** -8


def formulas(q, k, v, do, scale, keep=None):
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
    S = min(512, k.shape[0])
    c = k[torch.arange(S, device=k.device) * k.shape[0] // S].mean(0)
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
