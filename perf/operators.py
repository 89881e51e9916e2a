"""The training-side operators of the attention layer: what is measured.

Four operators.  dense: one training step through dense attention, forward (output and log-sum-exp) and
backward (dQ, dK, dV).  sparse: the same through the variable-block sparse attention on a plan of kept
(Q cluster, K cluster) pairs, with the row permutations of the layer.  norm: layer norm over the last
dimension (the norm in front of Q and K, or of the layer's input).  norm_bwd: its gradients.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
# elements of one float32 score matrix that a plain pass holds at a time (planes are taken together up to it)
PLAIN_SCORES = 1 << 31


def listed():
    return [
        # a short clip's crop on one head of 64: the smallest call, where launches count
        dict(name="dense 1x100 d64", op="dense", B=1, H=1, N=100, d=64),
        # a small batch of odd length on the narrow head: every tile ragged
        dict(name="dense 6x1333 d64", op="dense", B=2, H=3, N=1333, d=64),
        # the 480p-like layer of the tests (8 heads of 12480 tokens), the dense fine-tuning step
        dict(name="dense 8x12480 d128", op="dense", B=1, H=8, N=12480, d=128),
        # two heads of the 720p video layer, the longest sequence
        dict(name="dense 2x75600 d128", op="dense", B=1, H=2, N=75600, d=128),
        # the tiny layer, one head: 16 x 32 clusters, a Q cluster that keeps nothing
        dict(name="sparse 1x4096 d64", op="sparse", B=1, H=1, N=4096, d=64, nQ=16, nK=32, density=0.5, empty=True),
        # the 480p-like layer at the density of a flat top-p selection
        dict(name="sparse 8x12480 d128", op="sparse", B=1, H=8, N=12480, d=128, nQ=64, nK=256, density=0.6, empty=False),
        # two heads of the 720p layer at the density that sparse fine-tuning aims at
        dict(name="sparse 2x75600 d128", op="sparse", B=1, H=2, N=75600, d=128, nQ=100, nK=500, density=0.28, empty=False),
        # the norm of one tiny layer's Q rows in float32: launch-bound
        dict(name="norm 4096x64 f32", op="norm", rows=4096, width=64, dtype=F32, affine=True),
        # the norm of 40 heads' Q rows of the 720p layer: short rows, bandwidth
        dict(name="norm 3024000x128 bf16", op="norm", rows=3024000, width=128, dtype=BF16, affine=True),
        # gradients of an odd, small norm
        dict(name="norm_bwd 1333x77 bf16", op="norm_bwd", rows=1333, width=77, dtype=BF16, affine=True),
        # gradients of the Q norm of the 720p layer: a long reduction for two short vectors
        dict(name="norm_bwd 3024000x128 bf16", op="norm_bwd", rows=3024000, width=128, dtype=BF16, affine=True),
        # gradients of the norm of the layer's input (40 heads x 128 wide)
        dict(name="norm_bwd 75600x5120 bf16", op="norm_bwd", rows=75600, width=5120, dtype=BF16, affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dense", "sparse", "norm", "norm_bwd"))
    if op in ("dense", "sparse"):
        d = rng.choice((64, 128))
        N = _log(rng, 2 if op == "dense" else 200, 30000)
        planes = max(1, min(24, int(2e9 / (N * N)), int(3e5 / N)))
        B = rng.randint(1, min(3, planes))
        case = dict(op=op, B=B, H=rng.randint(1, planes // B), N=N, d=d)
        if op == "sparse":
            most = max(2, min(400, N // 20))
            case.update(nQ=_log(rng, 1, most), nK=_log(rng, 2, most), density=round(rng.uniform(0.15, 0.95), 2),
                        empty=rng.random() < 0.3)
        return case
    width = rng.choice((64, 128, 128, _log(rng, 3, 8000), 8 * _log(rng, 3, 1000)))
    return dict(op=op, rows=_log(rng, 1, min(2000000, int(2e8 / width))), width=width, dtype=rng.choice((BF16, BF16, F32)),
                affine=rng.random() < 0.8)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _planes(case, g):
    """Q, K as rows of a Gaussian mixture (shared component map, separate centres), V and dO normal; bf16."""
    P, N, d = case["B"] * case["H"], case["N"], case["d"]
    comps = max(1, min(200, N // 32))
    which = torch.randint(comps, (P, (N + 15) // 16), device="cuda", generator=g).repeat_interleave(16, 1)[:, :N]
    out = []
    for _ in range(2):
        centres = _rand(g, P, comps, d)
        x = centres.gather(1, which[..., None].expand(P, N, d)) + 0.25 * _rand(g, P, N, d)
        out.append(x.bfloat16())
    out += [_rand(g, P, N, d).bfloat16(), (0.02 * _rand(g, P, N, d)).bfloat16()]
    return [x.view(case["B"], case["H"], N, d) for x in out]


def _labels(case, k, g):
    """Cluster labels [P, N] with unequal sizes, some clusters empty where there are many."""
    P, N = case["B"] * case["H"], case["N"]
    w = 0.2 + torch.rand(P, k, device="cuda", generator=g)
    if k > 8:
        w[:, 3] = 0
    return torch.multinomial(w, N, replacement=True, generator=g)


def _clusters(lab, k):
    perm = torch.sort(lab, dim=1, stable=True).indices
    off = torch.zeros(lab.shape[0], k + 1, dtype=torch.int64, device="cuda")
    off[:, 1:] = torch.zeros_like(off[:, 1:]).scatter_add_(1, lab, torch.ones_like(lab)).cumsum(1)
    return perm, off


def _permuted(x, perm):
    B, H, N, d = x.shape
    return x.view(B * H, N, d).gather(1, perm[..., None].expand(-1, -1, d)).view(B, H, N, d)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("dense", "sparse"):
        B, H, N, d = (case[x] for x in ("B", "H", "N", "d"))
        s["scale"] = 1.0 / math.sqrt(d)
        s["Q"], s["K"], s["V"], s["dO"] = _planes(case, g)
        if case["op"] == "sparse":
            nQ, nK = case["nQ"], case["nK"]
            perm_q, q_off = _clusters(_labels(case, nQ, g), nQ)
            perm_k, k_off = _clusters(_labels(case, nK, g), nK)
            keep = torch.rand(B * H, nQ, nK, device="cuda", generator=g) < case["density"]
            keep[:, :, 0] = True
            if case["empty"]:
                keep[:, nQ // 2] = False
            i32 = lambda t, *shape: t.to(torch.int32).view(B, H, *shape).contiguous()  # noqa: E731
            s["Q"], s["K"], s["V"] = _permuted(s["Q"], perm_q), _permuted(s["K"], perm_k), _permuted(s["V"], perm_k)
            s.update(perm_q=i32(perm_q, N), perm_k=i32(perm_k, N), q_off=i32(q_off, nQ + 1), k_off=i32(k_off, nK + 1),
                     sel_count=i32(keep.sum(2), nQ),
                     sel_idx=i32(torch.sort(keep.to(torch.uint8), dim=2, descending=True, stable=True).indices, nQ, nK))
    else:
        dtype = torch.bfloat16 if case["dtype"] == BF16 else torch.float32
        R, W = case["rows"], case["width"]
        # activations: channels of unequal scale around unequal means
        x = _rand(g, R, W).mul_(0.5 + torch.rand(W, device="cuda", generator=g)).add_(0.3 * _rand(g, W))
        s["X"], s["eps"] = x.to(dtype), 1e-6
        del x
        s["gamma"] = 1 + 0.1 * _rand(g, W) if case["affine"] else None
        s["beta"] = 0.1 * _rand(g, W) if case["affine"] else None
        if case["op"] == "norm_bwd":
            s["dY"] = (0.02 * _rand(g, R, W)).to(dtype)
            # the forward pass's statistics, which a training program keeps
            s["mean"], s["rstd"] = _statistics(s["X"], s["eps"])
    if own:
        from sparse_attention_video_head_b200 import svg2
        if case["op"] == "dense":
            s["ws"] = svg2.dense_bwd_workspace(B, H, N, d)
        elif case["op"] == "sparse":
            s["ws"] = svg2.sparse_bwd_workspace(B, H, N, d, nQ, nK)
        elif case["op"] == "norm_bwd":
            s["ws"] = svg2.layer_norm_bwd_workspace(R, W)
    return s


def _statistics(x, eps):
    x = x.float()
    mean = x.mean(1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + eps)


def _attention(q, k, v, do, scale, keep):
    """One training step of softmax attention on float32 planes [P, N, d]; keep: which pairs count, or None."""
    s = (q @ k.mT).mul_(scale)
    if keep is not None:
        s.masked_fill_(~keep, -math.inf)
    m = s.amax(2, keepdim=True).clamp_(min=-1e30)
    p = s.sub_(m).exp_()
    l = p.sum(2, keepdim=True)
    lse = (m + l.log())[..., 0]
    p.div_(l.clamp(min=1e-30))
    o = p @ v
    dv = p.mT @ do
    dp = do @ v.mT
    ds = dp.sub_((p * dp).sum(2, keepdim=True)).mul_(p)
    return o, lse, (ds @ k).mul_(scale), (ds.mT @ q).mul_(scale), dv


def _kept_rows(s, P, N):
    """Per plane, what expands the plan to token pairs: the cluster of each permuted row, and the kept pairs."""
    nQ, nK = s["case"]["nQ"], s["case"]["nK"]
    rows = torch.arange(N, device="cuda").expand(P, N).contiguous()
    of = lambda off, n: torch.searchsorted(off.view(P, n + 1)[:, 1:].long().contiguous(), rows, right=True)  # noqa: E731
    listed_ = torch.arange(nK, device="cuda") < s["sel_count"].view(P, nQ, 1)
    keep = torch.zeros(P, nQ, nK, dtype=torch.bool, device="cuda")
    keep.scatter_(2, s["sel_idx"].view(P, nQ, nK).long(), listed_)
    return of(s["q_off"], nQ), of(s["k_off"], nK), keep


def _run_attention(s):
    case = s["case"]
    P, N, d = case["B"] * case["H"], case["N"], case["d"]
    q, k, v, do = (s[x].view(P, N, d) for x in ("Q", "K", "V", "dO"))
    sparse = case["op"] == "sparse"
    if sparse:
        cq, ck, kept = _kept_rows(s, P, N)
        to_q, to_k = s["perm_q"].view(P, N).long(), s["perm_k"].view(P, N).long()
        do = do.gather(1, to_q[..., None].expand(P, N, d))
    parts = []
    step = max(1, min(P, PLAIN_SCORES // (N * N)))
    for a in range(0, P, step):  # the score matrices of all planes together need not fit the card
        b = min(P, a + step)
        keep = None
        if sparse:
            plane = torch.arange(a, b, device="cuda")[:, None, None]
            keep = kept[plane, cq[a:b, :, None], ck[a:b, None, :]]
        parts.append(_attention(q[a:b].float(), k[a:b].float(), v[a:b].float(), do[a:b].float(), s["scale"], keep))
    o, lse, dq, dk, dv = (torch.cat(x) for x in zip(*parts))
    if sparse:  # rows back in token order
        back = lambda x, to: torch.empty_like(x).scatter_(1, to[..., None].expand(P, N, d), x)  # noqa: E731
        o, dq, dk, dv = back(o, to_q), back(dq, to_q), back(dk, to_k), back(dv, to_k)
    shape = (case["B"], case["H"], N)
    out = {n: x.bfloat16().view(*shape, d) for n, x in (("O", o), ("dQ", dq), ("dK", dk), ("dV", dv))}
    out["lse"] = lse.view(shape)
    return out


def _run_norm(s):
    x = s["X"].float()
    mean, rstd = _statistics(x, s["eps"])
    y = (x - mean[:, None]) * rstd[:, None]
    if s["gamma"] is not None:
        y = y * s["gamma"] + s["beta"]
    return {"Y": y.to(s["X"].dtype), "mean": mean, "rstd": rstd}


def _run_norm_bwd(s):
    dy = s["dY"].float()
    rstd = s["rstd"][:, None]
    xhat = (s["X"].float() - s["mean"][:, None]) * rstd
    out = {"dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    g = dy if s["gamma"] is None else dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    out["dX"] = dx.to(s["X"].dtype)
    return out


def _run_own(s):
    from sparse_attention_video_head_b200 import svg2
    case = s["case"]
    if case["op"] in ("dense", "sparse"):
        Q, K, V, dO, ws = (s[x] for x in ("Q", "K", "V", "dO", "ws"))
        O, dQ, dK, dV = (torch.empty_like(Q) for _ in range(4))
        lse = torch.empty(Q.shape[:3], dtype=torch.float32, device="cuda")
        if case["op"] == "dense":
            svg2.svg2_dense_attn_lse(Q, K, V, s["scale"], O, lse, ws)
            svg2.svg2_dense_attn_bwd(Q, K, V, O, lse, dO, s["scale"], dQ, dK, dV, ws)
        else:
            plan = [s[x] for x in ("q_off", "k_off", "sel_count", "sel_idx")]
            svg2.svg2_sparse_attn_lse(Q, K, V, *plan, s["scale"], O, lse, ws, perm_q=s["perm_q"])
            svg2.svg2_sparse_attn_bwd(Q, K, V, O, lse, dO, *plan, s["scale"], dQ, dK, dV, ws, perm_q=s["perm_q"],
                                      perm_k=s["perm_k"])
        return {"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}
    X = s["X"]
    if case["op"] == "norm":
        Y = torch.empty_like(X)
        mean, rstd = (torch.empty(X.shape[0], dtype=torch.float32, device="cuda") for _ in range(2))
        svg2.svg2_layer_norm(X, s["gamma"], s["beta"], s["eps"], Y, mean, rstd)
        return {"Y": Y, "mean": mean, "rstd": rstd}
    dX = torch.empty_like(X)
    dgamma, dbeta = (torch.empty(X.shape[1], dtype=torch.float32, device="cuda") for _ in range(2))
    svg2.svg2_layer_norm_bwd(X, s["dY"], s["gamma"], s["mean"], s["rstd"], dX, dgamma, dbeta, s["ws"])
    return {"dX": dX, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _run_norm(state) if op == "norm" else _run_norm_bwd(state) if op == "norm_bwd" else _run_attention(state)


def work(case):
    if case["op"] in ("dense", "sparse"):
        P, N, d = case["B"] * case["H"], case["N"], case["d"]
        pairs = P * N * N * case.get("density", 1.0)
        # Q, K, V, dO in, O, dQ, dK, dV out, the log-sum-exp; two products forward, five backward
        return {"bytes": P * N * (8 * 2 * d + 4), "flops": 14 * pairs * d}
    R, W, e = case["rows"], case["width"], 2 if case["dtype"] == BF16 else 4
    if case["op"] == "norm":
        return {"bytes": 2 * R * W * e + 8 * R + (8 * W if case["affine"] else 0), "flops": 8 * R * W}
    return {"bytes": 3 * R * W * e + 8 * R + (12 if case["affine"] else 8) * W, "flops": 14 * R * W}


def exact(case, seed):
    """The same in 64 bits, from the definitions: softmax row by row over the listed keys, gradients by the chain rule."""
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        x = s["X"].double()
        if case["op"] == "norm":
            mean = x.sum(1) / case["width"]
            x -= mean[:, None]
            rstd = ((x * x).sum(1) / case["width"] + s["eps"]) ** -0.5
            x *= rstd[:, None]
            if s["gamma"] is not None:
                x = x.mul_(s["gamma"].double()).add_(s["beta"].double())
            return {"Y": x, "mean": mean, "rstd": rstd}
        dy, r = s["dY"].double(), s["rstd"].double()[:, None]
        x = x.sub_(s["mean"].double()[:, None]).mul_(r)
        dgamma, dbeta = (dy * x).sum(0), dy.sum(0)
        if s["gamma"] is not None:
            dy *= s["gamma"].double()
        along = (dy * x).sum(1, keepdim=True) / case["width"]
        dy -= dy.sum(1, keepdim=True) / case["width"]
        return {"dX": dy.sub_(x.mul_(along)).mul_(r), "dgamma": dgamma, "dbeta": dbeta}
    B, H, N, d = (case[x] for x in ("B", "H", "N", "d"))
    f64 = dict(dtype=torch.float64, device="cuda")
    O, dQ, dK, dV = (torch.zeros(B, H, N, d, **f64) for _ in range(4))
    lse = torch.zeros(B, H, N, **f64)
    rows = max(1, (1 << 29) // N)
    for b in range(B):
        for h in range(H):
            q, k, v, do = (s[x][b, h].double() for x in ("Q", "K", "V", "dO"))
            tq = tk = torch.arange(N, device="cuda")
            weight = None
            if case["op"] == "sparse":
                tq, tk = s["perm_q"][b, h].long(), s["perm_k"][b, h].long()
                nQ, nK = case["nQ"], case["nK"]
                table = torch.zeros(nQ, nK, **f64)
                idx, cnt = s["sel_idx"][b, h].tolist(), s["sel_count"][b, h].tolist()
                for i in range(nQ):
                    table[i, idx[i][: cnt[i]]] = 1.0
                cluster = lambda off, n: torch.repeat_interleave(torch.arange(n, device="cuda"), off.long().diff())  # noqa: E731
                weight = table[:, cluster(s["k_off"][b, h], nK)]
                own_q = cluster(s["q_off"][b, h], nQ)
            gk, gv = torch.zeros(N, d, **f64), torch.zeros(N, d, **f64)
            for a in range(0, N, rows):
                at = slice(a, min(N, a + rows))
                x = q[at] @ k.T * s["scale"]
                if weight is not None:
                    x += weight[own_q[at]].log()
                top = x.max(1, keepdim=True).values
                top = torch.where(top > -math.inf, top, torch.zeros_like(top))
                x = torch.exp(x.sub_(top))
                total = x.sum(1, keepdim=True)
                lse[b, h, at] = (total.log() + top)[:, 0]
                x /= torch.where(total > 0, total, torch.ones_like(total))
                g = do[tq[at]]
                O[b, h, tq[at]] = x @ v
                gv += x.T @ g
                y = g @ v.T
                y = x * (y - (x * y).sum(1, keepdim=True))
                dQ[b, h, tq[at]] = y @ k * s["scale"]
                gk += y.T @ q[at] * s["scale"]
                del x, y
            dK[b, h, tk], dV[b, h, tk] = gk, gv
    return {"O": O, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}
