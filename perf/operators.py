"""Cases that time the training-step operators around the reparameterised linears.

norm_fwd, norm_bwd   layer norm or RMS norm of token rows, optionally of the sum
                     with a residual stream, and its backward with the summed
                     weight and bias gradients
muon                 one optimiser step on the packed skew parameters: momentum,
                     Newton-Schulz orthogonalisation of every b x b block, decay
orth                 the same orthogonalisation of dense rows x cols matrices

With `own` false, run() computes the operators from elementary torch operations;
with `own` true it makes the library's calls on the same state.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
EPS = 1e-5  # norm
NS_STEPS, NS_A, NS_B, NS_C, NS_EPS = 5, 3.4445, -4.7750, 2.0315, 1e-7
LR, BETA, DECAY, RMS = 1e-3, 0.95, 0.1, 0.2  # muon

LLAMA60M = "512,512,512,512,512,512,512,512,512,1376,512,1376,1376,512"
LLAMA8B = "4096,4096,4096,1024,4096,1024,4096,4096,4096,14336,4096,14336,14336,4096"


def listed():
    return [
        # one token of a decoder layer of hidden size 4096: the latency of a call
        {"name": "norm_fwd_token", "op": "norm_fwd", "T": 1, "d": 4096, "dt": "bf16", "kind": "rms", "res": True},
        # the Llama-60M layer's 2048 tokens
        {"name": "norm_fwd_60m", "op": "norm_fwd", "T": 2048, "d": 512, "dt": "bf16", "kind": "layer", "res": False},
        # odd rows of an odd width (the Llama-1.3B MLP's) in fp32: no row is 16-byte aligned but every fourth
        {"name": "norm_fwd_odd", "op": "norm_fwd", "T": 1021, "d": 5461, "dt": "f32", "kind": "layer", "res": False},
        # the Llama-8B layer's 8192 tokens, residual added on the way in
        {"name": "norm_fwd_8b", "op": "norm_fwd", "T": 8192, "d": 4096, "dt": "bf16", "kind": "rms", "res": True},
        # the smallest workload's 64 tokens of 256
        {"name": "norm_bwd_small", "op": "norm_bwd", "T": 64, "d": 256, "dt": "f32", "kind": "layer", "res": False},
        # a ragged batch of an MLP-wide input
        {"name": "norm_bwd_odd", "op": "norm_bwd", "T": 3001, "d": 1376, "dt": "bf16", "kind": "layer", "res": False},
        # the Llama-1.3B layer's 16384 tokens, the residual's gradient added on the way out
        {"name": "norm_bwd_1p3b", "op": "norm_bwd", "T": 16384, "d": 2048, "dt": "bf16", "kind": "rms", "res": True},
        # one 256 x 256 linear of block size 32: 8 small blocks per side
        {"name": "muon_256", "op": "muon", "dims": "256,256", "b": 32, "fresh": False},
        # every side of the Llama-60M layer, block size 256, last blocks of 96; the first step after a merge (q = 0)
        {"name": "muon_60m", "op": "muon", "dims": LLAMA60M, "b": 256, "fresh": True},
        # every side of the Llama-8B layer, block size 512: 160 blocks
        {"name": "muon_8b", "op": "muon", "dims": LLAMA8B, "b": 512, "fresh": False},
        # a Llama-60M MLP matrix kept dense, fp32
        {"name": "orth_60m", "op": "orth", "count": 1, "rows": 512, "cols": 1376, "dt": "f32"},
        # a Llama-8B MLP matrix kept dense, bf16
        {"name": "orth_8b", "op": "orth", "count": 1, "rows": 4096, "cols": 14336, "dt": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "muon", "orth"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log_int(rng, 32, 14336)
        dt = rng.choice(["f32", "bf16"])
        T = min(_log_int(rng, 1, 16384), (1 << 26) // (ES[dt] * d))
        return {"op": op, "T": max(1, T), "d": d, "dt": dt, "kind": rng.choice(["layer", "rms"]),
                "res": rng.random() < 0.5}
    if op == "muon":
        b = _log_int(rng, 8, 1024)
        room, dims = 120.0 * 512**3, []
        for _ in range(2 * rng.randint(1, 7)):
            d = min(_log_int(rng, 32, 14336), b * int(room / b**3))
            if d < 2:
                break
            dims.append(d)
            room -= -(-d // b) * float(b) ** 3
        return {"op": op, "dims": ",".join(map(str, dims)), "b": b, "fresh": rng.random() < 0.3}
    rows, cols, dt = _log_int(rng, 16, 4096), _log_int(rng, 16, 14336), rng.choice(["f32", "bf16"])
    count = rng.choice([1, 1, 1, 2, 3])
    while count * min(rows, cols) * rows * cols > (1 << 37):
        rows, cols = max(16, rows * 3 // 4), max(16, cols * 3 // 4)
    return {"op": op, "count": count, "rows": rows, "cols": cols, "dt": dt}


def _norm_state(case, g):
    T, d, dt = case["T"], case["d"], DT[case["dt"]]
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    # a residual stream: rows of differing scale and offset, a few wide columns
    X = new(T, d) * (0.5 + torch.rand(T, 1, device="cuda", generator=g) * 2) + 0.3 * new(T, 1)
    X[:, :: max(1, d // 7)] *= 6
    s = {"case": case, "w": 1 + 0.2 * new(d), "b": 0.1 * new(d) if case["kind"] == "layer" else None}
    if case["op"] == "norm_fwd":
        s["X"] = X.to(dt)
        s["R"] = new(T, d).to(dt) if case["res"] else None
        return s
    s["S"] = X.to(dt)
    s["dY"] = (0.1 * new(T, d)).to(dt)
    s["dS"] = (0.1 * new(T, d)).to(dt) if case["res"] else None
    # what the forward of these rows saved: the means (layer norm) and reciprocal deviations
    S = s["S"].double()
    mean = S.mean(1) if case["kind"] == "layer" else torch.zeros(T, device="cuda", dtype=torch.float64)
    rstd = ((S - mean[:, None]).square().mean(1) + EPS).rsqrt()
    s["stats"] = (torch.stack([mean, rstd]) if case["kind"] == "layer" else rstd[None]).float()
    return s


def _muon_state(case, g):
    dims, b = [int(x) for x in case["dims"].split(",")], case["b"]
    nb = [-(-d // b) for d in dims]
    r = torch.tensor([min(b, d - k * b) for d, n in zip(dims, nb) for k in range(n)], device="cuda")
    i, j = torch.triu_indices(b, b, 1, device="cuda")
    live = j[None, :] < r[:, None]  # the other slots of a partial block hold no parameter

    def packed(std, rank):
        """Skew gradients as training gives them: a few strong directions over noise."""
        U = torch.randn(len(r), b, rank, device="cuda", generator=g)
        V = torch.randn(len(r), rank, b, device="cuda", generator=g) / math.sqrt(rank)
        D = torch.bmm(U, V) + 0.5 * torch.randn(len(r), b, b, device="cuda", generator=g)
        return torch.where(live, std * (D[:, i, j] - D[:, j, i]), 0.0)

    q = torch.where(live, (0.0 if case["fresh"] else 0.005) * torch.randn(live.shape, device="cuda", generator=g), 0.0)
    return {"case": case, "dims": dims, "b": b, "nb": nb, "r": r, "i": i, "j": j, "live": live, "q": q,
            "dq": packed(3.0, 4), "m": packed(2.0, 8)}


def _orth_state(case, g):
    n, m, c = case["rows"], case["cols"], case["count"]
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    rank = max(1, min(n, m) // 16)
    G = torch.bmm(new(c, n, rank), new(c, rank, m)) / math.sqrt(rank) + 0.7 * new(c, n, m)
    return {"case": case, "G": (1e-3 * G).to(DT[case["dt"]])}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "muon":
        return _muon_state(case, g)
    return _orth_state(case, g) if case["op"] == "orth" else _norm_state(case, g)


# ------------------------------------------------------------ plain forms ---
def _plain_norm_fwd(s):
    dt, layer = DT[s["case"]["dt"]], s["case"]["kind"] == "layer"
    S = s["X"] if s["R"] is None else (s["X"].float() + s["R"].float()).to(dt)
    x = S.float()
    mean = x.mean(1) if layer else None
    xc = x - mean[:, None] if layer else x
    rstd = (xc.square().mean(1) + EPS).rsqrt()
    y = xc * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    out = {"Y": y.to(dt), "stats": torch.stack([mean, rstd]) if layer else rstd[None]}
    if s["R"] is not None:
        out["S"] = S
    return out


def _plain_norm_bwd(s):
    dt, layer = DT[s["case"]["dt"]], s["case"]["kind"] == "layer"
    x, dy, rstd = s["S"].float(), s["dY"].float(), s["stats"][-1][:, None]
    xh = (x - s["stats"][0][:, None]) * rstd if layer else x * rstd
    g = dy * s["w"]
    t = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        t = t - g.mean(1, keepdim=True)
    dx = t * rstd
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    out = {"dX": dx.to(dt), "dw": (dy * xh).sum(0)}
    if layer:
        out["db"] = dy.sum(0)
    return out


def _ns_step(X, A, c=NS_C):
    return NS_A * X + torch.bmm(NS_B * A + c * torch.bmm(A, A), X)


def _plain_muon(s):
    q, m, i, j, b = s["q"], s["m"], s["i"], s["j"], s["b"]
    m.mul_(BETA).add_(s["dq"], alpha=1 - BETA)
    u = BETA * m + (1 - BETA) * s["dq"]
    X = torch.zeros(len(q), b, b, device="cuda")
    X[:, i, j] = u
    X = X - X.transpose(1, 2)
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        X = _ns_step(X, -torch.bmm(X, X))
    scale = RMS * s["r"].float().sqrt()[:, None]
    new = q - LR * (scale * X[:, i, j] + DECAY * q)
    q.copy_(torch.where(s["live"], new, q))
    return {"q": q, "m": m}


def _plain_orth(s):
    X = s["G"].float()
    if X.shape[1] > X.shape[2]:
        X = X.transpose(1, 2).contiguous()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        X = _ns_step(X, torch.bmm(X, X.transpose(1, 2).contiguous()))
    X = X * (RMS * math.sqrt(max(X.shape[1:])))
    if s["G"].shape[1] > s["G"].shape[2]:
        X = X.transpose(1, 2)
    return X.to(s["G"].dtype).contiguous()


# -------------------------------------------------------- library's calls ---
def _own(s):
    from orthogonal_reparameterized_cnp_amd import binding as B

    case, op = s["case"], s["case"]["op"]
    if op == "muon":
        if "ws" not in s:  # the workspace and the per-side views that a program keeps
            s["ws"] = torch.empty(B.poetx_muon_workspace_size(s["dims"], s["b"]), dtype=torch.uint8, device="cuda")
            s["sides"] = [list(s[k].split(s["nb"])) for k in ("q", "dq", "m")]
            s["hp"] = B.muon_params(lr=LR, beta=BETA, weight_decay=DECAY, rms=RMS, nesterov=True, steps=NS_STEPS)
        q, dq, m = s["sides"]
        B.poetx_muon_step_batch(q, dq, m, s["dims"], s["b"], s["hp"], s["ws"], s["ws"].numel())
        return {"q": s["q"], "m": s["m"]}
    if op == "orth":
        c, n, m = s["G"].shape
        dt = B.DTYPES[case["dt"]]
        if "ws" not in s:
            s["ws"] = torch.empty(B.poetx_orthogonalize_workspace_size(c, n, m, dt), dtype=torch.uint8, device="cuda")
            s["hp"] = B.ns_params(rms=RMS, steps=NS_STEPS)
        out = torch.empty_like(s["G"])
        B.poetx_orthogonalize(c, n, m, dt, s["G"], m, n * m, out, m, n * m, s["hp"], s["ws"], s["ws"].numel())
        return out
    T, d = case["T"], case["d"]
    if "desc" not in s:
        s["desc"] = B.norm_desc(d, case["kind"], case["dt"], EPS)
    if op == "norm_fwd":
        out = {"Y": torch.empty_like(s["X"]),
               "stats": torch.empty(2 if case["kind"] == "layer" else 1, T, device="cuda")}
        if s["R"] is not None:
            out["S"] = torch.empty_like(s["X"])
        B.poetx_norm_fwd(s["desc"], T, s["X"], d, s["R"], d, s["w"], s["b"], out.get("S"), d, out["Y"], d, out["stats"])
        return out
    if "ws" not in s:
        s["ws"] = torch.empty(B.poetx_norm_workspace_size(s["desc"], T), dtype=torch.uint8, device="cuda")
    out = {"dX": torch.empty_like(s["S"]), "dw": torch.empty_like(s["w"])}
    if s["b"] is not None:
        out["db"] = torch.empty_like(s["b"])
    B.poetx_norm_bwd(s["desc"], T, s["dY"], d, s["S"], d, s["w"], s["stats"], s["dS"], d, out["dX"], d, out["dw"],
                     out.get("db"), s["ws"], s["ws"].numel())
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "muon": _plain_muon,
            "orth": _plain_orth}[state["case"]["op"]](state)


# ------------------------------------------------------------------ costs ---
def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        e = case["T"] * case["d"]
        passes = 2 + (2 if op == "norm_fwd" else 1) * case["res"] + (op == "norm_bwd")
        vecs = 1 + (case["kind"] == "layer")
        return {"bytes": passes * e * ES[case["dt"]] + 4 * vecs * (case["T"] + case["d"] * (1 if op == "norm_fwd" else 2)),
                "flops": (8 if op == "norm_fwd" else 14) * e}
    if op == "muon":
        b, slots, cube = case["b"], 0, 0
        for d in (int(x) for x in case["dims"].split(",")):
            for k in range(-(-d // b)):
                r = min(b, d - k * b)
                slots += r * (r - 1) // 2
                cube += r**3
        # three products a step whose results are symmetric or skew: half of 2 r^3 each
        return {"bytes": 20 * slots, "flops": 3 * NS_STEPS * cube}
    r, k = sorted((case["rows"], case["cols"]))
    return {"bytes": 2 * case["count"] * r * k * ES[case["dt"]],
            "flops": case["count"] * NS_STEPS * (r * r * k + r**3 + 2 * r * r * k)}


# ------------------------------------------------ the definition in 64 bits ---
def _exact_norm(case, s):
    layer, x = case["kind"] == "layer", s["X" if case["op"] == "norm_fwd" else "S"].double()
    w = s["w"].double()
    if case["op"] == "norm_fwd":
        out = {}
        if s["R"] is not None:
            out["S"] = x + s["R"].double()
            x = out["S"].to(DT[case["dt"]]).double()  # the stored sum is what is normalised
        n = x.shape[1]
        mu = x.sum(1, keepdim=True) / n * layer
        var = (x * x).sum(1, keepdim=True) / n - mu * mu
        sd = torch.sqrt(var + EPS)
        out["Y"] = (x - mu) / sd * w + (s["b"].double() if layer else 0.0)
        out["stats"] = torch.cat([mu, 1 / sd], 1).t().contiguous() if layer else (1 / sd).t().contiguous()
        return out
    st, n = s["stats"].double(), x.shape[1]
    mu, rs = (st[0][:, None], st[1][:, None]) if layer else (0.0, st[0][:, None])
    dy = s["dY"].double()
    # dL/dx_k = rs (w_k dy_k - (sum_i w_i dy_i) / n - xh_k (sum_i w_i dy_i xh_i) / n), the middle term for layer norm
    xh = (x - mu) * rs
    p1, p2 = (dy @ w)[:, None] / n * layer, ((dy * xh) @ w)[:, None] / n
    out = {"dX": rs * (dy * w - p1 - xh * p2) + (s["dS"].double() if s["dS"] is not None else 0.0),
           "dw": torch.einsum("td,td->d", dy, xh)}
    if layer:
        out["db"] = torch.ones(len(dy), device="cuda", dtype=torch.float64) @ dy
    return out


def _poly(X):
    """p(p(...p(X / |X|))), p(X) = (a + A (b + c A)) X with A = X X^T."""
    X = X / (torch.linalg.matrix_norm(X, keepdim=True) + NS_EPS)
    eye = torch.eye(X.shape[1], device="cuda", dtype=torch.float64)
    for _ in range(NS_STEPS):
        A = torch.bmm(X, X.transpose(1, 2))
        X = torch.bmm(NS_A * eye + torch.bmm(A, NS_B * eye + NS_C * A), X)
    return X


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s)
    if case["op"] == "orth":
        G = s["G"].double()
        flip = G.shape[1] > G.shape[2]
        O = _poly(G.transpose(1, 2).contiguous() if flip else G) * RMS * math.sqrt(max(G.shape[1:]))
        return O.transpose(1, 2).contiguous() if flip else O
    q, g, m, i, j, b = s["q"].double(), s["dq"].double(), s["m"].double(), s["i"], s["j"], s["b"]
    m = BETA * m + (1 - BETA) * g
    M = torch.zeros(len(q), b, b, device="cuda", dtype=torch.float64)
    u = BETA * m + (1 - BETA) * g
    M[:, i, j], M[:, j, i] = u, -u
    O = _poly(M)[:, i, j] * RMS * torch.sqrt(s["r"].double())[:, None]
    return {"q": torch.where(s["live"], (1 - LR * DECAY) * q - LR * O, q), "m": m}
