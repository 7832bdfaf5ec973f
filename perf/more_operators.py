"""Cases that time the operators between and behind a decoder layer's linears.

rope                 rotary positions on the query and key rows, forward or inverse
attn_fwd, attn_bwd   attention over packed sequences with shared key heads, and its
                     backward, which forms the probabilities again from the saved lse
logp_fwd, logp_bwd   log probability of a given token per row of logits, entropy and
                     the top alternatives, and the gradient of the logits

With `own` false, run() computes the operators from elementary torch operations;
with `own` true it makes the library's calls on the same state.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
NONE = -1  # a target that asks for nothing


def listed():
    return [
        # the Llama-8B layer's 8192 tokens, frequencies scaled for long contexts
        {"name": "rope_8b", "op": "rope", "T": 8192, "heads": 32, "kv": 8, "hd": 128, "rot": 128, "pairs": False,
         "scaled": True, "inverse": False, "dt": "bf16"},
        # gradients of an odd number of tokens, part of an odd head rotated, interleaved, fp32
        {"name": "rope_odd", "op": "rope", "T": 3001, "heads": 9, "kv": 3, "hd": 75, "rot": 34, "pairs": True,
         "scaled": False, "inverse": True, "dt": "f32"},
        # the Llama-60M layer's 2048 tokens as 8 sequences of 256
        {"name": "attn_fwd_60m", "op": "attn_fwd", "lq": _rep(256, 8), "lk": _rep(256, 8), "heads": 8, "kv": 8, "hd": 64,
         "causal": True, "window": 0, "dt": "bf16"},
        # the Llama-8B layer's 8192 tokens as 2 sequences of 4096
        {"name": "attn_fwd_8b", "op": "attn_fwd", "lq": "4096,4096", "lk": "4096,4096", "heads": 32, "kv": 8, "hd": 128,
         "causal": True, "window": 0, "dt": "bf16"},
        # 16 sequences that each add one token to the keys they have
        {"name": "attn_fwd_token", "op": "attn_fwd", "lq": _rep(1, 16), "heads": 32, "kv": 8, "hd": 128,
         "lk": "8192,5000,4096,4095,2047,1024,1000,777,512,300,129,128,64,31,2,1", "causal": True, "window": 0, "dt": "bf16"},
        # ragged packed sequences in fp32, an odd head, a window
        {"name": "attn_fwd_odd", "op": "attn_fwd", "lq": "1,513,0,1000,37,255", "lk": "1,513,5,1000,37,255", "heads": 9,
         "kv": 3, "hd": 75, "causal": True, "window": 300, "dt": "f32"},
        # the Llama-1.3B layer's 16384 tokens as ragged sequences
        {"name": "attn_bwd_1p3b", "op": "attn_bwd", "lq": "2048,2047,2000,1500,1999,1777,1024,1333,777,555,500,400,256,100,61,7",
         "lk": "", "heads": 16, "kv": 16, "hd": 128, "causal": True, "window": 0, "dt": "bf16"},
        # the Llama-8B layer's 8192 tokens as 2 sequences of 4096
        {"name": "attn_bwd_8b", "op": "attn_bwd", "lq": "4096,4096", "lk": "", "heads": 32, "kv": 8, "hd": 128,
         "causal": True, "window": 0, "dt": "bf16"},
        # one row of a large vocabulary with its 8 most likely tokens: a sampler's step
        {"name": "logp_fwd_token", "op": "logp_fwd", "T": 1, "V": 131072, "top": 8, "scale": 1.25, "dt": "bf16"},
        # 4096 rows of a generic vocabulary, no alternatives asked for: the loss of a training step
        {"name": "logp_fwd_rows", "op": "logp_fwd", "T": 4096, "V": 32000, "top": 0, "scale": 1.0, "dt": "bf16"},
        # an odd vocabulary in fp32, with the entropy's gradient
        {"name": "logp_bwd_odd", "op": "logp_bwd", "T": 1021, "V": 50001, "top": 0, "scale": 1.0, "dt": "f32", "ent": True},
        # the gradient of a training step's loss over 4096 rows of a generic vocabulary
        {"name": "logp_bwd_rows", "op": "logp_bwd", "T": 4096, "V": 32000, "top": 0, "scale": 1.0, "dt": "bf16", "ent": False},
    ]


def _rep(n, times):
    return ",".join([str(n)] * times)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_PAIRS = 2 * 32 * 4096 * 4096 * 128  # elements of a head times query-key pairs, as in the largest listed case


def _draw_attn(rng, op):
    hd = rng.choice([64, 128, 128, _log_int(rng, 8, 128), _log_int(rng, 8, 128)])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 3, 4])
    dt = rng.choice(["f32", "bf16", "bf16"])
    room, lq, lk = MOST_PAIRS // (1 if dt == "bf16" else 16) // (heads * max(hd, 64)), [], []
    long = _log_int(rng, 8, 4096)
    for _ in range(_log_int(rng, 1, 32)):
        n = _log_int(rng, 1, long)
        k = n if op == "attn_bwd" or rng.random() < 0.5 else n + _log_int(rng, 1, 4096)
        if sum(lq + [n]) > 16384 or max(lq + [n]) * max(lk + [k]) * (len(lq) + 1) > room:
            break
        lq.append(n)
        lk.append(k)
    lq, lk = lq or [16], lk or [16]
    return {"op": op, "lq": ",".join(map(str, lq)), "lk": ",".join(map(str, lk)), "heads": heads, "kv": kv, "hd": hd,
            "causal": rng.random() < 0.75, "window": rng.choice([0, 0, _log_int(rng, 1, 2048)]), "dt": dt}


def draw(rng):
    op = rng.choice(["rope", "attn_fwd", "attn_bwd", "logp_fwd", "logp_bwd"])
    if op in ("attn_fwd", "attn_bwd"):
        return _draw_attn(rng, op)
    dt = rng.choice(["f32", "bf16"])
    if op == "rope":
        hd, kv = rng.choice([64, 128, _log_int(rng, 8, 256)]), rng.choice([1, 2, 3, 8])
        heads = kv * rng.choice([1, 2, 4])
        T = min(_log_int(rng, 1, 16384), (1 << 26) // (ES[dt] * hd * (heads + kv)))
        rot = 2 * (hd // 2) if rng.random() < 0.6 else 2 * rng.randint(1, hd // 2)
        return {"op": op, "T": max(1, T), "heads": heads, "kv": kv, "hd": hd, "rot": rot, "pairs": rng.random() < 0.5,
                "scaled": rng.random() < 0.5, "inverse": rng.random() < 0.5, "dt": dt}
    V = _log_int(rng, 64, 131072)
    T = max(1, min(_log_int(rng, 1, 8192), (1 << 28) // (ES[dt] * V)))
    return {"op": op, "T": T, "V": V, "top": rng.choice([0, 0, 1, 5, 8, 20]) if op == "logp_fwd" else 0,
            "scale": rng.choice([1.0, 1.0, 0.7, 2.0]), "dt": dt, "ent": rng.random() < 0.5}


# ------------------------------------------------------------------ states ---
def _rope_state(case, g):
    T, hd, rot = case["T"], case["hd"], case["rot"]
    new = lambda *s: torch.randn(*s, device="cuda", generator=g).to(DT[case["dt"]])  # noqa: E731
    f = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if case["scaled"]:
        # wavelengths over the trained length of 8192 eight times as long, those under a quarter of it as they were
        smooth = ((8192 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = (1 - smooth) * f / 8 + smooth * f
    # packed sequences that begin at places of their own
    start = torch.randint(0, 131072, (1 + T // 1024,), device="cuda", generator=g)
    t = torch.arange(T, device="cuda")
    return {"case": case, "pos": (start[t // 1024] + t % 1024).int(), "f": f, "Q": new(T, case["heads"] * hd),
            "K": new(T, case["kv"] * hd)}


def _lens(case):
    lq = [int(x) for x in case["lq"].split(",")]
    return lq, [int(x) for x in case["lk"].split(",")] if case["lk"] else lq


def _cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def _padded(cu, lens):
    """Rows of a packed matrix as [sequences, longest], and which of them there are."""
    n = torch.arange(max(max(lens), 1), device="cuda")
    row = cu[:-1, None].long() + n
    live = row < cu[1:, None]
    return torch.where(live, row, 0), live


def _attn_state(case, g):
    lq, lk = _lens(case)
    H, G, hd, dt = case["heads"], case["kv"], case["hd"], DT[case["dt"]]
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    s = {"case": case, "cu_q": _cu(lq), "cu_k": _cu(lk), "Tq": sum(lq), "Tk": sum(lk), "batch": len(lq),
         "scale": 1 / math.sqrt(hd)}
    s["iq"], s["live_q"] = _padded(s["cu_q"], lq)
    s["ik"], s["live_k"] = _padded(s["cu_k"], lk)
    # queries and keys of some heads agree strongly with a few directions, so that rows differ in how sharp they are
    s["Q"] = (new(s["Tq"], H * hd) * (0.3 + 1.5 * torch.rand(s["Tq"], 1, device="cuda", generator=g))).to(dt)
    s["K"] = (new(s["Tk"], G * hd) + 0.5 * new(1, G * hd)).to(dt)
    s["V"] = (new(s["Tk"], G * hd) + 0.2).to(dt)
    if case["op"] == "attn_bwd":
        out = _plain_attn_fwd(s)  # what the forward of these rows saved
        s["O"], s["lse"] = out["O"], out["lse"]
        s["dO"] = (0.1 * new(s["Tq"], H * hd)).to(dt)
    return s


def _logp_state(case, g):
    T, V = case["T"], case["V"]
    # logits of a trained model: some tokens stand out, a few are switched off
    X = 2.0 * torch.randn(T, V, device="cuda", generator=g)
    X[:, :: max(1, V // 50)] += 4 * torch.rand(T, 1, device="cuda", generator=g)
    X[:, V // 3: V // 3 + min(7, V // 8)] = float("-inf")
    s = {"case": case, "X": X.to(DT[case["dt"]])}
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    t = torch.where((t >= V // 3) & (t < V // 3 + min(7, V // 8)), 0, t)
    s["target"] = torch.where(torch.rand(T, device="cuda", generator=g) < 0.05 * (T > 1), NONE, t).int()
    if case["op"] == "logp_bwd":
        x = s["X"].double() * case["scale"]
        lse = torch.logsumexp(x, 1)
        s["lse"] = lse.float()
        s["ent"] = (lse - torch.where(x > -math.inf, (x - lse[:, None]).exp() * x, 0.0).sum(1)).float()
        s["dlogp"] = -torch.rand(T, device="cuda", generator=g) / T
        s["dent"] = 0.01 * torch.randn(T, device="cuda", generator=g) / T if case["ent"] else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"rope": _rope_state, "attn": _attn_state, "logp": _logp_state}[case["op"].split("_")[0]](case, g)


# ------------------------------------------------------------ plain forms ---
def _plain_rope(s):
    case = s["case"]
    hd, rot = case["hd"], case["rot"]
    a = s["pos"].double()[:, None] * s["f"]
    c, n = a.cos().float()[:, None], a.sin().float()[:, None]
    if case["inverse"]:
        n = -n
    out = {}
    for name in ("Q", "K"):
        x = s[name].float().view(case["T"], -1, hd)
        y = x.clone()
        if case["pairs"]:
            e, o = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = e * c - o * n, o * c + e * n
        else:
            e, o = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = e * c - o * n, o * c + e * n
        out[name] = y.view(case["T"], -1).to(DT[case["dt"]])
    return out


def _heads(x, rows, n, hd):
    """[T, n hd] as [sequences, heads, longest, hd] in fp32."""
    return x.float().view(-1, n, hd)[rows].transpose(1, 2).contiguous()


def _masked_scores(s, q, k):
    """Scores of [sequences, kv heads, group * queries, keys], -inf where a query does not see a key."""
    case, (b, kv, _, hd) = s["case"], k.shape
    Lq, Lk = s["iq"].shape[1], k.shape[2]
    x = torch.matmul(q.view(b, kv, -1, hd), k.transpose(2, 3).contiguous()) * s["scale"]
    shift = (s["cu_k"].diff() - s["cu_q"].diff()).long()[:, None, None]
    i, j = torch.arange(Lq, device="cuda")[None, :, None] + shift, torch.arange(Lk, device="cuda")
    see = s["live_q"][:, :, None] & s["live_k"][:, None, :]
    if case["causal"]:
        see = see & (j <= i)
    if case["window"]:
        see = see & (j > i - case["window"])
        if not case["causal"]:
            see = see & (j < i + case["window"])
    return x.view(b, -1, Lq, Lk).masked_fill_(~see[:, None], -math.inf)


def _unpad(s, x, live, T):
    """The live rows of [sequences, heads, longest, hd], packed."""
    return x.transpose(1, 2)[live].reshape(T, -1)


def _plain_attn_fwd(s):
    case = s["case"]
    H, kv, hd = case["heads"], case["kv"], case["hd"]
    q, k, v = _heads(s["Q"], s["iq"], H, hd), _heads(s["K"], s["ik"], kv, hd), _heads(s["V"], s["ik"], kv, hd)
    x = _masked_scores(s, q, k)
    m = x.amax(3, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = x.sub_(m).exp_()
    z = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(len(q), kv, -1, p.shape[3]), v).view(q.shape)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (m + z.log()).squeeze(3)
    return {"O": _unpad(s, o, s["live_q"], s["Tq"]).to(DT[case["dt"]]),
            "lse": lse.transpose(1, 2)[s["live_q"]].t().contiguous()}


def _plain_attn_bwd(s):
    case = s["case"]
    H, kv, hd, dt = case["heads"], case["kv"], case["hd"], DT[case["dt"]]
    q, k, v = _heads(s["Q"], s["iq"], H, hd), _heads(s["K"], s["ik"], kv, hd), _heads(s["V"], s["ik"], kv, hd)
    do, o = _heads(s["dO"], s["iq"], H, hd), _heads(s["O"], s["iq"], H, hd)
    b, Lk = len(q), k.shape[2]
    lse = s["lse"].t()[s["iq"]].transpose(1, 2)[..., None]  # [sequences, heads, longest, 1]
    p = torch.where(lse > -math.inf, _masked_scores(s, q, k).sub_(lse).exp_(), 0.0)
    group = lambda x: x.reshape(b, kv, -1, x.shape[3])  # noqa: E731  the heads of one key head, one after another
    dv = torch.matmul(group(p).transpose(2, 3).contiguous(), group(do))
    dp = torch.matmul(group(do), v.transpose(2, 3).contiguous()).view(p.shape)
    ds = p.mul_(dp.sub_((do * o).sum(3, keepdim=True))).mul_(s["scale"])
    dq = torch.matmul(group(ds), k).view(q.shape)
    dk = torch.matmul(group(ds).transpose(2, 3).contiguous(), group(q))
    return {"dQ": _unpad(s, dq, s["live_q"], s["Tq"]).to(dt), "dK": _unpad(s, dk, s["live_k"], s["Tk"]).to(dt),
            "dV": _unpad(s, dv, s["live_k"], s["Tk"]).to(dt)}


def _plain_logp_fwd(s):
    case, raw = s["case"], s["X"].float()
    x = raw * case["scale"]
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    z = e.sum(1, keepdim=True)
    lse = m + z.log()
    t = s["target"].long()[:, None]
    at = torch.gather(x, 1, t.clamp(min=0)) - lse
    out = {"logp": torch.where(t >= 0, at, 0.0)[:, 0], "lse": lse[:, 0],
           "ent": (lse - torch.where(e > 0, e * x, 0.0).sum(1, keepdim=True) / z)[:, 0]}
    if case["top"]:
        # one whole number per logit, in the logits' order, the lower index first among equal ones
        bits = (raw + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = (order << 20) + ((1 << 20) - 1 - torch.arange(case["V"], device="cuda"))
        ids = key.topk(case["top"], 1).indices
        out["top_ids"], out["top_logp"] = ids.int(), torch.gather(x, 1, ids) - lse
    return out


def _plain_logp_bwd(s):
    case = s["case"]
    x = s["X"].float() * case["scale"] - s["lse"][:, None]
    p = x.exp()
    t = s["target"].long()[:, None]
    a = torch.where(t >= 0, s["dlogp"][:, None], 0.0)
    d = -a * p
    if s["dent"] is not None:
        d = d - torch.where(p > 0, s["dent"][:, None] * p * (x + s["ent"][:, None]), 0.0)
    d.scatter_add_(1, t.clamp(min=0), a)
    return (d * case["scale"]).to(DT[case["dt"]])


# -------------------------------------------------------- library's calls ---
def _own_attn(s):
    from orthogonal_reparameterized_cnp_amd import binding as B

    case, Tq, Tk = s["case"], s["Tq"], s["Tk"]
    H, kv, hd = case["heads"], case["kv"], case["hd"]
    if "desc" not in s:
        s["desc"] = B.attn_desc(H, kv, hd, case["dt"], causal=case["causal"], window=case["window"], scale=s["scale"])
        op = B.POETX_OP_FWD if case["op"] == "attn_fwd" else B.POETX_OP_BWD
        s["ws"] = torch.empty(B.poetx_attn_workspace_size(s["desc"], s["batch"], Tq, Tk, op), dtype=torch.uint8, device="cuda")
    if case["op"] == "attn_fwd":
        out = {"O": torch.empty_like(s["Q"]), "lse": torch.empty(H, Tq, device="cuda")}
        B.poetx_attn_fwd(s["desc"], s["batch"], Tq, Tk, s["cu_q"], s["cu_k"], s["Q"], H * hd, s["K"], kv * hd, s["V"], kv * hd,
                         out["O"], H * hd, out["lse"], s["ws"], s["ws"].numel())
        return out
    out = {"dQ": torch.empty_like(s["Q"]), "dK": torch.empty_like(s["K"]), "dV": torch.empty_like(s["V"])}
    B.poetx_attn_bwd(s["desc"], s["batch"], Tq, Tk, s["cu_q"], s["cu_k"], s["dO"], H * hd, s["Q"], H * hd, s["K"], kv * hd,
                     s["V"], kv * hd, s["O"], H * hd, s["lse"], out["dQ"], H * hd, out["dK"], kv * hd, out["dV"], kv * hd,
                     s["ws"], s["ws"].numel())
    return out


def _own(s):
    from orthogonal_reparameterized_cnp_amd import binding as B

    case, op = s["case"], s["case"]["op"]
    if op.startswith("attn"):
        return _own_attn(s)
    T = case["T"]
    if op == "rope":
        if "desc" not in s:
            s["desc"] = B.rope_desc(case["hd"], case["rot"], "pairs" if case["pairs"] else "half", case["dt"])
        hq, hk = case["heads"], case["kv"]
        nq, nk = hq * case["hd"], hk * case["hd"]
        out = {"Q": torch.empty_like(s["Q"]), "K": torch.empty_like(s["K"])}
        B.poetx_rope(s["desc"], T, s["pos"], s["f"], 1.0, case["inverse"], [s["Q"], s["K"]], [nq, nk], [hq, hk],
                     [out["Q"], out["K"]], [nq, nk])
        return out
    V = case["V"]
    if "desc" not in s:
        s["desc"] = B.logp_desc(V, case["dt"], case["top"], case["scale"])
    if op == "logp_bwd":
        dX = torch.empty_like(s["X"])
        B.poetx_logp_bwd(s["desc"], T, s["X"], V, s["target"], s["lse"], s["ent"], s["dlogp"], s["dent"], dX, V)
        return dX
    if "ws" not in s:
        s["ws"] = torch.empty(B.poetx_logp_workspace_size(s["desc"], T), dtype=torch.uint8, device="cuda")
    new = lambda *n: torch.empty(*n, device="cuda")  # noqa: E731
    out = {"logp": new(T), "lse": new(T), "ent": new(T)}
    if case["top"]:
        out["top_ids"] = torch.empty(T, case["top"], dtype=torch.int32, device="cuda")
        out["top_logp"] = new(T, case["top"])
    B.poetx_logp_fwd(s["desc"], T, s["X"], V, s["target"], out["logp"], out["lse"], out["ent"], out.get("top_ids"),
                     out.get("top_logp"), s["ws"], s["ws"].numel())
    return out


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd, "logp_fwd": _plain_logp_fwd,
            "logp_bwd": _plain_logp_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------------ costs ---
def _pairs(case):
    """Query-key pairs that see each other, over all sequences."""
    n = 0
    for q, k in zip(*_lens(case)):
        w = case["window"] or 1 << 40
        for i in range(k - q, k):
            hi = min(k, i + 1) if case["causal"] else min(k, i + w)
            n += max(0, hi - max(0, i - w + 1))
    return n


def work(case):
    op, es = case["op"], ES[case["dt"]]
    if op == "rope":
        e = case["T"] * (case["heads"] + case["kv"])
        return {"bytes": 2 * e * case["hd"] * es + 4 * case["T"] + 4 * case["rot"], "flops": 3 * e * case["rot"]}
    if op.startswith("attn"):
        lq, lk = _lens(case)
        q, k, n = sum(lq) * case["heads"], sum(lk) * case["kv"], _pairs(case) * case["heads"]
        if op == "attn_fwd":
            return {"bytes": (2 * q + 2 * k) * case["hd"] * es + 4 * q, "flops": 4 * case["hd"] * n}
        return {"bytes": (4 * q + 4 * k) * case["hd"] * es + 4 * q, "flops": 10 * case["hd"] * n}
    e = case["T"] * case["V"]
    if op == "logp_fwd":
        return {"bytes": e * es + case["T"] * (16 + 8 * case["top"]), "flops": 6 * e}
    return {"bytes": 2 * e * es + 20 * case["T"], "flops": 8 * e}


# ------------------------------------------------ the definition in 64 bits ---
def _exact_rope(case, s):
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                       (-1.0 if case["inverse"] else 1.0) * s["pos"].double()[:, None] * s["f"])[:, None]
    out = {}
    for name in ("Q", "K"):
        x = s[name].double().view(case["T"], -1, case["hd"])
        r = x[..., :case["rot"]]
        if not case["pairs"]:
            r = torch.stack(r.chunk(2, -1), -1)
        z = torch.view_as_complex(r.reshape(*x.shape[:2], -1, 2).contiguous()) * turn
        y = torch.view_as_real(z)
        y = y.flatten(-2) if case["pairs"] else torch.cat([y[..., 0], y[..., 1]], -1)
        out[name] = torch.cat([y, x[..., case["rot"]:]], -1).flatten(1)
    return out


def _exact_attn(case, s):
    lq, lk = _lens(case)
    H, kv, hd, bwd = case["heads"], case["kv"], case["hd"], case["op"] == "attn_bwd"
    share = torch.arange(H, device="cuda") // (H // kv)
    outs, a, c = [], 0, 0
    for n, m in zip(lq, lk):
        q = s["Q"][a:a + n].double().view(n, H, hd).permute(1, 0, 2)
        k, v = (s[x][c:c + m].double().view(m, kv, hd).permute(1, 0, 2)[share] for x in ("K", "V"))
        back = torch.arange(n, device="cuda")[:, None] + (m - n) - torch.arange(m, device="cuda")  # how far back a key is
        hide = torch.zeros(n, m, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= back < 0
        if case["window"]:
            hide |= back.abs() >= case["window"]
        x = (torch.bmm(q, k.permute(0, 2, 1)) / math.sqrt(hd)).masked_fill(hide, -math.inf)
        if not bwd:
            lse = torch.logsumexp(x, 2) if m else torch.full((H, n), -math.inf, device="cuda", dtype=torch.float64)
            p = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)[:, :, None])
            outs.append((torch.bmm(p, v).permute(1, 0, 2).reshape(n, H * hd), lse.t()))
        else:
            do, o = (s[y][a:a + n].double().view(n, H, hd).permute(1, 0, 2) for y in ("dO", "O"))
            lse = s["lse"][:, a:a + n].double()
            p = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)[:, :, None])
            g = p * (torch.bmm(do, v.permute(0, 2, 1)) - (do * o).sum(2, keepdim=True)) / math.sqrt(hd)
            fold = lambda t: t.view(kv, H // kv, m, hd).sum(1).permute(1, 0, 2).reshape(m, kv * hd)  # noqa: E731
            outs.append((torch.bmm(g, k).permute(1, 0, 2).reshape(n, H * hd), fold(torch.bmm(g.permute(0, 2, 1), q)),
                         fold(torch.bmm(p.permute(0, 2, 1), do))))
        a, c = a + n, c + m
    names = ("dQ", "dK", "dV") if bwd else ("O", "lse")
    out = {name: torch.cat([o[i] for o in outs]) for i, name in enumerate(names)}
    if not bwd:
        out["lse"] = out["lse"].t().contiguous()
    return out


def _exact_logp(case, s):
    T, V = s["X"].shape
    rows = torch.arange(T, device="cuda")
    lx = torch.log_softmax(s["X"].double() * case["scale"], 1)
    p = lx.exp()
    t = s["target"].long()
    given = t >= 0
    plogp = torch.where(p > 0, p * lx, 0.0)
    if case["op"] == "logp_fwd":
        best = s["X"].double().argmax(1)
        out = {"logp": torch.where(given, lx[rows, t.clamp(min=0)], 0.0),
               "lse": s["X"].double()[rows, best] * case["scale"] - lx[rows, best], "ent": -plogp.sum(1)}
        if case["top"]:
            by = s["X"].float().sort(dim=1, descending=True, stable=True).indices[:, :case["top"]]
            out["top_ids"], out["top_logp"] = by.int(), torch.gather(lx, 1, by)
        return out
    # at the saved lse and entropy, as the operator is given them
    x = s["X"].double() * case["scale"] - s["lse"].double()[:, None]
    p = x.exp()
    hit = torch.zeros_like(p)
    hit[rows[given], t[given]] = 1.0
    d = (s["dlogp"].double() * given)[:, None] * (hit - p)
    if s["dent"] is not None:
        d -= s["dent"].double()[:, None] * torch.where(p > 0, p * (x + s["ent"].double()[:, None]), 0.0)
    return d * case["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "logp": _exact_logp}[case["op"].split("_")[0]](case, s)
