"""The mixture-of-experts operators and the general linear product: cases to time, and their plain forms.

Four operators that a model with routed SwiGLU experts needs next to the dense
MLP of this package:

  linear        y = act(x . W + bias) + residual (the router's logits, a dense
                layer with another activation, a projection with a bias)
  route         scores of E experts -> the k chosen experts of every token,
                their weights, and the (token, choice) pairs sorted by expert
  experts_up    h[r] = silu(x[t] . W_gate[e]) * (x[t] . W_up[e]) for every
                pair r = (token t, expert e), rows sorted by expert
  experts_down  y[t] = residual[t] + sum_j weight[t, j] h[r(t, j)] . W_down[e(t, j)]

`run` computes them with elementary torch operations in 32 bits (`own` false)
or through the package's entry points (`own` true).  `exact` evaluates the
definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # A decode step's projection back to the model width: 117 MB of weights
        # against 8 rows, with a bias and the residual stream.
        dict(name="linear_decode", op="linear", M=8, K=14336, N=4096, layout="kn", act="none",
             bias=True, residual=True, out="bf16"),
        # The first product of a non-gated MLP over a prompt of 4096 tokens.
        dict(name="linear_prefill_gelu", op="linear", M=4096, K=4096, N=14336, layout="nk",
             act="gelu_tanh", bias=True, residual=False, out="bf16"),
        # A router's logits for a prompt: few output columns, in f32.
        dict(name="linear_router", op="linear", M=4096, K=4096, N=64, layout="nk", act="none",
             bias=True, residual=False, out="f32"),
        # One generated token: only latency counts.
        dict(name="route_one_token", op="route", T=1, E=64, k=8, score="softmax", bias=False,
             groups=1, topk_groups=1, group_score="max", renormalize=True, scale=1.0,
             logits="f32", masked=0.0),
        # A long prompt through sigmoid scores with a balance bias and limited groups.
        dict(name="route_grouped", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_score="top2", renormalize=True, scale=2.0,
             logits="f32", masked=0.0),
        # An odd batch with bf16 logits, disabled experts and padding tokens.
        dict(name="route_masked", op="route", T=5001, E=60, k=4, score="softmax", bias=False,
             groups=1, topk_groups=1, group_score="max", renormalize=False, scale=1.0,
             logits="bf16", masked=0.05),
        # One generated token through 8 of 64 small experts.
        dict(name="up_one_token", op="up", T=1, E=64, k=8, d=2048, d_ff=1024, layout="kn",
             skew=0.0, padded=0.0),
        # A decode batch that reaches every one of 8 large experts (1.9 GB of weights).
        dict(name="up_decode", op="up", T=32, E=8, k=2, d=4096, d_ff=14336, layout="nk",
             skew=0.3, padded=0.0),
        # A prompt through 64 small experts, unevenly loaded.
        dict(name="up_prefill", op="up", T=4096, E=64, k=8, d=2048, d_ff=1024, layout="kn",
             skew=0.5, padded=0.0),
        # The second product of the same token.
        dict(name="down_one_token", op="down", T=1, E=64, k=8, d=2048, d_ff=1024, layout="kn",
             skew=0.0, padded=0.0, residual=True),
        # An odd batch of the small model's sizes, some tokens of it padding.
        dict(name="down_ragged", op="down", T=333, E=8, k=2, d=896, d_ff=4864, layout="nk",
             skew=1.0, padded=0.1, residual=True),
        # A prompt through 8 large experts.
        dict(name="down_prefill", op="down", T=4096, E=8, k=2, d=4096, d_ff=14336, layout="kn",
             skew=0.3, padded=0.0, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m=8):
    return max(m, _log_int(rng, lo, hi) // m * m)


def draw(rng):
    cap_flops = max(work(c)["flops"] for c in listed())
    cap_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["linear", "route", "up", "down"])
        if op == "linear":
            out = rng.choice(["bf16", "bf16", "f32"])
            case = dict(op=op, M=_log_int(rng, 1, 4099), K=_mult(rng, 64, 16384),
                        N=_mult(rng, 16, 14336), layout=rng.choice(["kn", "nk"]),
                        act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                        bias=rng.random() < 0.7, residual=rng.random() < 0.5, out=out)
        elif op == "route":
            groups = rng.choice([1, 1, 4, 8])
            k = rng.choice([1, 2, 4, 6, 8])
            E = groups * rng.randint(max(2, -(-16 // groups)), 512 // groups)
            topk_groups = groups if groups == 1 else rng.randint(groups // 2, groups)
            score = rng.choice(["softmax", "sigmoid"])
            bias = rng.random() < 0.5
            case = dict(op=op, T=_log_int(rng, 1, 16385), E=E, k=k, score=score, bias=bias,
                        groups=groups, topk_groups=topk_groups,
                        group_score=rng.choice(["max", "top2"]),
                        renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                        logits=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.1]))
        else:
            E = rng.choice([4, 8, 16, 60, 64, 128])
            case = dict(op=op, T=_log_int(rng, 1, 4099), E=E, k=rng.choice([1, 2, 4]),
                        d=_mult(rng, 256, 4096), d_ff=_mult(rng, 128, 8192),
                        layout=rng.choice(["kn", "nk"]), skew=rng.choice([0.0, 0.5, 1.5]),
                        padded=rng.choice([0.0, 0.2]))
            if op == "down":
                case["residual"] = rng.random() < 0.5
            if E * case["d"] * case["d_ff"] * 4 > 2 << 30:
                continue
        w = work(case)
        if w["flops"] <= cap_flops and w["bytes"] <= cap_bytes:
            return case


# ---- inputs --------------------------------------------------------------------

def _device():
    return torch.device("cuda", 0) if torch.cuda.is_available() else torch.device("cpu")


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    """Normal values, a piece at a time so that large weights need little beside themselves."""
    out = torch.empty(shape, dtype=dtype, device=gen.device)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device=gen.device).mul_(scale).to(dtype)
    return out


def _choices(gen, T, E, k, skew, padded):
    """Chosen experts [T, k] (distinct in a row; -1 for padding tokens) and weights."""
    pop = torch.randn(E, generator=gen, device=gen.device) * skew
    ids = torch.argsort(torch.randn(T, E, generator=gen, device=gen.device) + pop, dim=1,
                        descending=True)[:, :k].to(torch.int32).contiguous()
    weights = torch.rand(T, k, generator=gen, device=gen.device) + 0.1
    weights = weights / weights.sum(1, keepdim=True)
    if padded:
        pad = torch.rand(T, generator=gen, device=gen.device) < padded
        ids[pad] = -1
        weights[pad] = 0.0
    return ids, weights


def _sorted_pairs(ids, E):
    """(offsets [E + 1], order [T k], position [T, k]), int32: the flat (token, choice)
    indices by expert, in flat order within an expert; -1 where nothing stands."""
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    by = torch.sort(key, stable=True)[1]
    counts = (key[:, None] == torch.arange(E, device=ids.device)[None, :]).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    rank = torch.arange(flat.numel(), device=ids.device)
    live = rank < offsets[E]
    order = torch.where(live, by, torch.full_like(by, -1))
    position = torch.full_like(flat, -1)
    position[by] = torch.where(live, rank, torch.full_like(rank, -1))
    return (offsets.to(torch.int32), order.to(torch.int32),
            position.to(torch.int32).reshape(ids.shape))


def _select(case, logits, bias, dt):
    """Scores [T, E] and selection values (-inf where an expert cannot be chosen) in `dt`."""
    l = logits.to(dt)
    none = torch.full_like(l, -math.inf)
    l = torch.where(l > -math.inf, l, none)
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        e = torch.where(l == m, torch.ones_like(l), torch.exp(l - m))
        e = torch.where(l > -math.inf, e, torch.zeros_like(l))
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total > 0, total, torch.ones_like(total))
    if bias is not None:
        v = torch.where(l > -math.inf, s + bias.to(dt), none)
        v = torch.where(v > -math.inf, v, none)
    else:
        v = l            # both scores grow with the logit
    return s, v


def _group_values(case, s, v):
    """[T, groups]: the groups' values.  Without a bias, "max" compares logits."""
    T, E, G = v.shape[0], v.shape[1], case["groups"]
    if case["group_score"] == "max":
        return v.reshape(T, G, E // G).amax(2)
    c = v if case["bias"] else torch.where(v > -math.inf, s, v)
    top = torch.sort(c.reshape(T, G, E // G), dim=2, descending=True)[0][:, :, :2]
    a = top[:, :, 0]
    if top.shape[2] < 2:
        return a
    return a + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], torch.zeros_like(a))


def _limit(case, s, v):
    """Selection values with the experts of the groups that are not kept taken out."""
    if case["groups"] == 1:
        return v
    T, E, G = v.shape[0], v.shape[1], case["groups"]
    kept = torch.sort(_group_values(case, s, v), dim=1, descending=True, stable=True)[1]
    kept = kept[:, :case["topk_groups"]]
    keep = (torch.arange(G, device=v.device)[None, :, None] == kept[:, None, :]).any(2)
    keep = keep[:, :, None].expand(T, G, E // G).reshape(T, E)
    return torch.where(keep, v, torch.full_like(v, -math.inf))


def _route(case, logits, bias, dt):
    s, v = _select(case, logits, bias, dt)
    v = _limit(case, s, v)
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    chosen = top > -math.inf
    w = torch.where(chosen, torch.gather(s, 1, ids), torch.zeros_like(top))
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    ids = torch.where(chosen, ids, torch.full_like(ids, -1)).to(torch.int32)
    return ids, w * case["scale"]


def _clear_rows(case, logits, bias):
    """Rows whose choice hangs on less than the rounding of 32 bits have more than one
    right answer: they get the logits of rows without such a pair."""
    s, v = _select(case, logits, bias, torch.float64)

    def close(values, n):
        if values.shape[1] < 2:
            return torch.zeros(values.shape[0], dtype=torch.bool, device=values.device)
        a = torch.sort(values, dim=1, descending=True)[0][:, :n + 1]
        gap = a[:, :-1] - a[:, 1:]
        return ((gap < 4e-6) & (a[:, 1:] > -math.inf)).any(1)

    bad = torch.zeros(v.shape[0], dtype=torch.bool, device=v.device)
    if bias is not None:
        bad |= close(_limit(case, s, v), case["k"])
    if case["groups"] > 1 and (bias is not None or case["group_score"] == "top2"):
        bad |= close(_group_values(case, s, v), case["topk_groups"])
    if bad.any() and not bad.all():
        good = torch.nonzero(~bad)[:, 0]
        rows = torch.nonzero(bad)[:, 0]
        logits[rows] = logits[good[torch.arange(rows.numel(), device=v.device) % good.numel()]]
    return logits


def _inputs(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        st["x"] = _randn(gen, M, K)
        st["w"] = _randn(gen, *((K, N) if case["layout"] == "kn" else (N, K)),
                         scale=K ** -0.5)
        st["bias"] = _randn(gen, N, scale=0.5) if case["bias"] else None
        st["residual"] = (_randn(gen, M, N, dtype=_DT[case["out"]])
                          if case["residual"] else None)
    elif op == "route":
        T, E = case["T"], case["E"]
        logits = _randn(gen, T, E, scale=1.5, dtype=_DT[case["logits"]])
        bias = _randn(gen, E, scale=0.1, dtype=torch.float32) if case["bias"] else None
        if case["masked"]:
            off = torch.rand(E, generator=gen, device=gen.device) < case["masked"]
            off[0] = False
            pad = torch.rand(T, generator=gen, device=gen.device) < case["masked"]
            logits[:, off] = -math.inf
            logits[pad] = -math.inf
        st["logits"], st["bias"] = _clear_rows(case, logits, bias), bias
    else:
        T, E, k, d, f = case["T"], case["E"], case["k"], case["d"], case["d_ff"]
        ids, weights = _choices(gen, T, E, k, case["skew"], case["padded"])
        st["ids"], st["weights"] = ids, weights
        st["offsets"], st["order"], st["position"] = _sorted_pairs(ids, E)
        kn = case["layout"] == "kn"
        if op == "up":
            shape = (E, d, f) if kn else (E, f, d)
            st["x"] = _randn(gen, T, d)
            st["w_gate"] = _randn(gen, *shape, scale=d ** -0.5)
            st["w_up"] = _randn(gen, *shape, scale=d ** -0.5)
        else:
            shape = (E, f, d) if kn else (E, d, f)
            st["h"] = _randn(gen, T * k, f, scale=0.6)
            st["w_down"] = _randn(gen, *shape, scale=f ** -0.5)
            st["residual"] = _randn(gen, T, d) if case["residual"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] in ("up", "down"):
        import swiglu_mlp_projection_gb300 as swg
        st["routing"] = swg.Routing(st["ids"], st["weights"], st["offsets"], st["order"],
                                    st["position"])
    return st


# ---- one pass ------------------------------------------------------------------

def _act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * (0.5 ** 0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _run_own(st):
    import swiglu_mlp_projection_gb300 as swg
    case = st["case"]
    op = case["op"]
    if op == "linear":
        return swg.linear(st["x"], st["w"], bias=st["bias"], residual=st["residual"],
                          activation=case["act"], out_dtype=_DT[case["out"]],
                          layout=case["layout"])
    if op == "route":
        r = swg.route(st["logits"], case["k"], score=case["score"], bias=st["bias"],
                      groups=case["groups"], topk_groups=case["topk_groups"],
                      group_score=case["group_score"], renormalize=case["renormalize"],
                      scale=case["scale"])
        return [r.ids, r.weights, r.offsets, r.order, r.position]
    if op == "up":
        return swg.experts_up(st["x"], st["w_gate"], st["w_up"], st["routing"],
                              layout=case["layout"])
    return swg.experts_down(st["h"], st["w_down"], st["routing"], residual=st["residual"],
                            layout=case["layout"])


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    kn = case.get("layout") == "kn"
    if op == "linear":
        w = state["w"].float()
        v = torch.matmul(state["x"].float(), w if kn else w.t())
        if state["bias"] is not None:
            v = v + state["bias"].float()
        v = _act(case["act"], v)
        if state["residual"] is not None:
            v = v + state["residual"].float()
        return v.to(_DT[case["out"]])
    if op == "route":
        ids, w = _route(case, state["logits"], state["bias"], torch.float32)
        return [ids, w, *_sorted_pairs(ids, case["E"])]
    bounds = state["offsets"].tolist()
    if op == "up":
        T, k = state["ids"].shape
        h = torch.zeros(T * k, case["d_ff"], dtype=torch.float32, device=state["x"].device)
        for e in range(case["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if lo == hi:
                continue
            x = state["x"][state["order"][lo:hi].long() // k].float()
            g, u = state["w_gate"][e].float(), state["w_up"][e].float()
            g, u = torch.matmul(x, g if kn else g.t()), torch.matmul(x, u if kn else u.t())
            h[lo:hi] = g / (1.0 + torch.exp(-g)) * u
        return h.to(torch.bfloat16)
    T, k = state["ids"].shape
    y = torch.zeros(T, case["d"], dtype=torch.float32, device=state["h"].device)
    z = torch.zeros(T * k + 1, case["d"], dtype=torch.float32, device=state["h"].device)
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        w = state["w_down"][e].float()
        z[lo:hi] = torch.matmul(state["h"][lo:hi].float(), w if kn else w.t())
    if state["residual"] is not None:
        y = y + state["residual"].float()
    for j in range(k):
        y = y + state["weights"][:, j:j + 1] * z[state["position"][:, j].long()]
    return y.to(torch.bfloat16)


# ---- work and the exact values -----------------------------------------------------

def _reached(case):
    """Experts that a batch reaches: all, or what T k choices with equal chances find."""
    E, pairs = case["E"], case["T"] * case["k"]
    return min(E, pairs, max(1, int(round(E * (1.0 - (1.0 - case["k"] / E) ** case["T"])))))


def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (M * K + K * N) + o * M * N * (2 if case["residual"] else 1)
                + (2 * N if case["bias"] else 0), "flops": 2 * M * K * N}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        e = 4 if case["logits"] == "f32" else 2
        return {"bytes": e * T * E + (4 * E if case["bias"] else 0) + 16 * T * k + 4 * (E + 1),
                "flops": 4 * T * E}
    T, k, d, f = case["T"], case["k"], case["d"], case["d_ff"]
    rows = T * k * (1.0 - case["padded"])
    if op == "up":
        return {"bytes": int(2 * (2 * _reached(case) * d * f + T * d + T * k * f) + 4 * T * k),
                "flops": int(4 * rows * d * f)}
    return {"bytes": int(2 * (_reached(case) * d * f + rows * f
                              + T * d * (2 if case["residual"] else 1)) + 8 * T * k),
            "flops": int(2 * rows * d * f)}


def _exact_route(case, st):
    """Token by token: scores, kept groups, chosen experts, then the pairs by expert."""
    logits = st["logits"].to(torch.float64).cpu().numpy()
    bias = None if st["bias"] is None else st["bias"].to(torch.float64).cpu().numpy()
    T, E = logits.shape
    k, G = case["k"], case["groups"]
    size = E // G
    ids = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = logits[t]
        live = np.nonzero(l > -math.inf)[0]
        if not len(live):
            continue
        if case["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l[live].max())
            s /= s[live].sum()
        key = l if bias is None else s + bias
        if G > 1:
            gkey = []
            for g in range(G):
                own_live = live[(live >= g * size) & (live < (g + 1) * size)]
                if case["group_score"] == "max":
                    gkey.append(key[own_live].max() if len(own_live) else -math.inf)
                else:
                    two = np.sort((s if bias is None else key)[own_live])[::-1][:2]
                    gkey.append(two.sum() if len(two) else -math.inf)
            kept = np.argsort(-np.array(gkey), kind="stable")[:case["topk_groups"]]
            live = live[np.isin(live // size, kept)]
        best = live[np.argsort(-key[live], kind="stable")][:k]
        w = s[best]
        if case["renormalize"] and len(best):
            w = w / w.sum()
        ids[t, :len(best)], weights[t, :len(best)] = best, w * case["scale"]
    flat = ids.reshape(-1)
    order = [np.nonzero(flat == e)[0] for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum([len(o) for o in order])]).astype(np.int32)
    order = np.concatenate(order).astype(np.int32)
    position = np.full(T * k, -1, dtype=np.int32)
    position[order] = np.arange(len(order), dtype=np.int32)
    order = np.concatenate([order, np.full(T * k - len(order), -1, dtype=np.int32)])
    return [ids, weights, offsets, order, position.reshape(T, k)]


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and column block by column block."""
    st = _inputs(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "route":
        return _exact_route(case, st)

    def product(a, w, kn):
        n = w.shape[1] if kn else w.shape[0]
        out = torch.empty(a.shape[0], n, dtype=D, device=a.device)
        for c in range(0, n, 2048):
            part = w[:, c:c + 2048].to(D) if kn else w[c:c + 2048].to(D).t()
            out[:, c:c + 2048] = a @ part
        return out

    kn = case["layout"] == "kn"
    if op == "linear":
        v = product(st["x"].to(D), st["w"], kn)
        if st["bias"] is not None:
            v += st["bias"].to(D)
        if case["act"] == "silu":
            v = v * torch.sigmoid(v)
        elif case["act"] == "relu":
            v = v.clamp_min(0)
        elif case["act"] == "gelu":
            v = v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
        elif case["act"] == "gelu_tanh":
            z = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
            v = v * torch.sigmoid(2.0 * z)
        if st["residual"] is not None:
            v += st["residual"].to(D)
        return v
    T, k = st["ids"].shape
    ids = st["ids"].cpu().reshape(-1).tolist()
    of = [[] for _ in range(case["E"])]
    for flat, e in enumerate(ids):
        if e >= 0:
            of[e].append(flat)
    dev = st["ids"].device
    row = 0
    if op == "up":
        h = torch.zeros(T * k, case["d_ff"], dtype=D, device=dev)
        for e, flats in enumerate(of):
            if not flats:
                continue
            tok = torch.tensor(flats, device=dev) // k
            a = st["x"][tok].to(D)
            g = product(a, st["w_gate"][e], kn)
            h[row:row + len(flats)] = g * torch.sigmoid(g) * product(a, st["w_up"][e], kn)
            row += len(flats)
        return h
    y = torch.zeros(T, case["d"], dtype=D, device=dev)
    if st["residual"] is not None:
        y += st["residual"].to(D)
    for e, flats in enumerate(of):
        if not flats:
            continue
        idx = torch.tensor(flats, device=dev)
        z = product(st["h"][row:row + len(flats)].to(D), st["w_down"][e], kn)
        y.index_add_(0, idx // k, z * st["weights"].to(D).reshape(-1)[idx, None])
        row += len(flats)
    return y
