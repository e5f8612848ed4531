"""The pre-norm of an MLP block, its 8-bit rows, and tokens sorted by expert: cases to time, and their plain forms.

What a model's MLP block needs around the products of this package, in serving
and in training:

  norm       s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight; y in the
             inputs' type, or as e4m3 codes with a scale for each row; and the
             gradients of x and weight
  up_fp8     the FP8 up projection of such rows: h = silu(x . W_gate) * (x . W_up)
             with x's codes and scales as they are
  permute    rows of x copied to the places of their k chosen experts (rows
             sorted by expert, as routing gives them), and the gradient of x
  unpermute  y[t] = residual[t] + sum_j weight[t, j] z[place of (t, j)], and the
             gradients of z and weight

`run` computes them with elementary torch operations in 32 bits (`own` false)
or through the package's entry points (`own` true).  `exact` evaluates the
definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
_E4M3_MAX = 448.0


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # One generated token on its way into the MLP: only latency counts.
        dict(name="norm_one_token", op="norm", M=1, d=4096, dtype="bf16", weight="bf16",
             residual=True, out="same", eps=1e-6),
        # A prompt's rows on their way into an FP8 product.
        dict(name="norm_prefill_fp8", op="norm", M=8192, d=8192, dtype="bf16", weight="bf16",
             residual=True, out="e4m3", eps=1e-5),
        # f32 rows of an odd width: no row but the first starts on a 16-byte boundary.
        dict(name="norm_f32_odd", op="norm", M=5001, d=897, dtype="f32", weight="f32",
             residual=False, out="same", eps=1e-6),
        # A training step's gradients of the block's input and of the norm's weight.
        dict(name="norm_backward", op="norm_backward", M=8192, d=4096, dtype="bf16",
             weight="bf16", ds=True, eps=1e-6),
        # The same for an odd batch of the small model.
        dict(name="norm_backward_ragged", op="norm_backward", M=333, d=896, dtype="f32",
             weight="f32", ds=False, eps=1e-6),
        # A decode step with rows that come quantized: the weights are read once.
        dict(name="up_fp8_decode", op="up_fp8", M=16, d=4096, d_ff=14336),
        # A prompt with rows that come quantized.
        dict(name="up_fp8_prefill", op="up_fp8", M=4096, d=4096, d_ff=14336),
        # One generated token to 8 of 64 experts.
        dict(name="permute_one_token", op="permute", T=1, E=64, k=8, d=2048, dtype="bf16",
             skew=0.0, padded=0.0),
        # A long prompt's quantized rows, with their scales.
        dict(name="permute_prefill_fp8", op="permute", T=16384, E=256, k=8, d=4096, dtype="e4m3",
             skew=0.5, padded=0.0),
        # The gradient of a padded odd batch's rows.
        dict(name="permute_backward_ragged", op="permute_backward", T=5001, E=60, k=4, d=2048,
             dtype="bf16", skew=0.5, padded=0.1),
        # The experts' results of a prompt, weighted and added to the residual stream.
        dict(name="unpermute_prefill", op="unpermute", T=4096, E=64, k=8, d=4096, dtype="bf16",
             skew=0.5, padded=0.05, residual=True),
        # Its gradients: of every expert's rows, and of the router's weights.
        dict(name="unpermute_backward", op="unpermute_backward", T=4096, E=64, k=8, d=2048,
             dtype="bf16", skew=0.5, padded=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A model width: most are multiples of 8, some of nothing."""
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.25 else max(8, d // 8 * 8)


def draw(rng):
    cap_flops = max(work(c)["flops"] for c in listed())
    cap_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "norm_backward", "up_fp8", "permute",
                         "permute_backward", "unpermute", "unpermute_backward"])
        if op in ("norm", "norm_backward"):
            dtype = rng.choice(["bf16", "bf16", "f32"])
            case = dict(op=op, M=_log_int(rng, 1, 16385), d=_width(rng, 64, 16384), dtype=dtype,
                        weight=rng.choice([dtype, "f32"]), eps=rng.choice([1e-6, 1e-5]))
            if op == "norm":
                case["residual"] = rng.random() < 0.6
                case["out"] = rng.choice(["same", "e4m3"])
            else:
                case["ds"] = rng.random() < 0.6
        elif op == "up_fp8":
            case = dict(op=op, M=_log_int(rng, 1, 4097),
                        d=max(128, _log_int(rng, 128, 8192) // 16 * 16),
                        d_ff=max(64, _log_int(rng, 64, 14336) // 8 * 8))
        else:
            dtype = rng.choice(["bf16", "bf16", "f32"] + (["e4m3"] if op == "permute" else []))
            case = dict(op=op, T=_log_int(rng, 1, 16385), E=rng.choice([8, 16, 60, 64, 128, 256]),
                        k=rng.choice([1, 2, 3, 4, 6, 8]), d=_width(rng, 128, 8192), dtype=dtype,
                        skew=rng.choice([0.0, 0.5, 1.5]), padded=rng.choice([0.0, 0.2]))
            if op == "unpermute":
                case["residual"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] <= cap_flops and w["bytes"] <= cap_bytes:
            return case


# ---- inputs --------------------------------------------------------------------

def _device():
    return torch.device("cuda", 0) if torch.cuda.is_available() else torch.device("cpu")


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    """Normal values, a piece at a time so that large tensors need little beside themselves."""
    out = torch.empty(shape, dtype=dtype, device=gen.device)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device=gen.device).mul_(scale).to(dtype)
    return out


def _stream_rows(gen, M, d, dtype):
    """A residual stream: rows of different sizes, a few columns far larger than the rest."""
    size = torch.exp(0.5 * torch.randn(M, 1, generator=gen, device=gen.device))
    col = 1.0 + 20.0 * (torch.rand(d, generator=gen, device=gen.device) < 0.004).float()
    return (torch.randn(M, d, generator=gen, device=gen.device) * size * col).to(dtype)


def _codes(rows):
    """(e4m3 codes as bytes, scales): each row over its largest magnitude, in 32 bits."""
    rows = rows.float()
    amax = rows.abs().amax(1, keepdim=True)
    inv = torch.where(amax > 0, _E4M3_MAX / amax, torch.zeros_like(amax))
    c = (rows * inv).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return c.view(torch.uint8), (amax / _E4M3_MAX)[:, 0].contiguous()


def _weight_codes(gen, n, k):
    """An [n, k] weight matrix in e4m3 with a scale per row, a block of rows at a time."""
    codes = torch.empty(n, k, dtype=torch.uint8, device=gen.device)
    scales = torch.empty(n, dtype=torch.float32, device=gen.device)
    step = max(1, (1 << 26) // k)
    for i in range(0, n, step):
        w = _randn(gen, min(step, n - i), k, scale=k ** -0.5)
        codes[i:i + step], scales[i:i + step] = _codes(w)
    return codes, scales


def _choices(gen, T, E, k, skew, padded):
    """Chosen experts [T, k] (distinct in a row; -1 for padding tokens and for single
    choices that found no room) and weights."""
    pop = torch.randn(E, generator=gen, device=gen.device) * skew
    ids = torch.argsort(torch.randn(T, E, generator=gen, device=gen.device) + pop, dim=1,
                        descending=True)[:, :k].to(torch.int32).contiguous()
    weights = torch.rand(T, k, generator=gen, device=gen.device) + 0.1
    weights = weights / weights.sum(1, keepdim=True)
    if padded:
        gone = torch.rand(T, 1, generator=gen, device=gen.device) < padded
        gone = gone | (torch.rand(T, k, generator=gen, device=gen.device) < 0.01)
        ids[gone.expand(T, k)] = -1
        weights[gone.expand(T, k)] = 0.0
    return ids, weights


def _sorted_pairs(ids, E):
    """(offsets [E + 1], order [T k], position [T, k]), int32: the flat (token, choice)
    indices by expert, in flat order within an expert; -1 where nothing stands."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    by = torch.sort(key, stable=True)[1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0)
    rank = torch.arange(flat.numel(), device=ids.device)
    live = rank < offsets[E]
    order = torch.where(live, by, torch.full_like(by, -1))
    position = torch.full_like(flat, -1)
    position[by] = torch.where(live, rank, torch.full_like(rank, -1))
    return (offsets.to(torch.int32), order.to(torch.int32),
            position.to(torch.int32).reshape(ids.shape))


def _inputs(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_backward"):
        M, d, dt = case["M"], case["d"], _DT[case["dtype"]]
        st["x"] = _stream_rows(gen, M, d, dt)     # norm_backward: s
        st["weight"] = (1.0 + 0.3 * torch.randn(d, generator=gen, device=gen.device)).to(
            _DT[case["weight"]])
        if op == "norm":
            st["residual"] = _randn(gen, M, d, dtype=dt) if case["residual"] else None
        else:
            st["dy"] = _randn(gen, M, d, dtype=dt)
            st["ds"] = _randn(gen, M, d, scale=2.0, dtype=dt) if case["ds"] else None
    elif op == "up_fp8":
        st["codes"], st["scales"] = _codes(_randn(gen, case["M"], case["d"]))
        st["w_gate"], st["s_gate"] = _weight_codes(gen, case["d_ff"], case["d"])
        st["w_up"], st["s_up"] = _weight_codes(gen, case["d_ff"], case["d"])
    else:
        T, E, k, d = case["T"], case["E"], case["k"], case["d"]
        st["ids"], st["weights"] = _choices(gen, T, E, k, case["skew"], case["padded"])
        st["offsets"], st["order"], st["position"] = _sorted_pairs(st["ids"], E)
        dt = _DT.get(case["dtype"], torch.bfloat16)
        if op == "permute":
            st["x"] = _randn(gen, T, d, dtype=dt)
            if case["dtype"] == "e4m3":
                st["x"], st["scales"] = _codes(st["x"])
        else:
            st["z"] = _randn(gen, T * k, d, dtype=dt)
            if op == "unpermute":
                st["residual"] = _randn(gen, T, d, dtype=dt) if case["residual"] else None
            if op == "unpermute_backward":
                st["dy"] = _randn(gen, T, d, dtype=dt)
    return st


def prepare(case, seed):
    return _inputs(case, seed)


# ---- one pass ------------------------------------------------------------------

def _run_own(st):
    import swiglu_mlp_projection_gb300 as swg
    case = st["case"]
    op = case["op"]
    if op == "norm":
        call = swg.rms_norm_fp8 if case["out"] == "e4m3" else swg.rms_norm
        r = call(st["x"], st["weight"], residual=st["residual"], eps=case["eps"])
        y, s = r if case["residual"] else (r, None)
        y = [y.codes.view(torch.float8_e4m3fn), y.scales] if case["out"] == "e4m3" else [y]
        return y if s is None else y + [s]
    if op == "norm_backward":
        return swg.rms_norm_backward(st["dy"], st["x"], st["weight"], ds=st["ds"],
                                     eps=case["eps"])
    if op == "up_fp8":
        return swg.swiglu_up_fp8(swg.Fp8Rows(st["codes"], st["scales"]),
                                 swg.Fp8Weights(st["w_gate"], st["w_up"], st["s_gate"],
                                                st["s_up"]))
    r = swg.Routing(st["ids"], st["weights"], st["offsets"], st["order"], st["position"])
    if op == "permute":
        if case["dtype"] == "e4m3":
            rows = swg.permute(swg.Fp8Rows(st["x"], st["scales"]), r)
            return [rows.codes.view(torch.float8_e4m3fn), rows.scales]
        return swg.permute(st["x"], r)
    if op == "permute_backward":
        return swg.permute_backward(st["z"], r)
    if op == "unpermute":
        return swg.unpermute(st["z"], r, residual=st["residual"])
    return swg.unpermute_backward(st["dy"], st["z"], r)


def _rows_of(z, position):
    """z's rows in 32 bits at [T, k], zero where a choice has none."""
    live = (position >= 0)[:, :, None]
    rows = z[position.clamp_min(0).long()].float()
    return torch.where(live, rows, torch.zeros_like(rows)), live


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "norm":
        s = state["x"].float()
        if state["residual"] is not None:
            s = s + state["residual"].float()
        y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + case["eps"]) * state["weight"].float()
        if case["out"] == "e4m3":
            codes, scales = _codes(y)
            y = [codes.view(torch.float8_e4m3fn), scales]
        else:
            y = [y.to(_DT[case["dtype"]])]
        return y + [s.to(_DT[case["dtype"]])] if state["residual"] is not None else y
    if op == "norm_backward":
        s, dy = state["x"].float(), state["dy"].float()
        r = torch.rsqrt((s * s).mean(1, keepdim=True) + case["eps"])
        g = dy * state["weight"].float()
        dx = r * (g - s * (r * r * (g * s).mean(1, keepdim=True)))
        if state["ds"] is not None:
            dx = dx + state["ds"].float()
        dw = (dy * (s * r)).sum(0)
        return [dx.to(_DT[case["dtype"]]), dw.to(_DT[case["weight"]])]
    if op == "up_fp8":
        x = state["codes"].view(torch.float8_e4m3fn).float() * state["scales"][:, None]
        g = torch.matmul(x, (state["w_gate"].view(torch.float8_e4m3fn).float()
                             * state["s_gate"][:, None]).t())
        u = torch.matmul(x, (state["w_up"].view(torch.float8_e4m3fn).float()
                             * state["s_up"][:, None]).t())
        return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
    position, weights = state["position"], state["weights"]
    if op == "permute":
        order = state["order"]
        token = order.clamp_min(0).long() // case["k"]
        live = (order >= 0)[:, None]
        rows = state["x"][token]
        rows = torch.where(live, rows, torch.zeros_like(rows))
        if case["dtype"] != "e4m3":
            return rows
        scales = state["scales"][token]
        return [rows.view(torch.float8_e4m3fn),
                torch.where(live[:, 0], scales, torch.zeros_like(scales))]
    if op == "permute_backward":
        return _rows_of(state["z"], position)[0].sum(1).to(_DT[case["dtype"]])
    if op == "unpermute":
        rows, _ = _rows_of(state["z"], position)
        y = (weights[:, :, None] * rows).sum(1)
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return y.to(_DT[case["dtype"]])
    rows, live = _rows_of(state["z"], position)
    dy = state["dy"].float()
    dweights = (rows * dy[:, None, :]).sum(2)
    order = state["order"]
    pair = order.clamp_min(0).long()
    dz = weights.reshape(-1)[pair][:, None] * dy[pair // case["k"]]
    dz = torch.where((order >= 0)[:, None], dz, torch.zeros_like(dz))
    return [dz.to(_DT[case["dtype"]]), dweights]


# ---- work and the exact values -----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        M, d, e = case["M"], case["d"], _SIZE[case["dtype"]]
        o = d + 4 if case["out"] == "e4m3" else d * e
        return {"bytes": M * (d * e * (3 if case["residual"] else 1) + o)
                + d * _SIZE[case["weight"]], "flops": 5 * M * d}
    if op == "norm_backward":
        M, d, e = case["M"], case["d"], _SIZE[case["dtype"]]
        return {"bytes": M * d * e * (4 if case["ds"] else 3) + 2 * d * _SIZE[case["weight"]],
                "flops": 10 * M * d}
    if op == "up_fp8":
        M, d, f = case["M"], case["d"], case["d_ff"]
        return {"bytes": 2 * d * f + 8 * f + M * (d + 4) + 2 * M * f, "flops": 4 * M * d * f}
    T, k, d, e = case["T"], case["k"], case["d"], _SIZE[case["dtype"]]
    live = T * k * (1.0 - case["padded"])
    if op == "permute":
        extra = 4 * T * (1 + k) if case["dtype"] == "e4m3" else 0
        return {"bytes": T * d * e * (1 + k) + 4 * T * k + extra, "flops": 0}
    if op == "permute_backward":
        return {"bytes": int(live * d * e + T * d * e + 4 * T * k), "flops": int(live * d)}
    if op == "unpermute":
        return {"bytes": int(live * d * e + T * d * e * (2 if case["residual"] else 1)
                             + 8 * T * k), "flops": int(2 * live * d)}
    return {"bytes": int(T * d * e + live * d * e + T * k * d * e + 12 * T * k),
            "flops": int(3 * live * d)}


def exact(case, seed):
    """The definitions in 64 bits: rows, columns and choices a block or one at a time."""
    st = _inputs(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "norm":
        s = st["x"].to(D)
        if st["residual"] is not None:
            s += st["residual"].to(D)
        y = s / ((s ** 2).sum(1, keepdim=True) / case["d"] + case["eps"]).sqrt()
        y *= st["weight"].to(D)
        if case["out"] == "e4m3":
            scale = y.abs().amax(1) / _E4M3_MAX
            y = [y / scale.clamp_min(1e-300)[:, None], scale]
        else:
            y = [y]
        return y + [s] if st["residual"] is not None else y
    if op == "norm_backward":
        d = case["d"]
        w = st["weight"].to(D)
        dx = torch.empty(case["M"], d, dtype=D, device=w.device)
        dw = torch.zeros(d, dtype=D, device=w.device)
        for i in range(0, case["M"], 4096):
            s, dy = st["x"][i:i + 4096].to(D), st["dy"][i:i + 4096].to(D)
            n = ((s ** 2).sum(1, keepdim=True) / d + case["eps"]).sqrt()
            hat = s / n                                   # y = hat * w
            dw += (dy * hat).sum(0)
            a = dy * w
            dx[i:i + 4096] = (a - hat * (a * hat).sum(1, keepdim=True) / d) / n
            if st["ds"] is not None:
                dx[i:i + 4096] += st["ds"][i:i + 4096].to(D)
        return [dx, dw]
    if op == "up_fp8":
        x = st["codes"].view(torch.float8_e4m3fn).to(D) * st["scales"].to(D)[:, None]
        h = torch.empty(case["M"], case["d_ff"], dtype=D, device=x.device)
        for c in range(0, case["d_ff"], 2048):
            g, u = (x @ (st[n][c:c + 2048].view(torch.float8_e4m3fn).to(D)
                         * st[m][c:c + 2048].to(D)[:, None]).t()
                    for n, m in (("w_gate", "s_gate"), ("w_up", "s_up")))
            h[:, c:c + 2048] = g * torch.sigmoid(g) * u
        return h
    # The places of the pairs, found anew: expert by expert.
    ids = st["ids"].reshape(-1)
    k, n, dev = case["k"], ids.numel(), ids.device
    pairs = torch.cat([torch.nonzero(ids == e)[:, 0] for e in range(case["E"])])
    rows = torch.arange(pairs.numel(), device=dev)
    if op == "permute":
        out = torch.zeros(n, case["d"], dtype=D, device=dev)
        if case["dtype"] == "e4m3":
            out[rows] = st["x"].view(torch.float8_e4m3fn).to(D)[pairs // k]
            scales = torch.zeros(n, dtype=D, device=dev)
            scales[rows] = st["scales"].to(D)[pairs // k]
            return [out, scales]
        out[rows] = st["x"][pairs // k].to(D)
        return out
    z = st["z"][rows]
    w = torch.ones(n, dtype=D, device=dev) if op == "permute_backward" \
        else st["weights"].to(D).reshape(-1)
    if op in ("permute_backward", "unpermute"):
        y = torch.zeros(case["T"], case["d"], dtype=D, device=dev)
        if st.get("residual") is not None:
            y += st["residual"].to(D)
        for i in range(0, pairs.numel(), 16384):
            p = pairs[i:i + 16384]
            y.index_add_(0, p // k, z[i:i + 16384].to(D) * w[p, None])
        return y
    dz = torch.zeros(n, case["d"], dtype=D, device=dev)
    dweights = torch.zeros(n, dtype=D, device=dev)
    for i in range(0, pairs.numel(), 16384):
        p = pairs[i:i + 16384]
        dy = st["dy"][p // k].to(D)
        dz[i:i + 16384][:p.numel()] = w[p, None] * dy
        dweights[p] = (z[i:i + 16384].to(D) * dy).sum(1)
    return [dz, dweights.reshape(st["ids"].shape)]
