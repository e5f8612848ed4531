"""Run one shape through swiglu_up (swiglu_down, swiglu_moe) repeatedly, for
timing and profiling.

    python -m swiglu_mlp_projection_gb300 --M 16 --d 4096 --d_ff 14336 [--dtype bf16]
        [--op up|down|moe|block|rows] [--path auto|simt|skinny|tc] [--iters 20] [--warmup 3]
        [--copies 1] [--fp8] [--experts 8] [--top_k 2]

--op down times y = h . W_down + residual (bf16; h [M, d_ff], W_down
[d_ff, d], residual [M, d]).  --fp8 quantizes the weights to e4m3 once
(outside the timed calls) and times swiglu_up_fp8 / swiglu_down_fp8 instead
(bf16 activations and outputs).

--op moe times the mixture-of-experts MLP (bf16; M tokens through top_k of the
experts, each of d, d_ff): router logits, routing, the experts' up and down
projections and the residual, with the time of each step.

--op block times the pre-norm MLP block (bf16, or --fp8) and each of its steps:
the norm with the residual's addition, the up and the down projection.  --op
rows times a training step's row operators on M tokens through top_k of the
experts (bf16): the norm and its gradient, rows sorted by expert and back, and
their gradients.

Inputs are the seeded synthetic operands of swiglu_mlp_projection_gb300.inputs.
Prints the median time per call and the achieved GB/s and TFLOP/s.
"""
import argparse
import json
import statistics


def main():
    import torch
    import swiglu_mlp_projection_gb300 as swg
    from swiglu_mlp_projection_gb300 import inputs, workload

    ap = argparse.ArgumentParser()
    ap.add_argument("--M", type=int, default=16)
    ap.add_argument("--d", type=int, default=4096)
    ap.add_argument("--d_ff", type=int, default=14336)
    ap.add_argument("--dtype", default="bf16", choices=["bf16", "f32"])
    ap.add_argument("--path", default="auto", choices=sorted(swg.PATHS))
    ap.add_argument("--iters", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--copies", type=int, default=1, help="weight copies rotated per call")
    ap.add_argument("--fp8", action="store_true", help="e4m3 weights (swiglu_up_fp8)")
    ap.add_argument("--op", default="up", choices=["up", "down", "moe", "block", "rows"])
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top_k", type=int, default=2)
    a = ap.parse_args()
    dev = torch.device("cuda", 0)
    if a.op == "down":
        return run_down(a, dev)
    if a.op == "moe":
        return run_moe(a, dev)
    if a.op == "block":
        return run_block(a, dev)
    if a.op == "rows":
        return run_rows(a, dev)
    x, wg, wu = inputs.make_inputs(a.M, a.d, a.d_ff, a.dtype, seed=0)
    x = x.to(dev)
    ws = [(wg.to(dev), wu.to(dev)) for _ in range(a.copies)]
    h = torch.empty(a.M, a.d_ff, dtype=x.dtype, device=dev)
    if a.fp8:
        if a.dtype != "bf16":
            raise SystemExit("--fp8 takes bf16 x and weights")
        qs = [swg.quantize_weights_fp8(g, u) for g, u in ws]
        call = lambda i: swg.swiglu_up_fp8(x, qs[i % a.copies], out=h, path=a.path)
    else:
        call = lambda i: swg.swiglu_up(x, *ws[i % a.copies], out=h, path=a.path)
    ms = time_calls(call, a.warmup, a.iters)
    swg.check_device_status()
    by = (workload.fp8_bytes(a.M, a.d, a.d_ff) if a.fp8
          else workload.algorithmic_bytes(a.M, a.d, a.d_ff, a.dtype))
    fl = workload.flops(a.M, a.d, a.d_ff)
    print(json.dumps({"M": a.M, "d": a.d, "d_ff": a.d_ff, "dtype": "e4m3" if a.fp8 else a.dtype,
                      "path": swg.plan(a.M, a.d, a.d_ff, a.dtype, a.path)["path"],
                      "us": round(ms * 1e3, 2), "GB/s": round(by / ms / 1e6, 1),
                      "TFLOP/s": round(fl / ms / 1e9, 2)}))


def run_down(a, dev):
    import torch
    import swiglu_mlp_projection_gb300 as swg
    from swiglu_mlp_projection_gb300 import inputs, workload
    if a.dtype != "bf16":
        raise SystemExit("the down projection takes bf16")
    h = inputs.make_inputs(a.M, a.d_ff, 8, "bf16", seed=0, x_only=True)[0].to(dev)
    r = inputs.make_inputs(a.M, a.d, 8, "bf16", seed=2, x_only=True)[0].to(dev)
    wds = [inputs.make_inputs(1, a.d_ff, a.d, "bf16", seed=1 + i)[1].to(dev)
           for i in range(a.copies)]
    y = torch.empty(a.M, a.d, dtype=torch.bfloat16, device=dev)
    if a.fp8:
        qs = [swg.quantize_weight_fp8(w) for w in wds]
        call = lambda i: swg.swiglu_down_fp8(h, qs[i % a.copies], residual=r, out=y, path=a.path)
    else:
        call = lambda i: swg.swiglu_down(h, wds[i % a.copies], residual=r, out=y, path=a.path)
    ms = time_calls(call, a.warmup, a.iters)
    swg.check_device_status()
    by = (workload.fp8_down_bytes(a.M, a.d_ff, a.d) if a.fp8
          else workload.down_bytes(a.M, a.d_ff, a.d, "bf16"))
    fl = workload.down_flops(a.M, a.d_ff, a.d)
    print(json.dumps({"op": "down", "M": a.M, "d": a.d, "d_ff": a.d_ff,
                      "dtype": "e4m3" if a.fp8 else "bf16",
                      "path": swg.down_plan(a.M, a.d_ff, a.d, "bf16", a.path)["path"],
                      "us": round(ms * 1e3, 2), "GB/s": round(by / ms / 1e6, 1),
                      "TFLOP/s": round(fl / ms / 1e9, 2)}))


def run_moe(a, dev):
    import torch
    import swiglu_mlp_projection_gb300 as swg
    if a.dtype != "bf16" or a.fp8:
        raise SystemExit("the mixture of experts takes bf16")
    gen = torch.Generator(device=dev).manual_seed(0)
    E, k = a.experts, a.top_k
    x = normal(gen, a.M, a.d)
    wr = normal(gen, a.d, E, scale=a.d ** -0.5)
    ws = [(normal(gen, E, a.d, a.d_ff, scale=a.d ** -0.5),
           normal(gen, E, a.d, a.d_ff, scale=a.d ** -0.5),
           normal(gen, E, a.d_ff, a.d, scale=a.d_ff ** -0.5)) for _ in range(a.copies)]
    wg, wu, wd = ws[0]
    logits = swg.linear(x, wr, out_dtype=torch.float32)
    r = swg.route(logits, k)
    h = swg.experts_up(x, wg, wu, r)
    steps = {
        "router": lambda i: swg.linear(x, wr, out_dtype=torch.float32),
        "route": lambda i: swg.route(logits, k),
        "up": lambda i: swg.experts_up(x, *ws[i % a.copies][:2], r, out=h),
        "down": lambda i: swg.experts_down(h, ws[i % a.copies][2], r, residual=x),
        "all": lambda i: swg.swiglu_moe(x, wr, *ws[i % a.copies], k, residual=x),
    }
    us = {n: round(time_calls(f, a.warmup, a.iters) * 1e3, 2) for n, f in steps.items()}
    swg.check_device_status()
    reached = int((r.offsets[1:] > r.offsets[:-1]).sum())
    by = 6 * reached * a.d * a.d_ff + 2 * a.d * E + 2 * a.M * a.d * 3
    fl = 6 * a.M * k * a.d * a.d_ff
    print(json.dumps({"op": "moe", "M": a.M, "d": a.d, "d_ff": a.d_ff, "experts": E, "top_k": k,
                      "experts_reached": reached, "us": us,
                      "GB/s": round(by / us["all"] / 1e3, 1),
                      "TFLOP/s": round(fl / us["all"] / 1e6, 2)}))


def normal(gen, *shape, scale=1.0):
    import torch
    return (torch.randn(*shape, generator=gen, device=gen.device) * scale).to(torch.bfloat16)


def run_block(a, dev):
    import torch
    import swiglu_mlp_projection_gb300 as swg
    if a.dtype != "bf16":
        raise SystemExit("the MLP block takes bf16")
    gen = torch.Generator(device=dev).manual_seed(0)
    x, r = normal(gen, a.M, a.d), normal(gen, a.M, a.d)
    nw = normal(gen, a.d, scale=0.1) + 1
    sets = []
    for _ in range(a.copies):
        wg, wu = (normal(gen, a.d, a.d_ff, scale=a.d ** -0.5) for _ in range(2))
        wd = normal(gen, a.d_ff, a.d, scale=a.d_ff ** -0.5)
        sets.append((swg.quantize_weights_fp8(wg, wu), swg.quantize_weight_fp8(wd)) if a.fp8
                    else ((wg, wu), wd))
    if a.fp8:
        norm, up = swg.rms_norm_fp8, swg.swiglu_up_fp8
        down = swg.swiglu_down_fp8
    else:
        norm, down = swg.rms_norm, swg.swiglu_down
        up = lambda n, w: swg.swiglu_up(n, *w)
    n, s = norm(x, nw, residual=r)
    h = up(n, sets[0][0])
    steps = {
        "norm": lambda i: norm(x, nw, residual=r),
        "up": lambda i: up(n, sets[i % a.copies][0]),
        "down": lambda i: down(h, sets[i % a.copies][1], residual=s),
        "all": lambda i: swg.swiglu_block(x, nw, *sets[i % a.copies], residual=r),
    }
    us = {k: round(time_calls(f, a.warmup, a.iters) * 1e3, 2) for k, f in steps.items()}
    swg.check_device_status()
    by = 3 * a.d * a.d_ff * (1 if a.fp8 else 2) + 3 * 2 * a.M * a.d
    fl = 6 * a.M * a.d * a.d_ff
    print(json.dumps({"op": "block", "M": a.M, "d": a.d, "d_ff": a.d_ff,
                      "dtype": "e4m3" if a.fp8 else "bf16", "us": us,
                      "GB/s": round(by / us["all"] / 1e3, 1),
                      "TFLOP/s": round(fl / us["all"] / 1e6, 2)}))


def run_rows(a, dev):
    import torch
    import swiglu_mlp_projection_gb300 as swg
    if a.dtype != "bf16" or a.fp8:
        raise SystemExit("the row operators are timed in bf16")
    gen = torch.Generator(device=dev).manual_seed(0)
    x, r, dy = (normal(gen, a.M, a.d) for _ in range(3))
    nw = normal(gen, a.d, scale=0.1) + 1
    rt = swg.route(torch.randn(a.M, a.experts, generator=gen, device=dev), a.top_k)
    z = normal(gen, a.M * a.top_k, a.d)
    row = 2 * a.M * a.d            # bytes of the tokens' rows, and of the sorted ones
    rows = row * a.top_k
    steps = {
        "norm": (lambda i: swg.rms_norm(x, nw, residual=r), 4 * row),
        "norm_fp8": (lambda i: swg.rms_norm_fp8(x, nw, residual=r), 3 * row + row // 2),
        "norm_backward": (lambda i: swg.rms_norm_backward(dy, x, nw, ds=r), 4 * row),
        "permute": (lambda i: swg.permute(x, rt), row + rows),
        "permute_backward": (lambda i: swg.permute_backward(z, rt), row + rows),
        "unpermute": (lambda i: swg.unpermute(z, rt, residual=x), 2 * row + rows),
        "unpermute_backward": (lambda i: swg.unpermute_backward(dy, z, rt), row + 2 * rows),
    }
    us = {k: round(time_calls(f, a.warmup, a.iters) * 1e3, 2) for k, (f, _) in steps.items()}
    print(json.dumps({"op": "rows", "M": a.M, "d": a.d, "experts": a.experts, "top_k": a.top_k,
                      "us": us, "GB/s": {k: round(b / us[k] / 1e3, 1)
                                         for k, (_, b) in steps.items()}}))


def time_calls(call, warmup, iters):
    """Median milliseconds per call, each call timed with CUDA events."""
    import torch
    for i in range(warmup):
        call(i)
    torch.cuda.synchronize()
    times = []
    for i in range(iters):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        call(i)
        e1.record()
        e1.synchronize()
        times.append(e0.elapsed_time(e1))
    return statistics.median(times)


if __name__ == "__main__":
    main()
