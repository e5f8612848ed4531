"""Run one shape through swiglu_up (swiglu_down, swiglu_moe) repeatedly, for
timing and profiling.

    python -m swiglu_mlp_projection_gb300 --M 16 --d 4096 --d_ff 14336 [--dtype bf16]
        [--op up|down|moe] [--path auto|simt|skinny|tc] [--iters 20] [--warmup 3]
        [--copies 1] [--fp8] [--experts 8] [--top_k 2]

--op down times y = h . W_down + residual (bf16; h [M, d_ff], W_down
[d_ff, d], residual [M, d]).  --fp8 quantizes the weights to e4m3 once
(outside the timed calls) and times swiglu_up_fp8 / swiglu_down_fp8 instead
(bf16 activations and outputs).

--op moe times the mixture-of-experts MLP (bf16; M tokens through top_k of the
experts, each of d, d_ff): router logits, routing, the experts' up and down
projections and the residual, with the time of each step.

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
    ap.add_argument("--op", default="up", choices=["up", "down", "moe"])
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top_k", type=int, default=2)
    a = ap.parse_args()
    dev = torch.device("cuda", 0)
    if a.op == "down":
        return run_down(a, dev)
    if a.op == "moe":
        return run_moe(a, dev)
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

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(torch.bfloat16)
    E, k = a.experts, a.top_k
    x = normal(a.M, a.d)
    wr = normal(a.d, E, scale=a.d ** -0.5)
    ws = [(normal(E, a.d, a.d_ff, scale=a.d ** -0.5), normal(E, a.d, a.d_ff, scale=a.d ** -0.5),
           normal(E, a.d_ff, a.d, scale=a.d_ff ** -0.5)) for _ in range(a.copies)]
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
