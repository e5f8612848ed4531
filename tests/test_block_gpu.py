"""The norm, its 8-bit rows and the sorted rows as they are used together."""
import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64
BF = torch.bfloat16


def randn(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("path", ["auto", "tc"])
@pytest.mark.parametrize("M,d,d_ff", [(1, 64, 72), (7, 4096, 4096), (16, 896, 4864), (33, 1024, 520), (130, 512, 256),
                                      (600, 2048, 1032)])
def test_quantized_rows_give_the_same_bits(cuda_lib, M, d, d_ff, path):
    x = randn(1, M, d)
    w = swg.quantize_weights_fp8(randn(2, d, d_ff, scale=d ** -0.5), randn(3, d, d_ff, scale=d ** -0.5))
    ws = torch.zeros(swg.fp8_workspace_bytes(M, d, d_ff, path), device=DEV, dtype=torch.uint8)
    h = swg.swiglu_up_fp8(x, w, path=path, workspace=ws)
    at = (M * d + 255) // 256 * 256   # where the call leaves x's codes and scales
    rows = swg.Fp8Rows(ws[:M * d].view(M, d).clone(), ws[at:at + 4 * M].view(torch.float32).clone())
    assert torch.equal(swg.swiglu_up_fp8(rows, w, path=path), h)
    assert torch.equal(swg.swiglu_up_fp8(rows, w, path=path, workspace=ws), h)
    swg.check_device_status()


@pytest.mark.parametrize("M,d,d_ff", [(7, 4096, 4096), (16, 896, 4864), (600, 2048, 1032)])
def test_quantized_rows_where_the_up_projection_leaves_them(cuda_lib, M, d, d_ff):
    """Codes and scales in the workspace go on with its part behind them; the whole of it is refused."""
    w = swg.quantize_weights_fp8(randn(2, d, d_ff, scale=d ** -0.5), randn(3, d, d_ff, scale=d ** -0.5))
    ws = torch.zeros(swg.fp8_workspace_bytes(M, d, d_ff), device=DEV, dtype=torch.uint8)
    h = swg.swiglu_up_fp8(randn(1, M, d), w, workspace=ws)
    at = (M * d + 255) // 256 * 256
    end = at + (4 * M + 255) // 256 * 256
    rows = swg.Fp8Rows(ws[:M * d].view(M, d), ws[at:at + 4 * M].view(torch.float32))
    with pytest.raises(swg.SwiGLUError):
        swg.swiglu_up_fp8(rows, w, workspace=ws)
    for _ in range(2):
        assert torch.equal(swg.swiglu_up_fp8(rows, w, workspace=ws[end:]), h)
    swg.check_device_status()


def test_quantized_rows_refused(cuda_lib):
    w = swg.quantize_weights_fp8(randn(2, 64, 72), randn(3, 64, 72))
    c, s = torch.zeros(4, 64, device=DEV, dtype=torch.uint8), torch.ones(4, device=DEV)
    for rows in (swg.Fp8Rows(c[:, :32].contiguous(), s), swg.Fp8Rows(c, s[:3]), swg.Fp8Rows(c, s.double()),
                 swg.Fp8Rows(c.float(), s), swg.Fp8Rows(c.cpu(), s), swg.Fp8Rows(c, s.cpu())):
        with pytest.raises(ValueError):
            swg.swiglu_up_fp8(rows, w)
    with pytest.raises(swg.SwiGLUError):
        swg.swiglu_up_fp8(swg.Fp8Rows(c, s), w, path="simt")
    assert swg.swiglu_up_fp8(swg.Fp8Rows(c[:0], s[:0]), w).shape == (0, 72)


@pytest.mark.parametrize("M", [1, 16, 300])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("with_residual", [False, True])
def test_block(cuda_lib, M, fp8, with_residual):
    """The block's steps are the operators it is made of, and its value is its definition's."""
    d, d_ff = 896, 4864
    x, r = randn(1, M, d), randn(2, M, d) if with_residual else None
    nw = (1 + randn(3, d, scale=0.3).float()).to(BF)
    wg, wu = randn(4, d, d_ff, scale=d ** -0.5), randn(5, d, d_ff, scale=d ** -0.5)
    wd = randn(6, d_ff, d, scale=d_ff ** -0.5)
    if fp8:
        up, down = swg.quantize_weights_fp8(wg, wu), swg.quantize_weight_fp8(wd)
    else:
        up, down = (wg, wu), wd
    y = swg.swiglu_block(x, nw, up, down, residual=r)
    s = x.to(D) if r is None else x.to(D) + r.to(D)
    n = s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * nw.to(D)
    g, u = n @ wg.to(D), n @ wu.to(D)
    ref = s + (g * torch.sigmoid(g) * u) @ wd.to(D)
    # bf16: n, h, s and y are each rounded by at most 2^-8 of themselves, which through sums of
    # random signs is of the order of 2^-8 of the norm of y - s; e4m3: n, h and the weights by 2^-4
    rel = 4 * 2.0 ** -8 + (6 * 2.0 ** -4 if fp8 else 2.0 ** -8)
    assert (y.to(D) - ref).norm() <= rel * (ref - s).norm() + 2 * 2.0 ** -8 * s.norm()
    if r is not None and not fp8:   # layout [N, K]: the same value
        y2 = swg.swiglu_block(x, nw, (wg.t().contiguous(), wu.t().contiguous()), wd.t().contiguous(),
                              residual=r, layout="nk")
        assert (y2.to(D) - ref).norm() <= rel * (ref - s).norm() + 2 * 2.0 ** -8 * s.norm()
    st = torch.cuda.Stream()
    swg.swiglu_block(x, nw, up, down, residual=r)
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = swg.swiglu_block(x, nw, up, down, residual=r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, y)
    swg.check_device_status()


@pytest.mark.parametrize("M", [1, 16, 300])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("with_residual", [False, True])
def test_block_is_its_steps(cuda_lib, M, fp8, with_residual):
    """The block gives the bits of norm, up and down called in turn, and each product is within
    rounding of the 64-bit sums over the very operands that it multiplies, element by element.

    A sum of K products, however ordered, and its scales are off by less than (K + 4) 2^-23 of the sum of
    the products' sizes (twice the rounding of f32, for sums inside the tensor core); h = silu(g) u has
    |silu'| <= 1.1, and its exponential and quotient less than 2^-18 of h; h and y are rounded to bf16.
    """
    d, d_ff = 896, 4864
    x, r = randn(1, M, d), randn(2, M, d) if with_residual else None
    nw = (1 + randn(3, d, scale=0.3).float()).to(BF)
    wg, wu = randn(4, d, d_ff, scale=d ** -0.5), randn(5, d, d_ff, scale=d ** -0.5)
    wd = randn(6, d_ff, d, scale=d_ff ** -0.5)

    def rows64(codes, scales):
        return codes.view(torch.float8_e4m3fn).to(D) * scales.to(D)[:, None]
    if fp8:
        up, down = swg.quantize_weights_fp8(wg, wu), swg.quantize_weight_fp8(wd)
        wg, wu = rows64(up.w8_gate, up.s_gate).t(), rows64(up.w8_up, up.s_up).t()
        wd = rows64(down.w8, down.s).t()
        n = swg.rms_norm_fp8(x, nw, residual=r)
    else:
        up, down = (wg, wu), wd
        n = swg.rms_norm(x, nw, residual=r)
    n, s = (n, x) if r is None else n
    h = swg.swiglu_up_fp8(n, up) if fp8 else swg.swiglu_up(n, wg, wu)
    y = (swg.swiglu_down_fp8 if fp8 else swg.swiglu_down)(h, down, residual=s)
    assert torch.equal(swg.swiglu_block(x, nw, up, down, residual=r), y)

    n64, wg, wu, wd = (rows64(*n) if fp8 else n.to(D)), wg.to(D), wu.to(D), wd.to(D)
    g, u = n64 @ wg, n64 @ wu
    eg, eu = ((d + 4) * 2.0 ** -23 * (n64.abs() @ w.abs()) for w in (wg, wu))
    a = g * torch.sigmoid(g)
    tol = (2.0 ** -8 + 2.0 ** -18) * (a * u).abs() + 1.1 * eg * (u.abs() + eu) + a.abs() * eu
    assert bool(((h.to(D) - a * u).abs() <= tol + 2.0 ** -133).all())
    h64 = h.to(D)
    if fp8:   # the codes and scales of h that the call leaves at the start of its workspace
        need = cuda_lib.swiglu_down_fp8_workspace_bytes(M, d_ff, d, 0)
        ws = torch.zeros(need, device=DEV, dtype=torch.uint8)
        assert torch.equal(swg.swiglu_down_fp8(h, down, residual=s, workspace=ws), y)
        at = (M * d_ff + 255) // 256 * 256
        codes, scales = ws[:M * d_ff].view(M, d_ff), ws[at:at + 4 * M].view(torch.float32)
        # (448 / amax, amax / 448 and the product with h are rounded to f32)
        amax = h64.abs().amax(1)
        assert bool(((scales.to(D) * 448 - amax).abs() <= 2.0 ** -24 * amax).all())
        v = h64 * (448 / amax)[:, None]
        err = (codes.view(torch.float8_e4m3fn).to(D) - v).abs()
        assert bool((err <= v.abs() * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10).all())
        h64 = rows64(codes, scales)
    y64 = s.to(D) + h64 @ wd
    tol = 2.0 ** -8 * y64.abs() + (d_ff + 4) * 2.0 ** -23 * (h64.abs() @ wd.abs() + s.to(D).abs())
    assert bool(((y.to(D) - y64).abs() <= tol * (1 + 2.0 ** -7)).all())
    swg.check_device_status()


def test_training_step_of_routed_experts(cuda_lib):
    """norm -> permute -> experts of one matrix each -> unpermute, and back: the gradients of
    input, norm weight and routing weights against autograd in 64 bits."""
    T, E, k, d = 200, 8, 2, 128
    x, r, dy = (randn(i, T, d, dtype=torch.float32) for i in (1, 2, 3))
    nw = 1 + randn(4, d, scale=0.3, dtype=torch.float32)
    w = randn(5, E, d, d, scale=d ** -0.5, dtype=torch.float32)
    ids = torch.argsort(torch.rand(T, E, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV))
    ids = ids[:, :k].int().contiguous()
    ids[::7] = -1
    rt = swg.dispatch(ids, E, torch.softmax(randn(7, T, k, dtype=torch.float32), 1))
    off = rt.offsets.tolist()

    n, s = swg.rms_norm(x, nw, residual=r, eps=1e-5)
    rows = swg.permute(n, rt)
    z = torch.zeros_like(rows, dtype=D)
    for e in range(E):
        z[off[e]:off[e + 1]] = rows[off[e]:off[e + 1]].to(D) @ w[e].to(D)
    y = swg.unpermute(z.float(), rt, residual=s)
    dz, dweights = swg.unpermute_backward(dy, z.float(), rt)
    drows = torch.zeros_like(rows, dtype=D)
    for e in range(E):
        drows[off[e]:off[e + 1]] = dz[off[e]:off[e + 1]].to(D) @ w[e].to(D).t()
    dn = swg.permute_backward(drows.float(), rt)
    dx, dnw = swg.rms_norm_backward(dn, s, nw, ds=dy, eps=1e-5)

    x6, nw6, wt6 = (t.to(D).requires_grad_() for t in (x, nw, rt.weights))
    s6 = x6 + r.to(D)
    n6 = s6 / (s6.square().mean(1, keepdim=True) + 1e-5).sqrt() * nw6
    y6 = s6
    for j in range(k):
        live = ids[:, j] >= 0
        out = torch.einsum("td,tdf->tf", n6, w.to(D)[ids[:, j].clamp_min(0).long()])
        y6 = y6 + torch.where(live[:, None], wt6[:, j:j + 1] * out, torch.zeros_like(out))
    y6.backward(dy.to(D))
    # a chain of five f32 steps, each off by less than 2^-16 of its terms (2^-19 forward)
    for got, want in ((y, y6), (dx, x6.grad), (dnw, nw6.grad), (dweights, wt6.grad)):
        assert (got.to(D) - want).norm() <= 5 * 2.0 ** -16 * want.norm()


def test_decode_step_of_routed_experts_captured(cuda_lib):
    """norm -> router -> route -> experts on the sorted rows, replayed with other rows."""
    T, E, k, d, f = 3, 16, 4, 256, 192
    x, nw = randn(1, T, d), randn(2, d, dtype=torch.float32).abs() + 0.5
    wr, wg, wu = randn(3, d, E, scale=d ** -0.5), randn(4, E, d, f, scale=d ** -0.5), \
        randn(5, E, d, f, scale=d ** -0.5)
    wd = randn(6, E, f, d, scale=f ** -0.5)

    def step():
        n = swg.rms_norm(x, nw)
        rt = swg.route(swg.linear(n, wr, out_dtype=torch.float32), k)
        # rows sorted by hand: each is a token of its own with one choice
        rows = swg.permute(n, rt)
        mine = swg.experts_up(n, wg, wu, rt)
        e = torch.repeat_interleave(torch.arange(E, device=DEV, dtype=torch.int32),
                                    (rt.offsets[1:] - rt.offsets[:-1]).long(), output_size=T * k)
        own = swg.dispatch(e.view(-1, 1), E, torch.ones(T * k, 1, device=DEV))
        h = swg.experts_up(rows, wg, wu, own)
        z = swg.experts_down(h, wd, own)
        return mine, h, swg.unpermute(z, rt, residual=x), swg.experts_down(mine, wd, rt, residual=x)
    step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        mine, h, y, want = step()
    for seed in (7, 8):
        x.copy_(randn(seed, T, d))
        graph.replay()
        torch.cuda.synchronize()
        # (the two calls may cut the products along K in other places)
        assert (mine.to(D) - h.to(D)).norm() <= 2 * 2.0 ** -8 * mine.to(D).norm()
        # z is rounded to bf16 between the steps here: 2^-8 of each weighted term
        assert (y.to(D) - want.to(D)).norm() <= 2 * 2.0 ** -8 * want.to(D).norm()
