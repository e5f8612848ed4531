"""The RMS norm, its 8-bit rows and its gradient against their definitions in 64 bits.

Tolerances, with u = 2^-24.  A row's sum of squares adds at most 32 values in a
thread, then 32 lanes, then 32 warps: 42 roundings, and 2 u of each square from
the rounding of s, so mean(s^2) + eps is off by at most 46 u, the root of it by
23 u, and 3 u come from dividing and taking the root; t = s w, the product with
the root and s itself add 3 u more: y is off by less than 32 u = 2^-19 of
itself, and by half a step of its type (2^-8 in bf16).  e4m3 codes: half a step,
2^-4 of the value or 2^-10 below the normal range, and 2^-18 for the two f32
values whose quotient it rounds.  Gradient: r is off by 28 u (4 of them
its approximation), r^3 by 84 u, mean(g s) by
48 u of mean |g s|, products by 8 u: less than 2^-16 of the terms' sizes.
dweight adds each row's term (32 u) over the rows of a CTA (at most M / 64, or
64), 32 groups and 32 lanes.
"""
import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -126}   # (a rounding below the normal range)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(seed, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * scale).to(dtype)


def inputs(M, d, dtype, wdtype, seed=0):
    x = randn(seed, M, d, dtype=dtype) * torch.exp(randn(seed + 1, M, 1, dtype=F32)).to(dtype)
    w = (1 + 0.5 * torch.randn(d, generator=gen(seed + 2), device=DEV)).to(wdtype)
    return x, randn(seed + 3, M, d, dtype=dtype), w


def ref_norm(x, residual, w, eps):
    s = x.to(D) if residual is None else x.to(D) + residual.to(D)
    return s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w.to(D), s


def check_norm(y, s, x, residual, w, eps):
    ref, s64 = ref_norm(x, residual, w, eps)
    err = (y.to(D) - ref).abs()
    assert bool((err <= ref.abs() * (HALF[y.dtype] + 2.0 ** -19) + TINY[y.dtype]).all()), err.max()
    if s is not None:
        assert torch.equal(s, (x.to(F32) + residual.to(F32)).to(x.dtype))


def check_fp8(rows, x, residual, w, eps):
    ref, _ = ref_norm(x, residual, w, eps)
    amax = ref.abs().amax(1)
    assert bool(((rows.scales.to(D) - amax / 448).abs() <= 2.0 ** -19 * amax / 448).all())
    v = ref * torch.where(amax > 0, 448 / amax, torch.zeros_like(amax))[:, None]
    err = (rows.codes.view(torch.float8_e4m3fn).to(D) - v).abs()
    assert bool((err <= v.abs() * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10).all()), err.max()


SIZES = [(1, 1), (1, 8), (1, 4096), (1, 4099), (1, 32768), (1, 32752), (1, 32751), (2, 7), (3, 64), (5, 896),
         (7, 897), (16, 4096), (33, 2047), (150, 8192), (151, 129), (153, 1), (200, 8), (200, 13),
         (300, 130), (333, 896), (400, 1000), (400, 1024), (300, 1031), (260, 2056), (257, 4100), (160, 16384),
         (154, 16391), (155, 32768), (156, 32737), (1000, 509),
         # each number of warps that may share a row, and several rows for each of them
         (170, 1400), (333, 1801), (160, 2048), (157, 3301), (155, 5000), (159, 7001), (154, 9001), (153, 10000),
         (170, 13001), (15001, 40), (15001, 43), (8000, 601), (2100, 4099), (2100, 4096),
         # rows that several CTAs share
         (200, 20000), (160, 20003), (240, 12000), (230, 9003), (90, 24571)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,d", SIZES)
def test_norm(cuda_lib, M, d, dtype, wdtype):
    x, r, w = inputs(M, d, dtype, wdtype)
    check_norm(swg.rms_norm(x, w), None, x, None, w, 1e-6)
    y, s = swg.rms_norm(x, w, residual=r, eps=1e-5)
    check_norm(y, s, x, r, w, 1e-5)


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,d", SIZES)
def test_norm_fp8(cuda_lib, M, d, dtype, wdtype):
    x, r, w = inputs(M, d, dtype, wdtype, 9)
    rows = swg.rms_norm_fp8(x, w)
    check_fp8(rows, x, None, w, 1e-6)
    rows, s = swg.rms_norm_fp8(x, w, residual=r, eps=1e-5)
    check_fp8(rows, x, r, w, 1e-5)
    assert torch.equal(s, (x.to(F32) + r.to(F32)).to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", [(4, 897), (300, 896), (300, 899), (200, 4096), (3, 16384)])
def test_outputs_on_top_of_inputs(cuda_lib, M, d, dtype):
    x, r, w = inputs(M, d, dtype, dtype)
    y, s = swg.rms_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    y2, s2 = swg.rms_norm(a, w, residual=b, out=a, sum_out=b)
    assert y2 is a and s2 is b and torch.equal(a, y) and torch.equal(b, s)
    a, b = x.clone(), r.clone()
    swg.rms_norm(a, w, residual=b, out=b, sum_out=a)
    assert torch.equal(b, y) and torch.equal(a, s)
    rows, s = swg.rms_norm_fp8(x, w, residual=r)
    a = x.clone()
    rows2, s2 = swg.rms_norm_fp8(a, w, residual=r, sum_out=a)
    assert torch.equal(a, s) and torch.equal(rows.codes, rows2.codes)
    dy, ds = randn(20, M, d, dtype=dtype), randn(21, M, d, dtype=dtype)
    dx, dw = swg.rms_norm_backward(dy, x, w, ds=ds)
    for n in range(3):
        t = [dy.clone(), x.clone(), ds.clone()]
        dx2, dw2 = swg.rms_norm_backward(t[0], t[1], w, ds=t[2], out=t[n])
        assert dx2 is t[n] and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("d", [896, 4096, 5000, 4099])
@pytest.mark.parametrize("M", [5, 400])
def test_rows_that_are_not_ordinary(cuda_lib, M, d):
    x, _, w = inputs(M, d, BF, BF)
    x[0] = 0
    x[1, d // 2] = float("inf")
    x[2, 3] = float("nan")
    x[3] = 0
    x[3, 5] = 2.0 ** -126           # t stays below 2^-118
    x[4] *= 2.0 ** -60              # eps dominates
    y = swg.rms_norm(x, w)
    assert not bool(y[0].any())
    assert bool(y[1, d // 2].isnan()) and not bool(y[1, :d // 2].any())
    assert bool(y[2].isnan().all())
    rows = [0, *range(3, M)]
    check_norm(y[rows], None, x[rows], None, w, 1e-6)
    f = swg.rms_norm_fp8(x, w)
    assert f.scales[0] == 0 and not bool(f.codes[0].view(torch.float8_e4m3fn).float().any())
    assert bool(f.scales[1].isnan()) and bool(f.scales[2].isnan())
    assert f.scales[3] == 0 and not bool(f.codes[3].view(torch.float8_e4m3fn).float().any())
    rows = range(4, M)
    check_fp8(swg.Fp8Rows(f.codes[4:], f.scales[4:]), x[4:], None, w, 1e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", [(1, 1), (3, 64), (300, 896), (300, 1031), (2, 4099), (200, 8192), (157, 3301),
                                 (154, 9001), (153, 10000), (170, 13001), (3, 20003), (160, 32751)])
def test_nan_of_the_weight(cuda_lib, M, d, dtype):
    """amax = max |y| is NaN if one y is: the row's scale says so, wherever the NaN stands."""
    x, r, w = inputs(M, d, dtype, F32, 95)
    x[-1] = 0
    for at in {0, d // 2, d - 1}:
        v = w.clone()
        v[at] = float("nan")
        for rows in (swg.rms_norm_fp8(x, v), swg.rms_norm_fp8(x, v, residual=r)[0]):
            assert bool(rows.scales.isnan().all())
            assert bool(rows.codes.view(torch.float8_e4m3fn).float()[:, at].isnan().all())
        y = swg.rms_norm(x, v)
        assert bool(y[:, at].isnan().all()) and int(y.isnan().sum()) == M
    rows = swg.rms_norm_fp8(x, w)
    check_fp8(rows, x, None, w, 1e-6)


def ref_backward(dy, s, w, ds, eps):
    """(dx, dweight, sizes of dx's terms, sizes of dweight's terms)."""
    dy, s, w = dy.to(D), s.to(D), w.to(D)
    r = 1 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    g = dy * w
    dx = r * (g - s * r * r * (g * s).mean(1, keepdim=True))
    size = r * (g.abs() + s.abs() * r * r * (g * s).abs().mean(1, keepdim=True))
    if ds is not None:
        dx = dx + ds.to(D)
        size = size + ds.to(D).abs()
    t = dy * s * r
    return dx, t.sum(0), size, t.abs().sum(0)


def check_backward(dx, dw, dy, s, w, ds, eps):
    rx, rw, size, wsize = ref_backward(dy, s, w, ds, eps)
    err = (dx.to(D) - rx).abs()
    assert bool((err <= rx.abs() * HALF[dx.dtype] + 2.0 ** -16 * size + TINY[dx.dtype]).all()), err.max()
    rows = max(64, dy.shape[0] / 64)
    err = (dw.to(D) - rw).abs()
    tol = rw.abs() * HALF[dw.dtype] + 2.0 ** -24 * (32 + rows + 64) * wsize + TINY[dw.dtype]
    assert bool((err <= tol).all()), (err - tol).max()


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,d", SIZES + [(1300, 24), (5001, 97)])
def test_backward(cuda_lib, M, d, dtype, wdtype):
    x, dy, w = inputs(M, d, dtype, wdtype, 30)
    check_backward(*swg.rms_norm_backward(dy, x, w), dy, x, w, None, 1e-6)
    ds = randn(31, M, d, dtype=dtype, scale=3.0)
    check_backward(*swg.rms_norm_backward(dy, x, w, ds=ds, eps=1e-3), dy, x, w, ds, 1e-3)


@pytest.mark.parametrize("M,d", [(3, 40), (4, 33)])
def test_backward_against_differences(cuda_lib, M, d):
    x, dy, w = inputs(M, d, F32, F32, 40)
    eps = 1e-2
    dx, dw = swg.rms_norm_backward(dy, x, w, eps=eps)
    h = 2.0 ** -14   # (the error of the difference is of the order of h^2 = 4e-9 of its third derivative)

    def loss(s, w):
        return (ref_norm(s, None, w, eps)[0] * dy.to(D)).sum()
    for seed in range(4):
        v = randn(50 + seed, M, d, dtype=D)
        diff = (loss(x.to(D) + h * v, w) - loss(x.to(D) - h * v, w)) / (2 * h)
        size = (dx.to(D).abs() * v.abs()).sum() + (dy.to(D) * w.to(D)).abs().sum()
        assert abs((dx.to(D) * v).sum() - diff) <= 2.0 ** -16 * size
        v = randn(60 + seed, d, dtype=D)
        diff = (loss(x, w.to(D) + h * v) - loss(x, w.to(D) - h * v)) / (2 * h)
        assert abs((dw.to(D) * v).sum() - diff) <= 2.0 ** -16 * (dw.to(D).abs() * v.abs()).sum() \
            + 2.0 ** -16 * dy.to(D).abs().sum()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", [(3, 4096), (200, 896), (200, 1001), (5, 20000)])
@pytest.mark.parametrize("scale,eps", [(2.0 ** 45, 1e-6), (2.0 ** -50, 1e-30), (2.0 ** -20, 1.0), (1.0, 1e30)])
def test_sizes_of_values(cuda_lib, M, d, dtype, scale, eps):
    x, dy, w = inputs(M, d, dtype, F32, 90)
    x, r = x * scale, randn(93, M, d, dtype=dtype) * scale
    y, s = swg.rms_norm(x, w, residual=r, eps=eps)
    check_norm(y, s, x, r, w, eps)
    if scale > 2.0 ** -40 and eps < 1e10:   # (elsewhere t, or the scale, leaves the normal range)
        rows, s2 = swg.rms_norm_fp8(x, w, residual=r, eps=eps)
        check_fp8(rows, x, r, w, eps)
        assert torch.equal(s, s2)
    check_backward(*swg.rms_norm_backward(dy, s, w, eps=eps), dy, s, w, None, eps)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", [(3, 64), (200, 897), (3, 4096), (300, 1000), (4, 20000), (5, 30001)])
@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-39, 2.0 ** -126, 1e-37])
def test_smallest_eps(cuda_lib, M, d, dtype, eps):
    """Rows of zeros, and rows whose squares are below binary32, have finite gradients: r is at most
    2^74.5, and g r what dx then is.  (The squares that are lost would change r by less than 2^-28,
    eps in binary32 by less than 2^-22.)"""
    _, dy, w = inputs(M, d, dtype, F32, 97)
    s = torch.zeros(M, d, device=DEV, dtype=dtype)
    s[1] = 2.0 ** -90 * (1 + torch.arange(d, device=DEV) % 3)   # s^2 <= 9 * 2^-180
    s[2:] = inputs(M, d, dtype, F32, 98)[0][2:]
    y = swg.rms_norm(s, w, eps=eps)
    assert bool(y.isfinite().all()) and not bool(y[0].any())
    check_backward(*swg.rms_norm_backward(dy, s, w, eps=eps), dy, s, w, None, eps)


def test_nothing_to_do(cuda_lib):
    for M, d in ((0, 64), (4, 0), (0, 0)):
        x, w = torch.empty(M, d, device=DEV, dtype=BF), torch.ones(d, device=DEV, dtype=BF)
        assert swg.rms_norm(x, w).shape == (M, d)
        rows, s = swg.rms_norm_fp8(x, w, residual=x.clone())
        assert rows.codes.shape == (M, d) and not bool(rows.scales.any())
        dx, dw = swg.rms_norm_backward(x, x, w)
        assert dx.shape == (M, d) and dw.shape == (d,) and not bool(dw.any())
        assert swg.rms_norm_backward_workspace_bytes(M, d) == 0
    with pytest.raises(swg.SwiGLUError):
        swg.rms_norm_backward_workspace_bytes(4, -1)


def test_refusals(cuda_lib):
    x, r, w = inputs(4, 64, BF, BF)
    bad = [lambda: swg.rms_norm(x.t(), w), lambda: swg.rms_norm(x, w[:32]),
           lambda: swg.rms_norm(x, w[::2]), lambda: swg.rms_norm(x, w, residual=r[:2]),
           lambda: swg.rms_norm(x, w, residual=r.cpu()), lambda: swg.rms_norm(x, w, sum_out=r),
           lambda: swg.rms_norm(x, w, out=x.float()), lambda: swg.rms_norm(x[0], w),
           lambda: swg.rms_norm_fp8(x, w, out=(x, x)),
           lambda: swg.rms_norm_backward(x[:2], x, w)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: swg.rms_norm(x.half(), w), lambda: swg.rms_norm(x, w.half()),
                 lambda: swg.rms_norm(x, w, residual=r.float())):
        with pytest.raises(TypeError):
            call()
    odd = torch.empty(4 * 64 + 1, device=DEV, dtype=BF)[1:].view(4, 64)
    short = torch.empty(swg.rms_norm_backward_workspace_bytes(4, 64) - 1, device=DEV, dtype=torch.uint8)
    for call in (lambda: swg.rms_norm(x, w, eps=0.0), lambda: swg.rms_norm(odd, w),
                 lambda: swg.rms_norm(x, w, out=w.expand(4, 64).contiguous()[:4], residual=r,
                                      sum_out=r[:4], eps=-1.0),
                 lambda: swg.rms_norm_backward(x, x, w, workspace=short)):
        with pytest.raises(swg.SwiGLUError):
            call()


@pytest.mark.parametrize("M,d", [(16, 4096), (700, 897), (9, 20000)])
def test_streams_graphs_and_repeats(cuda_lib, M, d):
    x, r, w = inputs(M, d, BF, F32)
    dy = randn(70, M, d)

    def calls(stream=None, workspace=None):
        y, s = swg.rms_norm(x, w, residual=r, stream=stream)
        rows = swg.rms_norm_fp8(x, w, stream=stream)
        return [y, s, *rows, *swg.rms_norm_backward(dy, s, w, ds=y, stream=stream,
                                                    workspace=workspace)]

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))
    want = calls()
    n = swg.rms_norm_backward_workspace_bytes(M, d)
    assert same(want, calls(workspace=torch.empty(n, device=DEV, dtype=torch.uint8)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = calls(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert same(want, got)
    with torch.cuda.stream(st):
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = calls()
    x.copy_(randn(71, M, d))
    graph.replay()
    torch.cuda.synchronize()
    assert same(calls(), got)
    graph.replay()
    swg.rms_norm_backward(dy, x, w)
    graph.replay()
    torch.cuda.synchronize()
    assert same(calls(), got)


def test_offsets_past_32_bits(cuda_lib):
    M, d = 70001, 32752           # 2.29e9 elements
    x = torch.zeros(M, d, device=DEV, dtype=BF)
    w = torch.ones(d, device=DEV, dtype=BF)
    tail = randn(80, 3, d)
    x[-3:] = tail
    y = swg.rms_norm(x, w)
    check_norm(y[-3:], None, tail, None, w, 1e-6)
    assert not bool(y[:1000].any())
    del y
    rows = swg.rms_norm_fp8(x, w)
    check_fp8(swg.Fp8Rows(rows.codes[-3:], rows.scales[-3:]), tail, None, w, 1e-6)
    del rows
    dx, dw = swg.rms_norm_backward(x, x, w)
    rx, rw, size, wsize = ref_backward(tail, tail, w, None, 1e-6)
    assert bool(((dx[-3:].to(D) - rx).abs() <= rx.abs() * 2.0 ** -8 + 2.0 ** -16 * size).all())
    assert bool(((dw.to(D) - rw).abs() <= rw.abs() * 2.0 ** -8 + 2.0 ** -17 * wsize).all())
