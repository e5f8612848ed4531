"""The experts' products against their definitions in 64 bits.

Tolerance: the rule of the dense operations.  An f32 sum of K products is off
by about sqrt(K) 2^-24 sum |x w|; eight times that, through the sensitivity of
h = silu(g) u (1.1 |u| per g, |silu(g)| per u), or |weight| for a term of y;
plus 2^-8 of the result for its rounding to bf16 (half an ulp is 2^-9) and the
fast exponential, and, for y, 2^-8 of each weighted term.
"""
import math

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64
BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_ids(T, E, k, seed, skew=0.0, dropped=0.0):
    g = gen(seed)
    pop = torch.randn(E, generator=g, device=DEV) * skew
    ids = torch.argsort(torch.rand(T, E, generator=g, device=DEV) + pop, dim=1)[:, :k].int()
    if dropped:
        ids[torch.rand(T, k, generator=g, device=DEV) < dropped] = -1
    w = torch.rand(T, k, generator=g, device=DEV)
    return ids.contiguous(), w


def weights(E, K, N, seed, layout, scale=None):
    g = gen(seed)
    w = (torch.randn(E, K, N, generator=g, device=DEV) * (scale or max(1, K) ** -0.5)).to(BF)
    return w if layout == "kn" else w.transpose(1, 2).contiguous()


def ref_rows(rt, E, a, w, layout):
    """(sum, sum of absolute products) of every sorted row, in 64 bits; `a`
    is indexed by sorted row."""
    off = rt.offsets.tolist()
    N = w.shape[2] if layout == "kn" else w.shape[1]
    v = torch.zeros(a.shape[0], N, dtype=D, device=DEV)
    s = torch.zeros_like(v)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            we = (w[e] if layout == "kn" else w[e].t()).to(D)
            v[lo:hi] = a[lo:hi].to(D) @ we
            s[lo:hi] = a[lo:hi].to(D).abs() @ we.abs()
    return v, s


def check_up(h, x, wg, wu, rt, E, k, layout):
    n = rt.offsets[-1].item()
    tok = rt.order.long().clamp_min(0) // k
    a = x[tok] if n else x.new_zeros(tok.shape[0], x.shape[1])
    g, sg = ref_rows(rt, E, a, wg, layout)
    u, su = ref_rows(rt, E, a, wu, layout)
    ref = g * torch.sigmoid(g) * u
    f = 8 * math.sqrt(max(1, x.shape[1])) * 2.0 ** -24
    tol = 2.0 ** -8 * ref.abs() + f * (1.1 * sg * u.abs() + (g * torch.sigmoid(g)).abs() * su) \
        + f * f * 1.1 * sg * su
    err = (h.to(D) - ref).abs()
    assert bool((err[:n] <= tol[:n] + 1e-37).all()), (err - tol).max().item()
    assert not bool(h[n:].any())


def check_down(y, h, wd, rt, E, layout, residual):
    T, k = rt.position.shape
    z, s = ref_rows(rt, E, h, wd, layout)
    zero = torch.zeros(1, z.shape[1], dtype=D, device=DEV)
    z, s = torch.cat([z, zero]), torch.cat([s, zero])
    ref = torch.zeros(T, z.shape[1], dtype=D, device=DEV)
    tol = torch.zeros_like(ref)
    if residual is not None:
        ref += residual.to(D)
        tol += 2.0 ** -22 * residual.to(D).abs()
    f = 8 * math.sqrt(max(1, h.shape[1])) * 2.0 ** -24
    for j in range(k):
        p = rt.position[:, j].long()
        w = rt.weights[:, j:j + 1].to(D)
        ref += w * z[p]
        tol += w.abs() * (f * s[p] + 2.0 ** -8 * z[p].abs())
    tol += 2.0 ** -8 * ref.abs()
    err = (y.to(D) - ref).abs()
    assert bool((err <= tol + 1e-37).all()), (err - tol).max().item()


CASES = [  # T, E, k, d, d_ff, skew, dropped
    (1, 1, 1, 8, 8, 0, 0), (1, 8, 2, 64, 128, 0, 0), (1, 64, 8, 2048, 1024, 0, 0),
    (2, 4, 4, 72, 136, 0, 0), (5, 60, 4, 200, 264, 0, 0.3), (16, 8, 2, 896, 4864, 0, 0),
    (33, 5, 3, 264, 72, 1.0, 0.1), (64, 64, 8, 256, 256, 0, 0), (100, 3, 1, 1000, 40, 2.0, 0),
    (257, 2, 1, 128, 520, 0, 0), (300, 7, 2, 136, 256, 0.5, 0.2), (600, 1, 1, 328, 264, 0, 0),
    (700, 16, 4, 512, 640, 0.3, 0), (1500, 4, 2, 192, 1032, 3.0, 0.05),
    (40, 1024, 2, 64, 64, 0, 0), (2000, 128, 8, 128, 192, 0.5, 0)]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("T,E,k,d,d_ff,skew,dropped", CASES)
def test_up(cuda_lib, T, E, k, d, d_ff, skew, dropped, layout):
    ids, w = make_ids(T, E, k, T + E, skew, dropped)
    rt = swg.dispatch(ids, E, w)
    x = torch.randn(T, d, generator=gen(1), device=DEV).to(BF)
    wg, wu = weights(E, d, d_ff, 2, layout), weights(E, d, d_ff, 3, layout)
    h = swg.experts_up(x, wg, wu, rt, layout=layout)
    check_up(h, x, wg, wu, rt, E, k, layout)
    swg.check_device_status()


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("T,E,k,d,d_ff,skew,dropped", CASES)
def test_down(cuda_lib, T, E, k, d, d_ff, skew, dropped, layout):
    ids, w = make_ids(T, E, k, T + E, skew, dropped)
    rt = swg.dispatch(ids, E, w)
    h = torch.randn(T * k, d_ff, generator=gen(1), device=DEV).to(BF)
    wd = weights(E, d_ff, d, 2, layout)
    r = torch.randn(T, d, generator=gen(4), device=DEV).to(BF) if T % 2 else None
    y = swg.experts_down(h, wd, rt, residual=r, layout=layout)
    check_down(y, h, wd, rt, E, layout, r)
    swg.check_device_status()


def test_every_choice_dropped(cuda_lib):
    ids = torch.full((9, 2), -1, device=DEV, dtype=torch.int32)
    rt = swg.dispatch(ids, 4, torch.rand(9, 2, device=DEV))
    x = torch.randn(9, 64, device=DEV).to(BF)
    w = weights(4, 64, 72, 0, "kn")
    out = torch.full((18, 72), 3.0, device=DEV, dtype=BF)
    assert not bool(swg.experts_up(x, w, w, rt, out=out).any())
    wd = weights(4, 72, 64, 0, "kn")
    h = torch.full((18, 72), float("nan"), device=DEV, dtype=BF)
    assert not bool(swg.experts_down(h, wd, rt).any())
    assert torch.equal(swg.experts_down(h, wd, rt, residual=x), x)


def test_nan_stays_where_it_is(cuda_lib):
    # a dropped token's x, an unreached expert's weights, and the rows that a
    # k tail or a chunk's end runs into: none of them reaches another row
    T, E, d, d_ff = 70, 6, 72, 136
    ids = torch.randint(0, E, (T, 1), generator=gen(0), device=DEV, dtype=torch.int32)
    ids[ids == 3] = 2
    ids[5] = -1
    rt = swg.dispatch(ids, E, torch.ones(T, 1, device=DEV))
    x = torch.randn(T, d, generator=gen(1), device=DEV).to(BF)
    for layout in ("kn", "nk"):
        wg, wu = weights(E, d, d_ff, 2, layout), weights(E, d, d_ff, 3, layout)
        wd = weights(E, d_ff, d, 4, layout)
        h0 = swg.experts_up(x, wg, wu, rt, layout=layout)
        y0 = swg.experts_down(h0, wd, rt, layout=layout)
        assert bool(torch.isfinite(h0).all()) and not bool(y0[5].any())
        x1 = x.clone()
        x1[5] = float("nan")
        for m in (wg, wu, wd):
            m[3] = float("nan")
        assert torch.equal(swg.experts_up(x1, wg, wu, rt, layout=layout), h0)
        h1 = h0.clone()
        h1[rt.offsets[-1].item():] = float("inf")
        assert torch.equal(swg.experts_down(h1, wd, rt, layout=layout), y0)
        # ... and a NaN that belongs to a row stays in that row
        x1[7] = float("inf")
        h2 = swg.experts_up(x1, wg, wu, rt, layout=layout)
        row = rt.position[7, 0].item()
        keep = torch.arange(T, device=DEV) != row
        assert torch.equal(h2[keep], h0[keep]) and not bool(torch.isfinite(h2[row]).all())


def test_unlikely_routing_stays_inside(cuda_lib):
    # offsets and order that dispatch would not write: no row outside the
    # tensors is read or written (guard bands keep their value)
    T, E, k, d, d_ff = 20, 4, 2, 64, 72
    x = torch.randn(T, d, device=DEV).to(BF)
    w = weights(E, d, d_ff, 2, "kn")
    wd = weights(E, d_ff, d, 2, "kn")
    bad = torch.tensor([-5, 1000, 3, 2 ** 31 - 1, 2 ** 30], device=DEV, dtype=torch.int32)
    order = torch.full((T * k,), 2 ** 31 - 1, device=DEV, dtype=torch.int32)
    order[::3] = -7
    pos = torch.full((T, k), 2 ** 31 - 1, device=DEV, dtype=torch.int32)
    rt = swg.Routing(pos, torch.ones(T, k, device=DEV), bad, order, pos)
    buf = torch.full((T * k * d_ff + 1024,), 5.0, device=DEV, dtype=BF)
    h = buf[512:512 + T * k * d_ff].view(T * k, d_ff)
    swg.experts_up(x, w, w, rt, out=h)
    assert bool((buf[:512] == 5).all()) and bool((buf[512 + T * k * d_ff:] == 5).all())
    assert not bool(swg.experts_down(h, wd, rt).any())
    swg.check_device_status()


def test_empty_sizes(cuda_lib):
    ids, w = make_ids(6, 4, 2, 0)
    rt = swg.dispatch(ids, 4, w)
    x = torch.randn(6, 64, device=DEV).to(BF)
    e = torch.empty
    assert not bool(swg.experts_up(x[:, :0].contiguous(), e(4, 0, 16, device=DEV, dtype=BF),
                                   e(4, 0, 16, device=DEV, dtype=BF), rt).any())
    assert swg.experts_up(x, e(4, 64, 0, device=DEV, dtype=BF), e(4, 64, 0, device=DEV, dtype=BF),
                          rt).shape == (12, 0)
    y = swg.experts_down(e(12, 0, device=DEV, dtype=BF), e(4, 0, 64, device=DEV, dtype=BF), rt,
                         residual=x)
    assert torch.equal(y, x)
    none = swg.dispatch(e(0, 2, device=DEV, dtype=torch.int32), 4, e(0, 2, device=DEV))
    assert swg.experts_up(x[:0], weights(4, 64, 8, 0, "kn"), weights(4, 64, 8, 0, "kn"),
                          none).shape == (0, 8)
    assert swg.experts_down(e(0, 8, device=DEV, dtype=BF), weights(4, 8, 64, 0, "kn"),
                            none).shape == (0, 64)
    zero = swg.dispatch(e(6, 0, device=DEV, dtype=torch.int32), 4, e(6, 0, device=DEV))
    assert torch.equal(swg.experts_down(e(0, 8, device=DEV, dtype=BF), weights(4, 8, 64, 0, "kn"),
                                        zero, residual=x), x)


def test_residual_in_place(cuda_lib):
    ids, w = make_ids(50, 4, 2, 0)
    rt = swg.dispatch(ids, 4, w)
    h = torch.randn(100, 136, device=DEV).to(BF)
    wd = weights(4, 136, 72, 1, "kn")
    r = torch.randn(50, 72, device=DEV).to(BF)
    want = swg.experts_down(h, wd, rt, residual=r)
    got = r.clone()
    swg.experts_down(h, wd, rt, residual=got, out=got)
    assert torch.equal(got, want)


def test_same_bits_every_time(cuda_lib):
    for T, E, k, d, d_ff in [(1, 16, 4, 1024, 512), (200, 8, 2, 256, 520)]:
        ids, w = make_ids(T, E, k, 0)
        rt = swg.dispatch(ids, E, w)
        x = torch.randn(T, d, device=DEV).to(BF)
        wg, wu, wd = weights(E, d, d_ff, 0, "kn"), weights(E, d, d_ff, 1, "kn"), \
            weights(E, d_ff, d, 2, "kn")
        h = swg.experts_up(x, wg, wu, rt)
        y = swg.experts_down(h, wd, rt, residual=x)
        for _ in range(5):
            assert torch.equal(swg.experts_up(x, wg, wu, rt), h)
            assert torch.equal(swg.experts_down(h, wd, rt, residual=x), y)


def test_offsets_past_31_bits(cuda_lib):
    # h has more than 2^31 values
    T, E, k, d, d_ff = 140000, 2, 2, 8, 8192
    ids = torch.tensor([[0, 1]], device=DEV, dtype=torch.int32).expand(T, 2).contiguous()
    rt = swg.dispatch(ids, E, torch.full((T, k), 0.5, device=DEV))
    x = torch.randn(T, d, device=DEV).to(BF)
    wg, wu = weights(E, d, d_ff, 0, "kn"), weights(E, d, d_ff, 1, "kn")
    h = swg.experts_up(x, wg, wu, rt)
    assert h.numel() > 2 ** 31
    for lo in (0, T - 3, 2 * T - 40):
        e = 0 if lo + 40 <= T else 1
        lo = lo if lo + 40 <= T or lo >= T else T
        a = x[lo % T:lo % T + 40].to(D)
        g, u = a @ wg[e].to(D), a @ wu[e].to(D)
        ref = g * torch.sigmoid(g) * u
        assert bool(((h[lo:lo + a.shape[0]].to(D) - ref).abs() <= 2.0 ** -7 * ref.abs() + 1e-4).all())
    wd = weights(E, d_ff, d, 2, "kn")
    y = swg.experts_down(h, wd, rt)
    tail = torch.arange(T - 5, T, device=DEV)
    ref = 0.5 * (h[tail].to(D) @ wd[0].to(D) + h[tail + T].to(D) @ wd[1].to(D))
    assert bool(((y[tail].to(D) - ref).abs() <= 2.0 ** -6 * ref.abs() + 1e-2).all())


def moe_parts(T, E, k, d, d_ff, seed, layout="kn"):
    g = gen(seed)
    x = torch.randn(T, d, generator=g, device=DEV).to(BF)
    wr = (torch.randn(*((d, E) if layout == "kn" else (E, d)), generator=g, device=DEV)
          * d ** -0.5).to(BF)
    return x, wr, weights(E, d, d_ff, seed + 1, layout), weights(E, d, d_ff, seed + 2, layout), \
        weights(E, d_ff, d, seed + 3, layout)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("T,E,k,d,d_ff", [(1, 16, 4, 512, 256), (77, 8, 2, 256, 264)])
def test_moe(cuda_lib, T, E, k, d, d_ff, layout):
    x, wr, wg, wu, wd = moe_parts(T, E, k, d, d_ff, 0, layout)
    b = torch.randn(E, device=DEV)
    y, r = swg.swiglu_moe(x, wr, wg, wu, wd, k, router_bias=b, residual=x, layout=layout,
                          score="sigmoid", bias=torch.rand(E, device=DEV), scale=2.0)
    h = swg.experts_up(x, wg, wu, r, layout=layout)
    check_up(h, x, wg, wu, r, E, k, layout)
    check_down(y, h, wd, r, E, layout, x)


def test_moe_in_a_graph(cuda_lib):
    # one capture, replayed on inputs that route differently
    T, E, k, d, d_ff = 24, 8, 2, 256, 264
    x, wr, wg, wu, wd = moe_parts(T, E, k, d, d_ff, 0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, r = swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x)
    for seed in (1, 2, 3):
        x.copy_(torch.randn(T, d, generator=gen(seed), device=DEV).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        want, rw = swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x)
        assert torch.equal(r.ids, rw.ids) and torch.equal(y, want)
    swg.check_device_status()


def test_graph_shared_with_dense_calls(cuda_lib):
    # dense and routed calls of one capture share a workspace slice
    T, E, k, d, d_ff = 4, 4, 2, 4096, 4096
    x, wr, wg, wu, wd = moe_parts(T, E, k, d, d_ff, 0)

    def step():
        h = swg.swiglu_up(x, wg[0], wu[0])
        a = swg.swiglu_down(h, wd[0], residual=x)
        y, _ = swg.swiglu_moe(a, wr, wg, wu, wd, k, residual=a)
        h = swg.swiglu_up(y, wg[1], wu[1])
        return swg.swiglu_down(h, wd[1], residual=y)
    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    swg.check_device_status()


def test_two_streams(cuda_lib):
    T, E, k, d, d_ff = 40, 8, 2, 512, 264
    parts = [moe_parts(T, E, k, d, d_ff, s) for s in (10, 20)]
    want = [swg.swiglu_moe(*p, k, residual=p[0])[0] for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    got = []
    for _ in range(10):
        got = []
        for p, s in zip(parts, streams):
            with torch.cuda.stream(s):
                got.append(swg.swiglu_moe(*p, k, residual=p[0])[0])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals(cuda_lib):
    T, E, k, d, d_ff = 6, 4, 2, 64, 72
    ids, w = make_ids(T, E, k, 0)
    rt = swg.dispatch(ids, E, w)
    x = torch.randn(T, d, device=DEV).to(BF)
    wg = weights(E, d, d_ff, 0, "kn")
    wd = weights(E, d_ff, d, 0, "kn")
    h = torch.zeros(T * k, d_ff, device=DEV, dtype=BF)
    with pytest.raises(TypeError):
        swg.experts_up(x.float(), wg, wg, rt)
    with pytest.raises(ValueError):
        swg.experts_up(x, wg, wg, rt, layout="nk")
    with pytest.raises(ValueError):
        swg.experts_up(x, wg, wg.transpose(1, 2), rt)
    with pytest.raises(ValueError):
        swg.experts_up(x[:5], wg, wg, rt)
    with pytest.raises(ValueError):
        swg.experts_up(x, wg[:3].contiguous(), wg[:3].contiguous(), rt)
    with pytest.raises(TypeError):
        swg.experts_up(x, wg, wg, rt._replace(order=rt.order.long()))
    with pytest.raises(ValueError):
        swg.experts_up(x, wg, wg, rt, out=torch.empty(T, d_ff, device=DEV, dtype=BF))
    with pytest.raises(ValueError):
        swg.experts_down(h[:4], wd, rt)
    with pytest.raises(ValueError):
        swg.experts_down(h, wd, rt._replace(weights=None))
    with pytest.raises(ValueError):
        swg.experts_down(h, wd, rt, residual=x[:3])
    with pytest.raises(swg.SwiGLUError) as e:     # d_ff not a multiple of 8
        swg.experts_up(x, wg[:, :, :12].contiguous(), wg[:, :, :12].contiguous(), rt)
    assert e.value.status == 3
    with pytest.raises(swg.SwiGLUError) as e:     # a workspace that is too small
        swg.experts_up(x, wg, wg, rt, workspace=torch.empty(256, device=DEV, dtype=torch.uint8))
    assert e.value.status == 8


def test_workspace_of_the_caller(cuda_lib):
    T, E, k, d, d_ff = 6, 4, 2, 64, 72
    ids, w = make_ids(T, E, k, 0)
    rt = swg.dispatch(ids, E, w)
    x = torch.randn(T, d, device=DEV).to(BF)
    wg, wd = weights(E, d, d_ff, 0, "kn"), weights(E, d_ff, d, 0, "kn")
    nu = swg.experts_up_workspace_bytes(T, k, E, d, d_ff)
    nd = swg.experts_down_workspace_bytes(T, k, E, d_ff, d)
    ws = torch.full((max(nu, nd),), 255, device=DEV, dtype=torch.uint8)
    h = swg.experts_up(x, wg, wg, rt)
    assert torch.equal(swg.experts_up(x, wg, wg, rt, workspace=ws[:nu]), h)
    y = swg.experts_down(h, wd, rt)
    assert torch.equal(swg.experts_down(h, wd, rt, workspace=ws[:nd]), y)


def test_allocation_failure(cuda_lib, monkeypatch):
    x, wr, wg, wu, wd = moe_parts(4, 4, 2, 64, 72, 0)
    monkeypatch.setenv("SWIGLU_INJECT_OOM", "1")
    with pytest.raises(swg.SwiGLUError) as e:
        swg.linear(x, wr)
    assert e.value.status == 4
    monkeypatch.delenv("SWIGLU_INJECT_OOM")
    swg.swiglu_moe(x, wr, wg, wu, wd, 2)
    swg.check_device_status()
