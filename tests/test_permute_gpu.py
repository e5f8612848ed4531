"""Rows sorted by expert and back, and their gradients, against indexing and sums in 64 bits.

permute copies: equality.  unpermute: k + 1 terms added in f32, each step off by
u = 2^-24 of the terms' sizes, and half a step of the type.  dz: one product and
one rounding.  dweights: a thread adds at most d / 32 products, then 32 lanes and
eight warps.
"""
import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=gen(seed), device=DEV).to(dtype)


def routing(T, E, k, seed, dropped=0.0):
    g = gen(seed)
    ids = torch.argsort(torch.rand(T, E, generator=g, device=DEV), dim=1)[:, :k].int()
    ids[torch.rand(T, k, generator=g, device=DEV) < dropped] = -1
    return swg.dispatch(ids.contiguous(), E, torch.randn(T, k, generator=g, device=DEV))


def pairs(rt, E):
    """Flat (token, choice) indices by expert, from the ids alone."""
    ids = rt.ids.reshape(-1)
    return torch.cat([torch.nonzero(ids == e)[:, 0] for e in range(E)])


CASES = [  # T, E, k, d, dropped
    (1, 1, 1, 1, 0), (1, 64, 8, 2048, 0), (1, 8, 2, 4097, 0), (2, 40, 32, 24, 0.2), (3, 4, 4, 8, 0.5),
    (5, 60, 4, 200, 0.3), (17, 16, 9, 514, 0.1), (33, 5, 3, 36, 0.1), (64, 64, 8, 256, 0), (100, 3, 1, 1001, 0.4),
    (300, 7, 2, 136, 0.2), (1000, 128, 8, 768, 0.05), (2500, 4, 2, 20, 0), (40, 1024, 17, 65, 0.1),
    (333, 8, 2, 896, 1.0), (9, 8, 8, 16384, 0.1)]

# enough tokens for the kernels that copy rows ahead: long, middle and short rows, with few
# choices and many, in whole 16-byte pieces and not
LARGE = [(9000, 64, 8, 1024, 0.05), (8500, 64, 6, 1027, 0.05), (7000, 8, 2, 128, 0.1), (7000, 8, 1, 130, 0),
         (17000, 16, 6, 520, 0.02), (17000, 16, 5, 519, 0.02), (7000, 8, 3, 128, 0), (7000, 60, 4, 133, 0.3),
         (40000, 32, 9, 256, 0.02), (36000, 32, 7, 251, 0), (30000, 40, 17, 300, 0.1), (3000, 8, 2, 4096, 0.01)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,d,dropped", CASES + LARGE[:4])
def test_permute(cuda_lib, T, E, k, d, dropped, dtype):
    rt = routing(T, E, k, T + d, dropped)
    x = randn(1, T, d, dtype=dtype)
    p = pairs(rt, E)
    out = torch.full((T * k, d), float("nan"), device=DEV, dtype=dtype)
    assert swg.permute(x, rt, out=out) is out
    n = p.numel()
    assert torch.equal(out[:n], x[p // k]) and not bool(out[n:].any())
    # the gradient of x, with one that reaches it another way
    dout, r = randn(2, T * k, d, dtype=dtype), randn(3, T, d, dtype=dtype)
    dout[n:] = float("nan")   # rows of no pair
    for resid in (None, r):
        ref = torch.zeros(T, d, dtype=D, device=DEV) if resid is None else resid.to(D)
        size = ref.abs().index_add(0, p // k, dout[:n].to(D).abs())
        ref = ref.index_add(0, p // k, dout[:n].to(D))
        err = (swg.permute_backward(dout, rt, residual=resid).to(D) - ref).abs()
        assert bool((err <= ref.abs() * HALF[dtype] + (k + 1) * U * size).all())


@pytest.mark.parametrize("T,E,k,d,dropped", CASES + LARGE[:4])
def test_permute_fp8(cuda_lib, T, E, k, d, dropped):
    rt = routing(T, E, k, T + d, dropped)
    g = gen(4)
    x = swg.Fp8Rows(torch.randint(0, 256, (T, d), generator=g, device=DEV).to(torch.uint8),
                    torch.rand(T, generator=g, device=DEV) + 0.5)
    p = pairs(rt, E)
    n = p.numel()
    out = swg.permute(x, rt)
    assert torch.equal(out.codes[:n], x.codes[p // k]) and not bool(out.codes[n:].any())
    assert torch.equal(out.scales[:n], x.scales[p // k]) and not bool(out.scales[n:].any())
    mine = swg.Fp8Rows(torch.full_like(out.codes, 7), torch.full_like(out.scales, 7))
    again = swg.permute(x, rt, out=mine)
    assert again.codes is mine.codes and torch.equal(mine.codes, out.codes)
    assert torch.equal(mine.scales, out.scales)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,d,dropped", CASES + LARGE)
def test_unpermute(cuda_lib, T, E, k, d, dropped, dtype):
    rt = routing(T, E, k, T + d, dropped)
    z, r = randn(1, T * k, d, dtype=dtype), randn(3, T, d, dtype=dtype)
    p = pairs(rt, E)
    n = p.numel()
    z[n:] = float("nan")
    rt.weights[rt.ids < 0] = float("nan")   # a dropped choice adds nothing, whatever its weight
    w = rt.weights.to(D).reshape(-1)[p, None]
    for resid in (None, r):
        ref = torch.zeros(T, d, dtype=D, device=DEV) if resid is None else resid.to(D)
        size = ref.abs().index_add(0, p // k, (w * z[:n].to(D)).abs())
        ref = ref.index_add(0, p // k, w * z[:n].to(D))
        y = swg.unpermute(z, rt, residual=resid)
        err = (y.to(D) - ref).abs()
        assert bool((err <= ref.abs() * HALF[dtype] + (k + 1) * U * size).all())
    r2 = r.clone()
    assert swg.unpermute(z, rt, residual=r2, out=r2) is r2 and torch.equal(r2, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,d,dropped", CASES + LARGE)
def test_unpermute_backward(cuda_lib, T, E, k, d, dropped, dtype):
    rt = routing(T, E, k, T + d, dropped)
    z, dy = randn(1, T * k, d, dtype=dtype), randn(3, T, d, dtype=dtype)
    p = pairs(rt, E)
    n = p.numel()
    z[n:] = float("nan")
    rt.weights[rt.ids < 0] = float("nan")
    out = torch.full((T * k, d), float("nan"), device=DEV, dtype=dtype)
    dz, dw = swg.unpermute_backward(dy, z, rt, out=out)
    assert dz is out and not bool(dz[n:].any())
    g = dy[p // k].to(D)
    ref = rt.weights.to(D).reshape(-1)[p, None] * g
    assert bool(((dz[:n].to(D) - ref).abs() <= ref.abs() * (HALF[dtype] + U) + 2.0 ** -126).all())
    ref, size = torch.zeros(T * k, dtype=D, device=DEV), torch.zeros(T * k, dtype=D, device=DEV)
    ref[p], size[p] = (g * z[:n].to(D)).sum(1), (g * z[:n].to(D)).abs().sum(1)
    err = (dw.to(D).reshape(-1) - ref).abs()
    assert bool((err <= U * (d / 32 + 16) * size).all())
    assert not bool(dw[rt.ids < 0].any())


# rows shorter than 16 bytes, several to a piece: few tokens, and enough for the kernels that copy ahead
NARROW = [(3, 4, 2, 1, 0), (1, 10, 10, 1, 0), (5, 8, 2, 3, 0.2), (9, 8, 3, 7, 0), (7, 4, 1, 5, 0.3), (4, 9, 9, 2, 0),
          (50000, 8, 2, 1, 0.1), (50000, 16, 4, 3, 0), (50000, 4, 1, 7, 0.2)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,d,dropped", NARROW)
def test_rows_shorter_than_a_piece(cuda_lib, T, E, k, d, dropped, dtype):
    test_permute(cuda_lib, T, E, k, d, dropped, dtype)
    test_unpermute(cuda_lib, T, E, k, d, dropped, dtype)
    test_unpermute_backward(cuda_lib, T, E, k, d, dropped, dtype)
    test_permute_fp8(cuda_lib, T, E, k, d, dropped)


def test_gradients_against_differences(cuda_lib):
    T, E, k, d = 6, 5, 3, 20
    rt = routing(T, E, k, 7, 0.2)
    p = pairs(rt, E)
    x, z, dy = randn(1, T, d, dtype=F32), randn(2, T * k, d, dtype=F32), randn(3, T, d, dtype=F32)
    dout = randn(4, T * k, d, dtype=F32)
    dx = swg.permute_backward(dout, rt).to(D)
    dz, dw = (t.to(D) for t in swg.unpermute_backward(dy, z, rt))

    def sorted_rows(x):
        out = torch.zeros(T * k, d, dtype=D, device=DEV)
        out[:p.numel()] = x[p // k]
        return out

    def back(z, w):
        return torch.zeros(T, d, dtype=D, device=DEV).index_add(
            0, p // k, w.reshape(-1)[p, None] * z[:p.numel()])
    w = rt.weights.to(D)
    for seed in range(3):   # (all linear in what is moved: the difference is exact but for rounding)
        v, vz, vw = randn(10 + seed, T, d, dtype=D), randn(20 + seed, T * k, d, dtype=D), \
            randn(30 + seed, T, k, dtype=D)
        for got, diff, size in (
                ((dx * v).sum(), ((sorted_rows(x.to(D) + v) - sorted_rows(x.to(D) - v)) / 2 * dout.to(D)).sum(),
                 (dx.abs() * v.abs()).sum()),
                ((dz * vz).sum(), ((back(z.to(D) + vz, w) - back(z.to(D) - vz, w)) / 2 * dy.to(D)).sum(),
                 (dz.abs() * vz.abs()).sum()),
                ((dw * vw).sum(), ((back(z.to(D), w + vw) - back(z.to(D), w - vw)) / 2 * dy.to(D)).sum(),
                 (vw.abs().sum() * d * 4))):
            assert abs(got - diff) <= 2.0 ** -19 * size


@pytest.mark.parametrize("T,k,d", [(40, 3, 64), (40, 3, 65), (7000, 3, 128), (7000, 2, 130), (40000, 9, 256),
                                   (36000, 7, 251)])
def test_a_routing_of_another_making_stays_inside(cuda_lib, T, k, d):
    """Positions and offsets out of range move nothing outside the tensors."""
    E = 6
    g = gen(5)
    pos = torch.randint(-(1 << 30), 1 << 30, (T, k), generator=g, device=DEV).int()
    pos[::3] = torch.randint(0, T * k, pos[::3].shape, generator=g, device=DEV).int()
    w = torch.rand(T, k, generator=g, device=DEV)
    x = randn(1, T, d)
    for end in (-5, 7, T * k, 1 << 30):
        off = torch.full((E + 1,), end, device=DEV, dtype=torch.int32)
        rt = swg.Routing(pos, w, off, pos.reshape(-1), pos)
        band = torch.full(((T * k + 16) * d,), 3.0, device=DEV, dtype=BF)
        out = band[8 * d:(T * k + 8) * d].view(T * k, d)
        swg.permute(x, rt, out=out)
        z = randn(2, T * k, d)
        swg.unpermute(z, rt)
        swg.unpermute_backward(x, z, rt, out=out)
        assert bool((band[:8 * d] == 3).all()) and bool((band[(T * k + 8) * d:] == 3).all())


def test_nothing_to_do(cuda_lib):
    ids = torch.empty(0, 2, device=DEV, dtype=torch.int32)
    rt = swg.dispatch(ids, 4, torch.empty(0, 2, device=DEV))
    x = torch.empty(0, 64, device=DEV, dtype=BF)
    assert swg.permute(x, rt).shape == (0, 64) and swg.unpermute(x, rt).shape == (0, 64)
    assert swg.unpermute_backward(x, x, rt)[1].shape == (0, 2)
    rt = swg.dispatch(torch.empty(3, 0, device=DEV, dtype=torch.int32), 4, torch.empty(3, 0, device=DEV))
    x, z = randn(1, 3, 64), torch.empty(0, 64, device=DEV, dtype=BF)
    assert swg.permute(x, rt).shape == (0, 64)
    assert torch.equal(swg.unpermute(z, rt, residual=x), x) and not bool(swg.unpermute(z, rt).any())
    assert swg.unpermute_backward(x, z, rt)[0].shape == (0, 64)
    rt = routing(5, 4, 2, 1)
    x = torch.empty(5, 0, device=DEV, dtype=BF)
    z = torch.empty(10, 0, device=DEV, dtype=BF)
    assert swg.permute(x, rt).shape == (10, 0) and not bool(swg.unpermute_backward(x, z, rt)[1].any())
    s = swg.permute(swg.Fp8Rows(x.to(torch.uint8), torch.ones(5, device=DEV)), rt).scales
    assert bool((s == 1).all())


def test_refusals(cuda_lib):
    T, E, k, d = 4, 8, 2, 64
    rt = routing(T, E, k, 3)
    x, z = randn(1, T, d), randn(2, T * k, d)
    bad = [lambda: swg.permute(x[:3], rt), lambda: swg.permute(x.t(), rt),
           lambda: swg.permute(x, rt, out=x), lambda: swg.permute(swg.Fp8Rows(x.to(torch.uint8), x[0].float()), rt),
           lambda: swg.unpermute(x, rt), lambda: swg.unpermute(z, rt, residual=z),
           lambda: swg.unpermute(z, rt._replace(weights=None)),
           lambda: swg.unpermute(z, rt._replace(weights=rt.weights[:2])),
           lambda: swg.unpermute(z, rt._replace(position=rt.position.cpu())),
           lambda: swg.unpermute(z, rt._replace(position=rt.position.reshape(-1))),
           lambda: swg.unpermute_backward(x, z[:5], rt),
           lambda: swg.unpermute_backward(x, z, rt._replace(weights=None)),
           lambda: swg.permute(x, rt._replace(offsets=rt.offsets[:1]))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: swg.permute(x.half(), rt), lambda: swg.unpermute(z.half(), rt),
                 lambda: swg.permute(x, rt._replace(position=rt.position.long())),
                 lambda: swg.unpermute_backward(x, z.float(), rt),
                 lambda: swg.unpermute(z, rt, residual=x.float())):
        with pytest.raises(TypeError):
            call()
    y = torch.zeros(T * k, d, device=DEV, dtype=BF)
    with pytest.raises(swg.SwiGLUError):   # the result on top of an input
        swg.unpermute_backward(x, y, rt, out=y)
    swg.permute_backward(z, rt._replace(weights=None))   # (has no use for weights)


def test_streams_and_graphs(cuda_lib):
    T, E, k, d = 300, 16, 4, 520
    rt = routing(T, E, k, 3, 0.1)
    x, z = randn(1, T, d), randn(2, T * k, d)

    def calls(stream=None):
        return [swg.permute(x, rt, stream=stream), swg.unpermute(z, rt, residual=x, stream=stream),
                swg.permute_backward(z, rt, stream=stream),
                *swg.unpermute_backward(x, z, rt, stream=stream)]
    want = calls()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = calls(st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = calls()
    other = routing(T, E, k, 4, 0.3)   # another routing in the same tensors
    for a, b in zip(rt, other):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(calls(), got))


def test_offsets_past_32_bits(cuda_lib):
    T, E, k, d = 70001, 8, 2, 16384        # 2.29e9 elements in the sorted rows
    rt = routing(T, E, k, 6, 0.01)
    p = pairs(rt, E)
    n = p.numel()
    x = randn(1, T, 64).repeat(1, d // 64)
    out = swg.permute(x, rt)
    at = torch.cat([torch.arange(0, 50, device=DEV), torch.arange(n - 200, n, device=DEV)])
    assert torch.equal(out[at], x[p[at] // k]) and not bool(out[n:].any())
    t = torch.tensor([0, 1, T - 2, T - 1], device=DEV)
    y = swg.permute_backward(out, rt)
    assert torch.equal(y[t], (x[t].float() * (rt.ids[t] >= 0).sum(1, keepdim=True)).to(BF))
    dz, dw = swg.unpermute_backward(x, out, rt)
    f = p[at]
    ref = rt.weights.reshape(-1)[f, None].to(D) * x[f // k].to(D)
    assert bool(((dz[at].to(D) - ref).abs() <= ref.abs() * (2.0 ** -8 + U)).all())
    sq = x[f // k].to(D).square().sum(1)
    assert bool(((dw.reshape(-1)[f].to(D) - sq).abs() <= U * (d / 32 + 16) * sq).all())
