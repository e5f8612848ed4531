"""The general linear product y = act(x W + bias) + residual against its
definition in 64 bits.

Tolerance: the f32 sum of K products differs from the exact one by about
sqrt(K) 2^-24 sum |x w|; eight times that, through an activation whose slope
never exceeds 1.2, plus one rounding of the result: half an ulp is 2^-9 (bf16)
or 2^-24 (f32) of it, and the functions' own error is given as much again for
bf16 (2^-8 in all) and eight ulps for f32 (2^-20).
"""
import math

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64


def act64(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def make(M, K, N, layout, bias, residual, out_dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    w = (torch.randn(K, N, generator=g, device=DEV) * max(K, 1) ** -0.5).bfloat16()
    w = w if layout == "kn" else w.t().contiguous()
    b = torch.randn(N, generator=g, device=DEV).to(bias) if bias is not None else None
    r = torch.randn(M, N, generator=g, device=DEV).to(out_dtype) if residual else None
    return x, w, b, r


def check(y, x, w, b, r, act, layout):
    wk = (w if layout == "kn" else w.t()).to(D)
    v = x.to(D) @ wk
    s = x.to(D).abs() @ wk.abs()
    if b is not None:
        v = v + b.to(D)
        s = s + b.to(D).abs()
    ref = act64(act, v)
    if r is not None:
        ref = ref + r.to(D)
        s = s + r.to(D).abs()
    K = max(1, x.shape[1])
    tol = (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -20) * ref.abs() \
        + 1.2 * 8 * math.sqrt(K) * 2.0 ** -24 * s
    err = (y.to(D) - ref).abs()
    assert bool((err <= tol + 1e-37).all()), (err - tol).max().item()


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,K,N", [
    (1, 8, 8), (1, 64, 256), (1, 4096, 4096), (2, 72, 264), (7, 896, 4864), (8, 14336, 512),
    (31, 200, 40), (32, 128, 128), (33, 136, 520), (64, 1000, 1000), (127, 264, 72),
    (256, 512, 768), (257, 64, 64), (300, 4864, 896), (513, 192, 2056), (1111, 328, 136),
    (4099, 64, 8)])
def test_sizes(cuda_lib, M, K, N, layout):
    x, w, b, r = make(M, K, N, layout, torch.bfloat16, True, torch.bfloat16, seed=M + K)
    y = swg.linear(x, w, bias=b, residual=r, layout=layout)
    check(y, x, w, b, r, "none", layout)
    swg.check_device_status()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [(1, 2048, 64), (100, 2056, 64), (256, 4096, 128),
                                   (1025, 2040, 40), (700, 6000, 264)])
def test_few_outputs_of_long_sums(cuda_lib, M, K, N, out_dtype):
    # few units, cut along K in short shares; whole and ragged last blocks of K
    x, w, b, r = make(M, K, N, "nk", torch.float32, True, out_dtype, seed=K)
    for _ in range(2):
        y = swg.linear(x, w, bias=b, residual=r, activation="gelu", out_dtype=out_dtype,
                       layout="nk")
        check(y, x, w, b, r, "gelu", "nk")
    swg.check_device_status()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("bias,residual", [(None, False), (torch.float32, True),
                                           (torch.bfloat16, False)])
@pytest.mark.parametrize("M,K,N", [(3, 640, 264), (300, 264, 328)])
def test_epilogues(cuda_lib, M, K, N, act, bias, residual, out_dtype):
    x, w, b, r = make(M, K, N, "nk", bias, residual, out_dtype, seed=3)
    y = swg.linear(x, w, bias=b, residual=r, activation=act, out_dtype=out_dtype, layout="nk")
    assert y.dtype == out_dtype
    check(y, x, w, b, r, act, "nk")


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_large_arguments(cuda_lib, act):
    # sums far into the activations' tails: no NaN, the limits exactly
    x = torch.zeros(8, 8, device=DEV, dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([-3e4, -512.0, -90.0, -8.0, 8.0, 90.0, 512.0, 3e4], device=DEV)
    w = torch.zeros(8, 8, device=DEV, dtype=torch.bfloat16)
    w[0] = 1.0
    for out_dtype in (torch.bfloat16, torch.float32):
        y = swg.linear(x, w, activation=act, out_dtype=out_dtype)
        check(y, x, w, None, None, act, "kn")


def test_residual_in_place_and_out(cuda_lib):
    x, w, b, r = make(40, 256, 136, "kn", torch.float32, True, torch.bfloat16)
    want = swg.linear(x, w, bias=b, residual=r)
    got = r.clone()
    assert swg.linear(x, w, bias=b, residual=got, out=got) is got
    assert torch.equal(got, want)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [(1, 64, 1), (3, 4096, 60), (40, 72, 7), (300, 512, 130),
                                   (1000, 264, 257)])
def test_any_number_of_columns(cuda_lib, M, K, N, layout, out_dtype):
    x, w, b, r = make(M, K, N, layout, torch.float32, True, out_dtype)
    buf = torch.full((M * N + 64,), 7.0, device=DEV, dtype=out_dtype)
    out = buf[:M * N].view(M, N)
    swg.linear(x, w, bias=b, residual=r, activation="silu", out=out, layout=layout)
    check(out, x, w, b, r, "silu", layout)
    assert bool((buf[M * N:] == 7).all())


def test_nothing_to_sum(cuda_lib):
    x, w, b, r = make(5, 0, 16, "kn", torch.float32, True, torch.float32)
    y = swg.linear(x, w, bias=b, residual=r, activation="silu", out_dtype=torch.float32)
    check(y, x, w, b, r, "silu", "kn")
    assert swg.linear(torch.empty(0, 16, device=DEV, dtype=torch.bfloat16),
                      torch.empty(16, 8, device=DEV, dtype=torch.bfloat16)).shape == (0, 8)


def test_same_bits_every_time(cuda_lib):
    for M, K, N in [(8, 4096, 512), (700, 512, 640)]:
        x, w, b, r = make(M, K, N, "kn", torch.bfloat16, True, torch.bfloat16)
        first = swg.linear(x, w, bias=b, residual=r, activation="gelu")
        for _ in range(5):
            assert torch.equal(swg.linear(x, w, bias=b, residual=r, activation="gelu"), first)


def test_guard_bands(cuda_lib):
    # nothing is written outside y
    for M, N in [(5, 72), (33, 264)]:
        x, w, b, r = make(M, 200, N, "kn", torch.bfloat16, True, torch.bfloat16)
        buf = torch.full((M * N + 512,), 7.0, device=DEV, dtype=torch.bfloat16)
        out = buf[256:256 + M * N].view(M, N)
        swg.linear(x, w, bias=b, residual=r, out=out)
        check(out, x, w, b, r, "none", "kn")
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + M * N:] == 7).all())


def test_workspace_of_the_caller(cuda_lib):
    x, w, b, r = make(8, 4096, 512, "kn", torch.bfloat16, True, torch.bfloat16)
    n = swg.linear_workspace_bytes(8, 4096, 512)
    ws = torch.full((n,), 255, device=DEV, dtype=torch.uint8)
    want = swg.linear(x, w, bias=b, residual=r)
    assert torch.equal(swg.linear(x, w, bias=b, residual=r, workspace=ws), want)
    assert torch.equal(swg.linear(x, w, bias=b, residual=r, workspace=ws), want)
    with pytest.raises(swg.SwiGLUError) as e:
        swg.linear(x, w, workspace=ws[:n - 256])
    assert e.value.status == 8


def test_refusals(cuda_lib):
    x, w, b, r = make(4, 64, 32, "kn", torch.bfloat16, True, torch.bfloat16)
    with pytest.raises(ValueError):
        swg.linear(x.cpu(), w)
    with pytest.raises(ValueError):
        swg.linear(x.t(), w)
    with pytest.raises(TypeError):
        swg.linear(x.float(), w)
    with pytest.raises(ValueError):
        swg.linear(x, w, layout="nk")
    with pytest.raises(ValueError):
        swg.linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        swg.linear(x, w, bias=b[:8])
    with pytest.raises(TypeError):
        swg.linear(x, w, bias=b.half())
    with pytest.raises(ValueError):
        swg.linear(x, w, residual=r.float())
    with pytest.raises(ValueError):
        swg.linear(x, w, out=torch.empty(4, 24, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(swg.SwiGLUError) as e:     # K not a multiple of 8
        swg.linear(x[:, :12].contiguous(), w[:12].contiguous())
    assert e.value.status == 3
    base = torch.zeros(4 * 64 + 8, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(swg.SwiGLUError) as e:     # x off a 16-byte boundary
        swg.linear(base[1:1 + 256].view(4, 64), w)
    assert e.value.status == 3
    big = torch.zeros(4 * 64 + 4 * 32, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(swg.SwiGLUError) as e:     # y overlaps x
        swg.linear(big[:256].view(4, 64), w, out=big[192:320].view(4, 32))
    assert e.value.status == 1
