"""Activations where 1 + e^-z no longer fits binary32 although their values,
about v e^z, are still normal numbers.

Tolerance: the rounding of the result with the functions' own error (2^-8 of
it for bf16, whose exponential is off by 2^-16 at most down here; 2^-20 for
f32, as everywhere else), one quantum of a bf16 result below 2^-126 (2^-133),
and two quanta of a subnormal e^z (2^-149), which v multiplies.
"""
import math

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = torch.float64
BF = torch.bfloat16


def sigma(z):
    return torch.where(z < 0, torch.exp(z) / (1 + torch.exp(z)), 1 / (1 + torch.exp(-z)))


def ref(act, v):
    if act == "silu":
        return v * sigma(v)
    return v * sigma(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def close(y, want, v, out_dtype):
    rel, quantum = (2.0 ** -8, 2.0 ** -133) if out_dtype is BF else (2.0 ** -20, 2.0 ** -149)
    err = (y.to(D) - want).abs()
    tol = rel * want.abs() + quantum + 2 * v.abs() * 2.0 ** -149
    assert bool((err <= tol).all()), (v, y, want)


@pytest.mark.parametrize("out_dtype", [BF, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_tails(cuda_lib, act, out_dtype):
    if act == "silu":      # in halves, which bf16 holds, from -104 up through 0
        v = torch.arange(-208, 209, device=DEV, dtype=D) / 2
    else:                  # 2 z from -125 to 125
        v = torch.arange(-92, 93, device=DEV, dtype=D) / 8
    n = v.numel()
    x = torch.zeros(n, 8, device=DEV, dtype=BF)
    x[:, 0] = v.to(BF)
    assert torch.equal(x[:, 0].to(D), v)
    w = torch.zeros(8, 8, device=DEV, dtype=BF)
    w[0] = 1.0
    y = swg.linear(x, w, activation=act, out_dtype=out_dtype)
    if act == "gelu_tanh":   # (z itself is rounded to f32: 2^-22 of it moves e^z by |2 z| 2^-22)
        z = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        slack = (ref(act, v) * z.abs() * 2.0 ** -22).abs()
    else:
        slack = torch.zeros_like(v)
    want = ref(act, v)
    lo, hi = want - slack, want + slack
    nearest = torch.minimum(torch.maximum(y[:, 3].to(D), lo), hi)
    close(y[:, 3], nearest, v, out_dtype)
    assert bool((y == y[:, :1]).all())
    swg.check_device_status()


def test_gate_of_the_experts(cuda_lib):
    # gate sums from -104 to 104, up sums of 1
    v = torch.arange(-208, 209, device=DEV, dtype=D) / 2
    n = v.numel()
    x = torch.zeros(n, 8, device=DEV, dtype=BF)
    x[:, 0], x[:, 1] = v.to(BF), 1.0
    wg, wu = torch.zeros(1, 8, 8, device=DEV, dtype=BF), torch.zeros(1, 8, 8, device=DEV, dtype=BF)
    wg[0, 0], wu[0, 1] = 1.0, 1.0
    rt = swg.dispatch(torch.zeros(n, 1, device=DEV, dtype=torch.int32), 1)
    h = swg.experts_up(x, wg, wu, rt)
    close(h[:, 5], ref("silu", v), v, BF)
    swg.check_device_status()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu", "relu"])
def test_limits(cuda_lib, act):
    x = torch.zeros(4, 8, device=DEV, dtype=BF)
    x[:, 0] = torch.tensor([float("inf"), float("nan"), -3e38, 3e38], device=DEV)
    w = torch.zeros(8, 8, device=DEV, dtype=BF)
    w[0, :] = 1.0
    x[:2, 1:] = 0
    y = swg.linear(x, w, activation=act)
    assert bool((y[0] == float("inf")).all()) and bool(y[1].isnan().all())
    assert not bool(y[2].any()) and torch.equal(y[3], x[3, :1].expand(8))
