"""Routing and dispatch against a token-by-token definition.

Choices, offsets, order and positions have to be equal; the weights are within
2^-20 of the 64-bit ones (the exponential's few ulps, a sum of up to 1024 f32
terms in a tree, two divisions).  Biased candidates are kept at least 2^-18
apart, because a choice between values that differ by less than the scores'
rounding has more than one right answer.
"""
import math

import numpy as np
import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ref_route(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale):
    l = logits.double().cpu().numpy()
    l = np.where(l > -math.inf, l, -math.inf)
    T, E = l.shape
    size = E // groups
    b = None if bias is None else bias.double().cpu().numpy()
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    apart = np.ones(T, dtype=bool)
    for t in range(T):
        live = np.nonzero(l[t] > -math.inf)[0]
        if len(live) == 0:
            continue
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l[t]))
        else:
            m = l[t].max()
            s = np.where(l[t] == m, 1.0, np.exp(np.where(l[t] == m, 0.0, l[t] - m)))
            s = s / s.sum()
        key = l[t].copy() if b is None else s + b
        live = live[key[live] > -math.inf]
        if groups > 1:
            gk = np.full(groups, -math.inf)
            for g in range(groups):
                mem = live[live // size == g]
                if len(mem):
                    if group_score == "max":
                        gk[g] = key[mem].max()
                    else:
                        gk[g] = np.sort((s if b is None else key)[mem])[::-1][:2].sum()
            srt = np.sort(gk)[::-1]
            if (b is not None or group_score == "top2") and topk_groups < groups:
                gap = srt[topk_groups - 1] - srt[topk_groups]
                apart[t] &= not (gap < 2.0 ** -18)
            live = live[np.isin(live // size, np.argsort(-gk, kind="stable")[:topk_groups])]
        best = live[np.argsort(-key[live], kind="stable")][:k]
        if b is not None and len(live) > 1:
            top = np.sort(key[live])[::-1][:k + 1]
            apart[t] &= bool((top[:-1] - top[1:] >= 2.0 ** -18).all())
        ww = s[best]
        if renormalize and ww.sum() > 0:
            ww = ww / ww.sum()
        ids[t, :len(best)] = best
        w[t, :len(best)] = ww * scale
    return ids, w, apart


def ref_dispatch(ids, E):
    flat = ids.reshape(-1)
    lists = [np.nonzero(flat == e)[0] for e in range(E)]
    order = np.concatenate(lists) if lists else np.empty(0, dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(a) for a in lists])])
    position = np.full(flat.size, -1)
    position[order] = np.arange(len(order))
    order = np.concatenate([order, np.full(flat.size - len(order), -1)])
    return offsets, order, position.reshape(ids.shape)


def check_dispatch(r, E):
    o, order, pos = ref_dispatch(r.ids.cpu().numpy(), E)
    assert np.array_equal(r.offsets.cpu().numpy(), o)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), pos)


def check(logits, k, score="softmax", bias=None, groups=1, topk_groups=None, group_score="max",
          renormalize=True, scale=1.0):
    r = swg.route(logits, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups,
                  group_score=group_score, renormalize=renormalize, scale=scale)
    ids, w, apart = ref_route(logits, k, score, bias, groups, topk_groups or groups, group_score,
                              renormalize, scale)
    got = r.ids.cpu().numpy()
    assert np.array_equal(got[apart], ids[apart])
    assert apart.mean() > 0.5 or len(apart) < 4
    gw = r.weights.double().cpu().numpy()
    assert (np.abs(gw - w)[apart] <= 2.0 ** -20 * np.abs(w)[apart] + 1e-38).all()
    check_dispatch(r, logits.shape[1])
    return r


def randn(T, E, seed, dtype=torch.float32, scale=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(T, E, generator=g, device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (1, 64, 8), (3, 33, 32), (5, 60, 4),
                                   (17, 128, 8), (33, 160, 6), (64, 256, 8), (40, 500, 10),
                                   (9, 512, 32), (7, 1024, 16), (1000, 16, 1), (999, 7, 7)])
def test_plain(cuda_lib, T, E, k, score, dtype):
    # (bf16 logits tie often: ties go to the lowest index)
    for renormalize in (False, True):
        check(randn(T, E, T + E, dtype), k, score, renormalize=renormalize, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", [
    (1, 256, 8, 8, 4), (50, 64, 6, 4, 2), (33, 160, 6, 8, 3), (20, 32, 4, 32, 8),
    (20, 1024, 8, 32, 5), (30, 48, 8, 3, 1), (25, 24, 5, 1, 1)])
def test_groups_and_bias(cuda_lib, T, E, k, groups, topk_groups, bias, group_score, score):
    b = randn(1, E, 5, scale=0.2)[0].contiguous() if bias else None
    check(randn(T, E, E), k, score, b, groups, topk_groups, group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(256, 8), (512, 16), (1024, 32), (128, 5)])
def test_neighbours_chosen(cuda_lib, E, k, score):
    # all of a token's choices are neighbouring experts, in falling, rising and
    # equal order, at the start, at the end and across the middle
    l = randn(9, E, E, scale=0.1)
    fall = torch.linspace(6, 5, k, device=DEV)
    for row, at in ((0, 0), (3, E - k), (6, E // 2 - k // 2)):
        l[row, at:at + k] = fall
        l[row + 1, at:at + k] = fall.flip(0)
        l[row + 2, at:at + k] = 5.0
    check(l, k, score)
    check(l, k, score, torch.zeros(E, device=DEV))


def test_masks(cuda_lib):
    inf = math.inf
    l = randn(64, 40, 1)
    l[0] = -inf                      # nothing left
    l[1, 3:] = -inf                  # three left, four wanted
    l[2] = float("nan")              # NaN counts as masked
    l[3, ::2] = float("nan")
    l[4, 7] = inf                    # an infinite logit takes all the softmax
    l[5, 7] = l[5, 9] = inf
    l[6] = torch.finfo(torch.float32).min     # the type's lowest value is no mask
    l[7] = 0.0                       # every candidate equal
    l[8, :] = -0.0
    l[8, 20] = 0.0                   # -0 and 0 tie
    for score in ("softmax", "sigmoid"):
        for ren in (False, True):
            r = check(l, 4, score, renormalize=ren)
            assert r.ids[0].tolist() == [-1] * 4 and r.weights[0].tolist() == [0.0] * 4
            assert r.ids[1, 3].item() == -1
            assert r.ids[7].tolist() == [0, 1, 2, 3] and r.ids[8].tolist() == [0, 1, 2, 3]
            assert bool(torch.isfinite(r.weights).all())
    b = randn(1, 40, 3)[0].contiguous()
    b[5] = -inf
    b[6] = float("nan")
    r = check(l[9:].contiguous(), 4, "sigmoid", b)
    assert not bool(((r.ids == 5) | (r.ids == 6)).any())
    # a group without a candidate ranks last; a group of one live expert by it
    g = randn(8, 16, 4)
    g[:, 0:4] = -inf
    g[:, 5:8] = -inf
    for gs in ("max", "top2"):
        check(g, 4, "softmax", None, 4, 2, gs)
        check(g, 4, "sigmoid", torch.rand(16, device=DEV), 4, 3, gs)


@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (1, 8, 64), (100, 3, 5), (683, 3, 1024),
                                   (2049, 1, 7), (5000, 8, 60), (40000, 8, 256),
                                   (70000, 4, 1000)])
def test_dispatch(cuda_lib, T, k, E):
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device=DEV, dtype=torch.int32)
    r = swg.dispatch(ids, E)
    assert torch.equal(r.ids, ids)
    keep = ids.clone()
    keep[(ids < 0) | (ids >= E)] = -1
    check_dispatch(r._replace(ids=keep), E)


def test_dispatch_extremes(cuda_lib):
    for fill in (-1, 0, 6, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((3000, 2), fill, device=DEV, dtype=torch.int32)
        r = swg.dispatch(ids, 7)
        keep = ids if 0 <= fill < 7 else torch.full_like(ids, -1)
        check_dispatch(r._replace(ids=keep), 7)


def test_no_tokens(cuda_lib):
    r = swg.route(torch.empty(0, 8, device=DEV), 2)
    assert r.ids.shape == (0, 2) and r.offsets.tolist() == [0] * 9


def test_refusals(cuda_lib):
    l = randn(4, 16, 0)
    with pytest.raises(ValueError):
        swg.route(l.cpu(), 2)
    with pytest.raises(ValueError):
        swg.route(l.t(), 2)
    with pytest.raises(TypeError):
        swg.route(l.half(), 2)
    with pytest.raises(ValueError):
        swg.route(l, 2, score="tanh")
    with pytest.raises(ValueError):
        swg.route(l, 2, group_score="mean")
    with pytest.raises(ValueError):
        swg.route(l, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        swg.route(l, -1)
    for kw in (dict(k=17), dict(k=2, groups=3), dict(k=2, groups=4, topk_groups=5),
               dict(k=2, groups=4, topk_groups=0)):
        with pytest.raises(swg.SwiGLUError) as e:
            swg.route(l, **kw)
        assert e.value.status == 1
    for E, kw in ((2048, dict(k=2)), (64, dict(k=33)), (128, dict(k=2, groups=64))):
        with pytest.raises(swg.SwiGLUError) as e:
            swg.route(randn(2, E, 0), **kw)
        assert e.value.status == 2
    with pytest.raises(ValueError):
        swg.dispatch(torch.zeros(4, 2, device=DEV, dtype=torch.int64), 4)
