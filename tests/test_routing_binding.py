"""What the mixture-of-experts binding hands to the library: the addresses of
the tensors that the caller's Routing holds now.  The library's calls are
recorded, not made, so that this needs no GPU."""
import copy
import pickle

import pytest
import torch

from swiglu_mlp_projection_gb300 import _lib, moe

BF = torch.bfloat16
T, E, K, D, F = 3, 4, 2, 8, 16


class _Lib:
    """Stands for the library: every entry point is its own name."""

    def __getattr__(self, name):
        return name


@pytest.fixture
def calls(monkeypatch):
    """The library calls as (entry point, arguments); CPU tensors pass as device tensors."""
    made = []
    monkeypatch.setattr(_lib, "load", lambda: _Lib())
    monkeypatch.setattr(moe, "_call", lambda index, fn, *args: made.append((fn, args)))
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(moe, "_first", lambda t, name, dtype=None: 0)
    monkeypatch.setattr(moe, "_check", lambda t, name, index, dtype=None: t.data_ptr())
    return made


def made_routing():
    i32 = torch.int32
    return moe.Routing(torch.zeros(T, K, dtype=i32), torch.rand(T, K),
                       torch.zeros(E + 1, dtype=i32), torch.zeros(T * K, dtype=i32),
                       torch.zeros(T, K, dtype=i32))


def use(calls, r):
    """The addresses of offsets and order, and of offsets, position and weights, that an up
    and a down projection through `r` pass on."""
    del calls[:]
    w = torch.zeros(E, D, F, dtype=BF)
    h = moe.experts_up(torch.zeros(T, D, dtype=BF), w, w, r)
    moe.experts_down(h, torch.zeros(E, F, D, dtype=BF), r)
    (up, a), (down, b) = calls
    assert up == "swiglu_experts_up" and down == "swiglu_experts_down"
    return a[3:5], b[2:5]


def check(calls, r):
    up, down = use(calls, r)
    assert up == (r.offsets.data_ptr(), r.order.data_ptr())
    assert down == (r.offsets.data_ptr(), r.position.data_ptr(), r.weights.data_ptr())


def routings(calls):
    r = made_routing()
    use(calls, r)                                  # (used once: whatever that leaves behind)
    return r, moe.route(torch.zeros(T, E), K)      # ... and one that route made


def test_copies_use_their_own_tensors(calls):
    for r in routings(calls):
        for c in (copy.deepcopy(r), pickle.loads(pickle.dumps(r)), copy.copy(r),
                  r._replace(weights=r.weights.clone()), moe.Routing(*(t.clone() for t in r))):
            check(calls, c)


def test_exchanged_storage_is_seen(calls):
    for r in routings(calls):
        r.weights.data = torch.rand(T, K)
        check(calls, r)
        r.offsets.set_(torch.zeros(E + 1, dtype=torch.int32))
        check(calls, r)


def test_changed_shapes_are_refused(calls):
    for r in routings(calls):
        r.order.resize_(T * K - 1)
        with pytest.raises(ValueError):
            use(calls, r)
    for r in routings(calls):
        r.offsets.resize_(E)
        with pytest.raises(ValueError):
            use(calls, r)


@pytest.mark.gpu
def test_copies_outlive_the_original(cuda_lib):
    import swiglu_mlp_projection_gb300 as swg
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(BF)
    t, e, k, d, f = 50, 8, 2, 64, 72
    x, wg, wu, wd = normal(t, d), normal(e, d, f), normal(e, d, f), normal(e, f, d)
    r = swg.route(torch.randn(t, e, generator=g, device=dev), k)
    h = swg.experts_up(x, wg, wu, r)
    y = swg.experts_down(h, wd, r)
    copies = [copy.deepcopy(r), pickle.loads(pickle.dumps(r))]
    shapes = [(a.shape, a.dtype) for a in r]
    del r
    # the freed tensors' memory holds other values now
    other = [[torch.full(s, 1, dtype=dt, device=dev) for s, dt in shapes] for _ in range(4)]
    for c in copies:
        assert torch.equal(swg.experts_up(x, wg, wu, c), h)
        assert torch.equal(swg.experts_down(h, wd, c), y)
    del other
