"""Calls with a stream of their own (``stream=``): every tensor that a call
allocates belongs to that stream's allocator, so that neither earlier nor later
work of torch's current stream shares its memory while the kernels use it.
"""
import pytest
import torch

from swiglu_mlp_projection_gb300 import _lib, moe

BF = torch.bfloat16


class _Stream:
    cuda_stream = 7


class _Cuda:
    def __init__(self):
        self.now = None            # the stream that torch.cuda.stream has made current

    def stream(self, s):
        cuda = self

        class Context:
            def __enter__(self):
                cuda.before, cuda.now = cuda.now, s

            def __exit__(self, *exc):
                cuda.now = cuda.before
        return Context()

    def current_stream(self, device=None):
        return self.now


class _Tensor(torch.Tensor):
    """Notes the streams that its memory is kept from."""

    def record_stream(self, s):
        self.kept_from = getattr(self, "kept_from", []) + [s]


class _Torch:
    """torch, with allocations recorded as (tensor, current stream)."""

    def __init__(self):
        self.cuda, self.made = _Cuda(), []

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *a, **kw):
        t = torch.empty(*a, **kw).as_subclass(_Tensor)
        self.made.append((t, self.cuda.now))
        return t


@pytest.fixture
def fake(monkeypatch):
    class Library:
        def __getattr__(self, name):
            return name
    f = _Torch()
    f.streams = []
    monkeypatch.setattr(_lib, "load", lambda: Library())
    monkeypatch.setattr(moe, "_torch", lambda: f)
    monkeypatch.setattr(moe, "_call", lambda index, fn, *args: f.streams.append(args[-1]))
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 1)
    monkeypatch.setattr(moe, "_first", lambda t, name, dtype=None: 0)
    monkeypatch.setattr(moe, "_check", lambda t, name, index, dtype=None: t.data_ptr())
    return f


def run(stream):
    T, E, k, d, f = 3, 4, 2, 8, 16
    x = torch.zeros(T, d, dtype=BF)
    w = torch.zeros(E, d, f, dtype=BF)
    moe.swiglu_moe(x, torch.zeros(d, E, dtype=BF), w, w, torch.zeros(E, f, d, dtype=BF), k,
                   stream=stream)
    moe.dispatch(torch.zeros(T, k, dtype=torch.int32), E, stream=stream)


def test_allocations_belong_to_the_stream(fake):
    s = _Stream()
    run(s)
    assert fake.streams == [7] * 5
    assert len(fake.made) == 11            # logits, the routing's five, h, y; dispatch's three
    for t, stream in fake.made:
        assert stream is s
        assert t.kept_from == [None]       # ... and not reused before the current stream is past
    assert fake.cuda.now is None


def test_no_stream_uses_the_current_one(fake):
    run(None)
    assert fake.streams == [1] * 5
    assert all(stream is None and not hasattr(t, "kept_from") for t, stream in fake.made)


@pytest.mark.gpu
def test_temporaries_survive_the_current_stream(cuda_lib):
    # The side stream is held back; meanwhile the current stream allocates and
    # fills memory of every size that the call used.
    import swiglu_mlp_projection_gb300 as swg
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(0)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=dev) * 0.1).to(BF)
    T, E, k, d, f = 300, 8, 2, 256, 520
    x, wr = normal(T, d), normal(d, E)
    wg, wu, wd = normal(E, d, f), normal(E, d, f), normal(E, f, d)
    want, rw = swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):          # its workspace and code are there
        swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x)
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y, r = swg.swiglu_moe(x, wr, wg, wu, wd, k, residual=x, stream=side)
        junk = [torch.full(shape, float("nan"), device=dev, dtype=dt)
                for shape, dt in (((T * k, f), BF), ((T, E), torch.float32), ((T, d), BF)) * 4]
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(r.ids, rw.ids)
        assert torch.equal(r.position, rw.position)
        del junk, y, r
    swg.check_device_status()


@pytest.mark.gpu
def test_results_in_a_graph_on_a_forked_stream(cuda_lib):
    import swiglu_mlp_projection_gb300 as swg
    dev = torch.device("cuda", 0)
    T, E, k, d, f = 40, 8, 2, 256, 264
    g = torch.Generator(device=dev).manual_seed(1)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=dev) * 0.1).to(BF)
    x, wr = normal(T, d), normal(d, E)
    wg, wu, wd = normal(E, d, f), normal(E, d, f), normal(E, f, d)
    want = swg.swiglu_moe(x, wr, wg, wu, wd, k)[0]
    side = torch.cuda.Stream(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream(dev))
        y, _ = swg.swiglu_moe(x, wr, wg, wu, wd, k, stream=side)
        torch.cuda.current_stream(dev).wait_stream(side)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    swg.check_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["up", "packed", "down", "mlp", "fp8", "quantize"])
def test_dense_results_are_not_the_current_streams_memory(cuda_lib, op):
    # The current stream is held back before its last write to tensors that are
    # then dropped: a call on another stream does not get their memory.
    import swiglu_mlp_projection_gb300 as swg
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(2)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=dev) * 0.1).to(BF)
    M, d, f = 40, 256, 520
    x, wg, wu, wd = normal(M, d), normal(d, f), normal(d, f), normal(f, d)
    h = normal(M, f)
    wp = swg.pack_weights(wg, wu)
    w8 = swg.quantize_weights_fp8(wg, wu)
    call = {"up": lambda s: (swg.swiglu_up(x, wg, wu, stream=s),),
            "packed": lambda s: (swg.swiglu_up_packed(x, wp, f, stream=s),),
            "down": lambda s: (swg.swiglu_down(h, wd, residual=x, stream=s),),
            "mlp": lambda s: swg.swiglu_mlp(x, wg, wu, wd, stream=s),
            "fp8": lambda s: (swg.swiglu_up_fp8(x, w8, stream=s),),
            "quantize": lambda s: tuple(vars(swg.quantize_weights_fp8(wg, wu, stream=s))[n]
                                        for n in ("w8_gate", "w8_up", "s_gate", "s_up"))}[op]
    side = torch.cuda.Stream(dev)
    want = call(None)
    call(side)
    torch.cuda.synchronize()
    busy = [torch.empty_like(t) for t in want for _ in range(3)]
    torch.cuda._sleep(20_000_000)
    for t in busy:
        t.fill_(77)
    del busy, t
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    swg.check_device_status()
