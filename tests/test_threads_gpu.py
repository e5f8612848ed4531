"""Host threads that call on one stream: the kernels of a call hand partial
sums, counts and padded weights over in the stream's buffer, so the calls of
several threads have to enqueue one after another."""
import threading

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = torch.bfloat16


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(BF)


def jobs(seed):
    """Calls of several kernels each, at sizes of this seed; they return tensors."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = 40 * seed
    x, w = normal(g, 300 + n, 4864), normal(g, 4864, 896, scale=0.02)
    xp, wp = normal(g, 9 + seed, 512), normal(g, 512, 257 + seed, scale=0.05)
    logits = torch.randn(700 + 10 * n, 64, generator=g, device=DEV)
    ids = torch.randint(0, 60, (5000 + n, 8), generator=g, device=DEV, dtype=torch.int32)
    rt = swg.route(torch.randn(333 + n, 8, generator=g, device=DEV), 2)
    h = normal(g, 2 * (333 + n), 1024)
    wd = normal(g, 8, 1024, 264, scale=0.03)
    hd, wdd = normal(g, 16 + seed, 2048), normal(g, 2048, 1024, scale=0.02)
    return {
        "linear": lambda: [swg.linear(x, w)],                       # product, join
        "padded": lambda: [swg.linear(xp, wp, activation="silu")],  # copy, product
        "route": lambda: list(swg.route(logits, 6)),                # routing, places
        "dispatch": lambda: list(swg.dispatch(ids, 60))[2:],        # counts, places
        "down": lambda: [swg.experts_down(h, wd, rt)],              # product, weighted sum
        "dense": lambda: [swg.swiglu_down(hd, wdd)],                # product, sum
    }


@pytest.mark.parametrize("side", [False, True])
def test_two_threads_on_one_stream(cuda_lib, side):
    sets = [jobs(1), jobs(2)]
    want = [{n: f() for n, f in s.items()} for s in sets]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream(DEV) if side else torch.cuda.default_stream(DEV)
    swg.release_workspaces()          # the buffer grows while both threads use it
    start = threading.Barrier(len(sets))
    wrong = []

    def work(i):
        try:
            start.wait()
            with torch.cuda.stream(stream):
                for rep in range(60):
                    got = {n: f() for n, f in sets[i].items()}
                    for n, tensors in got.items():
                        same = [torch.equal(a, b) for a, b in zip(tensors, want[i][n])]
                        if not all(same):
                            wrong.append((i, rep, n))
        except Exception as e:        # shown by the main thread
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]
    swg.check_device_status()
