"""Grouped products whose last units are cut along K: shares joined by the last
pair of a unit (up; down to 32 rows), or by the weighted sum (down), compared
with their definitions, repeated, in memory that held other values, on two
streams, and with a routing that no call wrote.  That each size is cut comes
from the schedule itself, built for the host."""
import os
import shutil
import subprocess

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg
from tests.test_experts_gpu import check_down, check_up, gen, make_ids, weights

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_mlp_projection_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "grouped_plan.cuh"
// n_kb ncg chunks pairs min_kb -> the most shares of a cut unit (0: none is cut)
int main(int argc, char** v) {
  swg::Work w{};
  w.n_kb = atoi(v[1]);
  w.ncg = atoi(v[2]);
  w.min_kb = atoi(v[5]);
  w.cut = 1;
  const swg::Schedule s = swg::make_schedule(w, (uint32_t)atoi(v[3]), (uint32_t)atoi(v[4]));
  uint32_t most = 0;
  for (uint32_t u = s.whole; u < s.units; ++u) {
    const uint32_t n = swg::shares_of(w, s, u - s.whole).count;
    if (n > most) most = n;
  }
  printf("%u\n", most);
  return 0;
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    """shares(op, rt, E, K, N, n_max): the most shares of a unit of that call."""
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("schedule")
    (d / "s.cu").write_text(PROGRAM)
    r = subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-gencode",
                        "arch=compute_103a,code=sm_103a", str(d / "s.cu"), "-o", str(d / "s")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2

    def most(op, rt, E, K, N, n_max):
        rows = (rt.offsets[1:] - rt.offsets[:-1]).tolist()
        chunks = sum(-(-m // n_max) for m in rows)
        a = [-(-K // 64), -(-N // (128 if op == "up" else 256)), chunks, pairs, 16]
        r = subprocess.run([str(d / "s")] + [str(v) for v in a], capture_output=True, text=True)
        return int(r.stdout)
    return most


def longest_chunk(T, k, E, K, N):
    """n_max of a call, from the workspace of the up projection (whose only part
    that depends on it are four blocks of n_max x 128 f32 per pair)."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    counters = -(-pairs * 8 // 256) * 256
    return (swg.experts_up_workspace_bytes(T, k, E, K, N) - counters - 256) // (pairs * 2048)


# T, E, k, K, N, skew, dropped, n_max, fewest shares
UP = [(1, 8, 2, 4096, 264, 0, 0, 32, 4), (1, 1, 1, 14336, 264, 0, 0, 32, 14),
      (9, 4, 2, 4096, 264, 0, 0, 32, 4), (9, 2, 1, 14328, 40, 0, 0.2, 32, 14),
      (31, 2, 1, 8192, 136, 0, 0, 32, 8), (60, 4, 1, 4096, 264, 9.0, 0, 64, 4),
      (100, 8, 1, 4096, 264, 9.0, 0.1, 64, 4), (64, 3, 1, 14336, 72, 9.0, 0, 64, 14)]
DOWN = [(1, 8, 2, 4864, 264, 0, 0, 32, 5), (9, 4, 2, 9728, 520, 0, 0.2, 32, 7),
        (100, 2, 1, 4864, 264, 0, 0, 128, 5), (100, 2, 2, 9728, 136, 0, 0.1, 128, 10),
        (300, 4, 2, 14336, 72, 2.0, 0, 256, 12), (40, 1, 1, 14328, 40, 0, 0, 64, 14),
        (700, 2, 1, 4864, 264, 0, 0.05, 256, 5)]


def up_parts(T, E, k, K, N, skew, dropped, layout="kn"):
    ids, w = make_ids(T, E, k, T + N, skew, dropped)
    rt = swg.dispatch(ids, E, w)
    x = torch.randn(T, K, generator=gen(1), device=DEV).to(BF)
    return rt, x, weights(E, K, N, 2, layout), weights(E, K, N, 3, layout)


def down_parts(T, E, k, K, N, skew, dropped, layout="kn"):
    ids, w = make_ids(T, E, k, T + N, skew, dropped)
    rt = swg.dispatch(ids, E, w)
    h = torch.randn(T * k, K, generator=gen(1), device=DEV).to(BF)
    return rt, h, weights(E, K, N, 2, layout), torch.randn(T, N, generator=gen(4), device=DEV).to(BF)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("case", UP)
def test_up(cuda_lib, shares, case, layout):
    T, E, k, K, N, skew, dropped, n_max, fewest = case
    rt, x, wg, wu = up_parts(*case[:7], layout)
    assert longest_chunk(T, k, E, K, N) == n_max
    assert shares("up", rt, E, K, N, n_max) >= fewest
    if n_max == 64:
        assert (rt.offsets[1:] - rt.offsets[:-1]).max().item() > 32
    h = swg.experts_up(x, wg, wu, rt, layout=layout)
    check_up(h, x, wg, wu, rt, E, k, layout)
    for _ in range(10):
        assert torch.equal(swg.experts_up(x, wg, wu, rt, layout=layout), h)
    ws = torch.full((swg.experts_up_workspace_bytes(T, k, E, K, N),), 255, device=DEV,
                    dtype=torch.uint8)
    for _ in range(2):
        assert torch.equal(swg.experts_up(x, wg, wu, rt, layout=layout, workspace=ws), h)
    swg.check_device_status()


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("case", DOWN)
def test_down(cuda_lib, shares, case, layout):
    T, E, k, K, N, skew, dropped, n_max, fewest = case
    rt, h, wd, r = down_parts(*case[:7], layout)
    assert longest_chunk(T, k, E, K, N) == n_max
    assert shares("down", rt, E, K, N, n_max) >= fewest
    y = swg.experts_down(h, wd, rt, residual=r, layout=layout)
    check_down(y, h, wd, rt, E, layout, r)
    for _ in range(10):
        assert torch.equal(swg.experts_down(h, wd, rt, residual=r, layout=layout), y)
    ws = torch.full((swg.experts_down_workspace_bytes(T, k, E, K, N),), 255, device=DEV,
                    dtype=torch.uint8)
    for _ in range(2):
        assert torch.equal(swg.experts_down(h, wd, rt, residual=r, layout=layout, workspace=ws), y)
    swg.check_device_status()


def test_two_streams(cuda_lib):
    calls = []
    for case in (UP[1], UP[6]):
        calls.append((swg.experts_up, up_parts(*case[:7])))
    for case in (DOWN[1], DOWN[3]):
        calls.append((swg.experts_down, down_parts(*case[:7])))

    def run(fn, p):
        return fn(p[1], p[2], p[3], p[0]) if fn is swg.experts_up \
            else fn(p[1], p[2], p[0], residual=p[3])
    want = [run(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [[], []]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [run(*c) for c in calls]
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))
    swg.check_device_status()


def test_in_a_graph(cuda_lib):
    rt, h, wd, r = down_parts(*DOWN[3][:7])
    ru, x, wg, wu = up_parts(*UP[6][:7])
    y, hu = swg.experts_down(h, wd, rt, residual=r), swg.experts_up(x, wg, wu, ru)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [swg.experts_up(x, wg, wu, ru), swg.experts_down(h, wd, rt, residual=r),
               swg.experts_up(x, wg, wu, ru), swg.experts_down(h, wd, rt, residual=r)]
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], hu) and torch.equal(got[2], hu)
        assert torch.equal(got[1], y) and torch.equal(got[3], y)
    swg.check_device_status()


@pytest.mark.parametrize("bad", [[-5, 1000, 3, 2 ** 31 - 1, 2 ** 30], [7, 7, 2, 90, 5],
                                 [0, 200, 0, 200, 0], [100, 50, 20, 10, 0]])
def test_offsets_that_no_call_wrote(cuda_lib, bad):
    # positions and tokens inside the tensors, offsets that do not rise: wrong
    # rows, but none outside (the bands around the outputs keep their value)
    T, E, k = 100, 4, 2
    off = torch.tensor(bad, device=DEV, dtype=torch.int32)
    order = torch.randperm(T * k, generator=gen(0), device=DEV).int()
    pos = torch.randperm(T * k, generator=gen(1), device=DEV).int().view(T, k)
    rt = swg.Routing(pos, torch.rand(T, k, generator=gen(2), device=DEV), off, order, pos)

    def band(rows, cols):
        buf = torch.full((rows * cols + 1024,), 5.0, device=DEV, dtype=BF)
        return buf, buf[512:512 + rows * cols].view(rows, cols)

    def kept(buf):
        return bool((buf[:512] == 5).all()) and bool((buf[-512:] == 5).all())
    K, N = 4864, 136                       # n_max 128: the weighted sum joins
    buf, y = band(T, N)
    swg.experts_down(torch.randn(T * k, K, generator=gen(3), device=DEV).to(BF),
                     weights(E, K, N, 2, "kn"), rt, out=y)
    assert kept(buf)
    K, N = 4096, 136
    buf, h = band(T * k, N)
    x, w = torch.randn(T, K, generator=gen(4), device=DEV).to(BF), weights(E, K, N, 2, "kn")
    swg.experts_up(x, w, w, rt, out=h)
    assert kept(buf)
    T = 9                                  # n_max 32: the last pair joins
    small = swg.Routing(pos[:T].contiguous() % (T * k), rt.weights[:T].contiguous(),
                        off, order[:T * k].contiguous() % (T * k), pos[:T].contiguous() % (T * k))
    buf, h = band(T * k, N)
    swg.experts_up(x[:T].contiguous(), w, w, small, out=h)
    assert kept(buf)
    buf, y = band(T, N)
    swg.experts_down(torch.randn(T * k, K, generator=gen(5), device=DEV).to(BF), w, small, out=y)
    assert kept(buf)
    swg.check_device_status()


def test_whole_chain_without_tokens(cuda_lib):
    E, k, d, f = 8, 2, 64, 72
    x = torch.empty(0, d, device=DEV, dtype=BF)
    y, r = swg.swiglu_moe(x, weights(1, d, E, 0, "kn")[0], weights(E, d, f, 1, "kn"),
                          weights(E, d, f, 2, "kn"), weights(E, f, d, 3, "kn"), k, residual=x)
    assert y.shape == (0, d) and r.ids.shape == (0, k) and r.offsets.tolist() == [0] * (E + 1)
    swg.check_device_status()
