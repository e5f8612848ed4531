"""Waits that run out in the kernels themselves: with a limit of 1 ms, a call
whose units of work sum over a million products gives up waiting for them.  The
call has to end, report a timeout, and leave the next calls right.  (The limit
is read once per process, so the calls run in one of their own.)"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
import swiglu_mlp_projection_gb300 as swg
dev, bf = torch.device("cuda", 0), torch.bfloat16
op = sys.argv[1]

def ones(*shape):
    return torch.ones(*shape, device=dev, dtype=bf)

def call(rows, K):
    if op == "linear":
        return swg.linear(ones(rows, K), ones(K, 256))
    if op == "tile":
        w = ones(K, 128)
        return swg.swiglu_up(ones(rows, K), w, w, path="tc")
    if op in ("cluster", "stream"):      # 1 row; 6250 k blocks per CTA
        n = 64 if op == "cluster" or K < 1024 else 1856
        return swg.swiglu_up(ones(1, K), ones(K, n), ones(K, n), path="skinny")
    if op == "tile_down":
        return swg.swiglu_down(ones(rows, K), ones(K, 256), path="tc")
    rt = swg.dispatch(torch.zeros(rows, 1, device=dev, dtype=torch.int32), 1,
                      torch.ones(rows, 1, device=dev))
    if op == "up":
        w = ones(1, K, 128)
        return swg.experts_up(ones(rows, K), w, w, rt)
    return swg.experts_down(ones(rows, K), ones(1, K, 256), rt)

small = call(256, 64)            # code and workspace are there; its waits are short
swg.check_device_status()
for _ in range(2):
    call(256, 1 << 21)
    try:
        swg.check_device_status()
        print("no timeout")
    except swg.SwiGLUError as e:
        print("status", e.status)
    same = torch.equal(call(256, 64), small)
    swg.check_device_status()
    print("same", same)
"""


@pytest.mark.parametrize("op", ["linear", "up", "down", "tile", "tile_down", "cluster",
                                "stream"])
def test_given_up_waits_end_the_call(cuda_lib, op):
    env = dict(os.environ, SWIGLU_WAIT_TIMEOUT_MS="1", SWIGLU_GR_CUT="0", SWIGLU_TILE_SK="0",
               SWIGLU_SK_CLUSTER="2" if op == "cluster" else "0")
    r = subprocess.run([sys.executable, "-c", CHILD, op], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:4] == ["status 6", "same True"] * 2, r.stdout
