"""Argument checks of the norm and of rows sorted by expert that need no GPU:
invalid calls are refused before the device is looked at."""
import math

import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

A = 1 << 24   # a made-up, aligned address; nothing behind it is read


def norm(lib, x=A, r=None, w=2 * A, y=3 * A, s=None, M=4, d=64, eps=1e-6, dt=1, wt=1):
    return lib.swiglu_rms_norm(x, r, w, y, s, M, d, eps, dt, wt, None)


def norm8(lib, x=A, r=None, w=2 * A, y=3 * A, sc=4 * A, s=None, M=4, d=64, eps=1e-6, dt=1, wt=1):
    return lib.swiglu_rms_norm_fp8(x, r, w, y, sc, s, M, d, eps, dt, wt, None)


def back(lib, dy=A, s=2 * A, w=3 * A, ds=None, dx=4 * A, dw=5 * A, M=4, d=64, eps=1e-6, dt=1, wt=1,
         ws=None, nws=0):
    return lib.swiglu_rms_norm_backward(dy, s, w, ds, dx, dw, M, d, eps, dt, wt, ws, nws, None)


def permute(lib, x=A, sc=None, pos=2 * A, off=3 * A, out=4 * A, osc=None, T=4, k=2, E=8, d=64, dt=1):
    return lib.swiglu_permute(x, sc, pos, off, out, osc, T, k, E, d, dt, None)


def unpermute(lib, z=A, pos=2 * A, w=3 * A, r=None, y=4 * A, T=4, k=2, d=64, dt=1):
    return lib.swiglu_unpermute(z, pos, w, r, y, T, k, d, dt, None)


def unback(lib, dy=A, z=2 * A, pos=3 * A, off=4 * A, w=5 * A, dz=6 * A, dw=7 * A, T=4, k=2, E=8, d=64,
           dt=1):
    return lib.swiglu_unpermute_backward(dy, z, pos, off, w, dz, dw, T, k, E, d, dt, None)


def up_rows(lib, x=A, sx=2 * A, g=3 * A, u=4 * A, sg=5 * A, su=6 * A, h=7 * A, M=4, d=64, f=72, path=0):
    return lib.swiglu_up_fp8_rows(x, sx, g, u, sg, su, h, M, d, f, path, None, 0, None)


INVALID, UNSUPPORTED, ALIGN = 1, 2, 3


@pytest.mark.parametrize("fn,kw,status", [
    (norm, dict(M=-1), INVALID), (norm, dict(d=-1), INVALID), (norm, dict(x=None), INVALID),
    (norm, dict(w=None), INVALID), (norm, dict(y=None), INVALID), (norm, dict(dt=2), INVALID),
    (norm, dict(wt=2), INVALID), (norm, dict(eps=0.0), INVALID), (norm, dict(eps=-1.0), INVALID),
    (norm, dict(eps=math.nan), INVALID), (norm, dict(eps=math.inf), INVALID),
    (norm, dict(eps=1e-60), INVALID), (norm, dict(d=32769), UNSUPPORTED),
    (norm, dict(d=32761), UNSUPPORTED),
    (norm, dict(M=(1 << 30) + 1), UNSUPPORTED), (norm, dict(x=A + 8), ALIGN),
    (norm, dict(w=2 * A + 2), ALIGN), (norm, dict(y=3 * A + 4), ALIGN),
    (norm, dict(r=5 * A), INVALID), (norm, dict(s=5 * A), INVALID),
    (norm, dict(y=A + 16), INVALID), (norm, dict(y=2 * A), INVALID),
    (norm, dict(r=5 * A, s=3 * A), INVALID), (norm, dict(r=5 * A, s=5 * A + 16), INVALID),
    (norm, dict(r=5 * A, s=A + 16), INVALID), (norm, dict(r=5 * A, s=2 * A), INVALID),
    (norm8, dict(sc=None), INVALID), (norm8, dict(y=A), INVALID), (norm8, dict(sc=A), INVALID),
    (norm8, dict(sc=3 * A), INVALID), (norm8, dict(sc=4 * A + 2), ALIGN),
    (norm8, dict(r=5 * A, s=3 * A), INVALID), (norm8, dict(r=5 * A, s=4 * A), INVALID),
    (back, dict(dy=None), INVALID), (back, dict(s=None), INVALID), (back, dict(dx=None), INVALID),
    (back, dict(dw=None), INVALID), (back, dict(dx=A + 16), INVALID), (back, dict(dx=3 * A), INVALID),
    (back, dict(dw=A), INVALID), (back, dict(dw=4 * A), INVALID), (back, dict(dw=3 * A), INVALID),
    (back, dict(ds=6 * A + 8), ALIGN), (back, dict(eps=0.0), INVALID), (back, dict(d=40000), UNSUPPORTED),
    (back, dict(ws=4 * A, nws=1 << 20), INVALID),
    (permute, dict(T=-1), INVALID), (permute, dict(k=33), UNSUPPORTED), (permute, dict(E=0), INVALID),
    (permute, dict(E=1025), UNSUPPORTED), (permute, dict(dt=3), INVALID),
    (permute, dict(T=1 << 29, k=4), UNSUPPORTED), (permute, dict(x=None), INVALID),
    (permute, dict(off=None), INVALID), (permute, dict(out=A), INVALID),
    (permute, dict(out=2 * A), INVALID), (permute, dict(sc=5 * A), INVALID),
    (permute, dict(osc=5 * A), INVALID), (permute, dict(dt=2), INVALID),
    (permute, dict(dt=2, sc=5 * A), INVALID), (permute, dict(dt=2, sc=5 * A, osc=4 * A), INVALID),
    (permute, dict(dt=2, sc=5 * A, osc=5 * A), INVALID), (permute, dict(x=A + 2), ALIGN),
    (permute, dict(pos=2 * A + 2), ALIGN), (permute, dict(d=(1 << 28) + 1), UNSUPPORTED),
    (unpermute, dict(z=None), INVALID), (unpermute, dict(pos=None), INVALID),
    (unpermute, dict(y=None), INVALID), (unpermute, dict(y=A), INVALID),
    (unpermute, dict(r=4 * A + 16), INVALID), (unpermute, dict(dt=2), INVALID),
    (unpermute, dict(w=4 * A), INVALID), (unpermute, dict(w=3 * A + 1), ALIGN),
    (unpermute, dict(d=-8), INVALID),
    (unback, dict(w=None), INVALID), (unback, dict(dz=2 * A), INVALID), (unback, dict(dz=A), INVALID),
    (unback, dict(dw=5 * A), INVALID), (unback, dict(dw=6 * A), INVALID), (unback, dict(dt=2), INVALID),
    (unback, dict(E=0), INVALID), (unback, dict(off=None), INVALID),
    (up_rows, dict(sx=None), INVALID), (up_rows, dict(sx=2 * A + 2), ALIGN),
    (up_rows, dict(d=72), ALIGN), (up_rows, dict(h=2 * A), INVALID), (up_rows, dict(h=A), INVALID),
    (up_rows, dict(x=None), INVALID),
])
def test_refused(cuda_lib, fn, kw, status):
    assert fn(cuda_lib, **kw) == status
    assert cuda_lib.swiglu_last_error_string()


@pytest.mark.parametrize("at", [A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A])
def test_quantized_rows_refuse_an_input_in_the_workspace(cuda_lib, at):
    """At the start of the workspace, where swiglu_up_fp8 leaves codes, and at its end."""
    for ws, nws in ((at, 1 << 20), (at - (1 << 20), (1 << 20) + 1)):
        assert cuda_lib.swiglu_up_fp8_rows(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, 4, 64, 72, 0, ws, nws,
                                           None) == INVALID
        assert b"workspace" in cuda_lib.swiglu_last_error_string()


@pytest.mark.parametrize("at", [A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A])
def test_gradient_of_the_norm_refuses_a_tensor_in_the_workspace(cuda_lib, at):
    for ws, nws in ((at, 1 << 20), (at - (1 << 20), (1 << 20) + 1)):
        assert back(cuda_lib, ds=6 * A, ws=ws, nws=nws) == INVALID
        assert b"workspace" in cuda_lib.swiglu_last_error_string()


def test_workspace_query_refuses_invalid_sizes(cuda_lib):
    assert cuda_lib.swiglu_rms_norm_backward_workspace_bytes(-1, 64, 1) == 0
    assert cuda_lib.swiglu_rms_norm_backward_workspace_bytes(4, 64, 2) == 0
    assert cuda_lib.swiglu_rms_norm_backward_workspace_bytes(4, 1 << 20, 1) == 0


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    r = swg.Routing(ids, ids.float(), torch.zeros(5, dtype=torch.int32), ids.reshape(-1), ids)
    for call in (lambda: swg.rms_norm(x, w), lambda: swg.rms_norm_fp8(x, w),
                 lambda: swg.rms_norm_backward(x, x, w), lambda: swg.permute(x, r),
                 lambda: swg.unpermute(x, r), lambda: swg.permute_backward(x, r),
                 lambda: swg.unpermute_backward(x, x, r),
                 lambda: swg.permute(swg.Fp8Rows(x.to(torch.uint8), w), r)):
        with pytest.raises(ValueError):
            call()
