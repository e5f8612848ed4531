"""Argument checks of the mixture-of-experts entry points that need no GPU:
invalid calls are refused before the device is looked at."""
import ctypes

import pytest

A = 1 << 20   # a made-up, aligned address; nothing behind it is read


def linear(lib, x=A, w=2 * A, bias=None, resid=None, y=3 * A, M=4, K=64, N=32, act=0, bd=1, od=1,
           layout=0):
    return lib.swiglu_linear(x, w, bias, resid, y, M, K, N, act, bd, od, layout, None, 0, None)


def route(lib, logits=A, bias=None, ids=2 * A, w=3 * A, off=4 * A, order=5 * A, pos=6 * A, T=4, E=16,
          k=2, dt=0, score=0, groups=1, tg=1, gs=0):
    return lib.swiglu_route(logits, bias, ids, w, off, order, pos, T, E, k, dt, score, groups, tg,
                            gs, 1, 1.0, None)


def up(lib, x=A, g=2 * A, u=3 * A, off=4 * A, order=5 * A, h=6 * A, T=4, k=2, E=4, d=64, f=72,
       layout=0):
    return lib.swiglu_experts_up(x, g, u, off, order, h, T, k, E, d, f, layout, None, 0, None)


def down(lib, h=A, w=2 * A, off=3 * A, pos=4 * A, wt=5 * A, r=None, y=6 * A, T=4, k=2, E=4, f=72,
         d=64, layout=0):
    return lib.swiglu_experts_down(h, w, off, pos, wt, r, y, T, k, E, f, d, layout, None, 0, None)


INVALID, UNSUPPORTED, ALIGN = 1, 2, 3


@pytest.mark.parametrize("fn,kw,status", [
    (linear, dict(M=-1), INVALID), (linear, dict(x=None), INVALID), (linear, dict(y=None), INVALID),
    (linear, dict(act=5), INVALID), (linear, dict(act=-1), INVALID), (linear, dict(od=2), INVALID),
    (linear, dict(bd=7), INVALID), (linear, dict(layout=2), INVALID), (linear, dict(K=12), ALIGN),
    (linear, dict(x=A + 8), ALIGN), (linear, dict(bias=A + 1), ALIGN),
    (linear, dict(M=(1 << 30) + 1), UNSUPPORTED), (linear, dict(K=1 << 24, N=1 << 24), UNSUPPORTED),
    (linear, dict(y=A + 128), INVALID), (linear, dict(y=2 * A), INVALID),
    (linear, dict(resid=3 * A + 16), INVALID),
    (route, dict(T=-1), INVALID), (route, dict(E=0, k=0), INVALID), (route, dict(k=17), INVALID),
    (route, dict(E=1025), UNSUPPORTED), (route, dict(E=64, k=33), UNSUPPORTED),
    (route, dict(dt=3), INVALID), (route, dict(score=2), INVALID), (route, dict(gs=2), INVALID),
    (route, dict(groups=3), INVALID), (route, dict(groups=0), INVALID),
    (route, dict(groups=4, tg=5), INVALID), (route, dict(E=128, groups=64), UNSUPPORTED),
    (route, dict(order=None), INVALID), (route, dict(ids=A), INVALID),
    (route, dict(w=2 * A + 4), INVALID), (route, dict(off=4 * A + 2), ALIGN),
    (up, dict(k=5), INVALID), (up, dict(E=2000), UNSUPPORTED), (up, dict(d=60), ALIGN),
    (up, dict(f=12), ALIGN), (up, dict(u=None), INVALID), (up, dict(order=None), INVALID),
    (up, dict(h=A), INVALID), (up, dict(layout=-1), INVALID), (up, dict(g=2 * A + 8), ALIGN),
    (up, dict(T=1 << 29, k=4), UNSUPPORTED),
    (down, dict(wt=None), INVALID), (down, dict(pos=None), INVALID), (down, dict(y=A), INVALID),
    (down, dict(r=6 * A + 16), INVALID), (down, dict(d=12), ALIGN), (down, dict(layout=3), INVALID),
])
def test_refused(cuda_lib, fn, kw, status):
    assert fn(cuda_lib, **kw) == status
    assert cuda_lib.swiglu_last_error_string()


def test_dispatch_refused(cuda_lib):
    f = cuda_lib.swiglu_dispatch
    assert f(None, A, 2 * A, 3 * A, 4, 2, 8, None) == INVALID
    assert f(A, A, 2 * A, 3 * A, 4, 2, 8, None) == INVALID
    assert f(A, 4 * A, 2 * A, 2 * A, 4, 2, 8, None) == INVALID
    assert f(A, 4 * A, 2 * A, 3 * A, 4, 9, 8, None) == INVALID
    assert f(A, 4 * A + 2, 2 * A, 3 * A, 4, 2, 8, None) == ALIGN


def test_workspace_queries_refuse_invalid_sizes(cuda_lib):
    assert cuda_lib.swiglu_linear_workspace_bytes(-1, 64, 64) == 0
    assert cuda_lib.swiglu_experts_up_workspace_bytes(4, 9, 8, 64, 64) == 0
    assert cuda_lib.swiglu_experts_down_workspace_bytes(4, 2, 8, 60, 64) == 0
    assert ctypes.c_char_p(cuda_lib.swiglu_last_error_string()).value
