"""What surrounds the products in an MLP block (see ``include/swiglu.h`` for the
exact definitions): the root-mean-square norm with the residual's addition, in
the inputs' type (``rms_norm``) or as e4m3 rows with their scales
(``rms_norm_fp8``), its gradient (``rms_norm_backward``), and ``swiglu_block``,
which runs the norm and both projections.

As the rest of the binding, these only marshal torch tensors into the C ABI;
calls are asynchronous on torch's current stream (or ``stream``).  torch's
autograd does not see them: a gradient is a call of its own.
"""
from . import _lib
from . import Fp8Rows, Fp8Weights, _call, _empty, _raw_stream, _torch
from . import swiglu_down, swiglu_down_fp8, swiglu_up, swiglu_up_fp8
from .moe import _check, _first, _out, _row_code, _workspace


def _rows(torch, x, weight, x_name):
    """Checks of rows x [M, d] and weight [d]: (device, codes of their dtypes)."""
    index = _first(x, x_name)
    dt = _row_code(torch, x, x_name)
    if x.dim() != 2:
        raise ValueError("expected %s [M, d]" % x_name)
    _check(weight, "weight", index)
    wt = _row_code(torch, weight, "weight")
    if weight.dim() != 1 or weight.shape[0] != x.shape[1]:
        raise ValueError("weight must be [d] = [%d]" % x.shape[1])
    return index, dt, wt


def _like(t, name, x, index):
    """Address of a tensor of x's shape and dtype."""
    p = _check(t, name, index, x.dtype)
    if t.shape != x.shape:
        raise ValueError("%s must be of shape %s" % (name, tuple(x.shape)))
    return p


def rms_norm(x, weight, residual=None, eps=1e-6, out=None, sum_out=None, stream=None):
    """y = s / sqrt(mean(s^2) + eps) * weight with s = x + residual.

    x and residual [M, d] are contiguous CUDA tensors of one dtype (bfloat16 or
    float32), weight [d] either; d up to 32768.  Returns y in x's dtype, or with
    a residual (y, s).  ``out`` takes y and ``sum_out`` s; each may be x or
    residual itself.
    """
    torch = _torch()
    index, dt, wt = _rows(torch, x, weight, "x")
    shape, dtype, dev = x.shape, x.dtype, x.device
    pr = ps = s = None
    if residual is not None:
        pr = _like(residual, "residual", x, index)
        s = _out(torch, sum_out, shape, dtype, index, dev, stream)
        ps = s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    y = _out(torch, out, shape, dtype, index, dev, stream)
    M, d = shape
    _call(index, _lib.load().swiglu_rms_norm, x.data_ptr(), pr, weight.data_ptr(), y.data_ptr(), ps,
          M, d, eps, dt, wt, stream.cuda_stream if stream is not None else _raw_stream(index))
    return y if residual is None else (y, s)


def rms_norm_fp8(x, weight, residual=None, eps=1e-6, out=None, sum_out=None, stream=None):
    """As ``rms_norm``, with y as an Fp8Rows: e4m3 codes [M, d] (uint8) and
    float32 scales [M], quantized per row from the float32 values, which
    ``swiglu_up_fp8`` and ``permute`` take as they are.  ``out``: an Fp8Rows."""
    torch = _torch()
    index, dt, wt = _rows(torch, x, weight, "x")
    shape, dev = x.shape, x.device
    M, d = shape
    pr = ps = s = None
    if residual is not None:
        pr = _like(residual, "residual", x, index)
        s = _out(torch, sum_out, shape, x.dtype, index, dev, stream)
        ps = s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    codes, scales = (None, None) if out is None else out
    codes = _out(torch, codes, shape, torch.uint8, index, dev, stream)
    scales = _out(torch, scales, (M,), torch.float32, index, dev, stream)
    _call(index, _lib.load().swiglu_rms_norm_fp8, x.data_ptr(), pr, weight.data_ptr(),
          codes.data_ptr(), scales.data_ptr(), ps, M, d, eps, dt, wt,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    y = Fp8Rows(codes, scales)
    return y if residual is None else (y, s)


def rms_norm_backward(dy, s, weight, ds=None, eps=1e-6, out=None, workspace=None, stream=None):
    """The gradients of ``rms_norm`` (or, with the quantization as the identity,
    of ``rms_norm_fp8``) at s, its sum (x where there was no residual).

    dy, s [M, d]: contiguous, of one dtype; ds: the gradient that reaches s past
    the norm, or None.  Returns (dx, dweight): dx [M, d], the gradient of x and
    of the residual (``out`` if given; it may be dy, s or ds), and dweight [d] of
    weight's dtype.
    """
    torch = _torch()
    index, dt, wt = _rows(torch, s, weight, "s")
    M, d = s.shape
    py = _like(dy, "dy", s, index)
    pd = None if ds is None else _like(ds, "ds", s, index)
    dx = _out(torch, out, s.shape, s.dtype, index, s.device, stream)
    dw = _empty(torch, (d,), weight.dtype, s.device, stream)
    ws, nws = _workspace(workspace, index)
    _call(index, _lib.load().swiglu_rms_norm_backward, py, s.data_ptr(), weight.data_ptr(),
          pd, dx.data_ptr(),
          dw.data_ptr(), M, d, eps, dt, wt, ws, nws,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return dx, dw


def rms_norm_backward_workspace_bytes(M, d, dtype="bf16"):
    """Workspace bytes ``rms_norm_backward`` needs on the current device."""
    n = int(_lib.load().swiglu_rms_norm_backward_workspace_bytes(
        M, d, _lib.BF16 if dtype in ("bf16", _lib.BF16) else _lib.F32))
    if n == 0 and M != 0 and d != 0:   # a call with rows needs some
        _lib.check(1)
    return n


def swiglu_block(x, norm_weight, up, down, residual=None, eps=1e-6, layout="kn", stream=None):
    """The MLP block of a pre-norm transformer layer: with s = x + residual (s = x
    without one), y = s + down(swiglu(up(rms_norm(s)))).

    x and residual [M, d] are bfloat16; up is (w_gate, w_up) and down w_down, as
    ``swiglu_up`` and ``swiglu_down`` take them (``layout``), or up is an
    Fp8Weights and down an Fp8Matrix: the norm then writes the e4m3 rows that
    the up projection reads.  Returns y [M, d].
    """
    if x.dtype is not _torch().bfloat16:
        raise TypeError("x must be bfloat16, got %s" % x.dtype)
    fp8 = isinstance(up, Fp8Weights)
    n = (rms_norm_fp8 if fp8 else rms_norm)(x, norm_weight, residual=residual, eps=eps,
                                            stream=stream)
    n, s = (n, x) if residual is None else n
    if fp8:
        h = swiglu_up_fp8(n, up, stream=stream)
        return swiglu_down_fp8(h, down, residual=s, stream=stream)
    w_gate, w_up = up
    h = swiglu_up(n, w_gate, w_up, stream=stream, layout=layout)
    return swiglu_down(h, down, residual=s, stream=stream, layout=layout)
