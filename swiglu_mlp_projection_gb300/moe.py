"""The mixture-of-experts MLP and the general linear product (see
``include/swiglu.h`` for the exact definitions): ``linear``, ``route``,
``dispatch``, ``experts_up``, ``experts_down``, and ``swiglu_moe``, which runs
them in turn; and rows sorted by expert and back (``permute``, ``unpermute``,
their gradients ``permute_backward``, ``unpermute_backward``) for experts of
another kind.

As the rest of the binding, these only marshal torch tensors into the C ABI;
calls are asynchronous on torch's current stream (or ``stream``).  What a call
with a ``stream`` allocates belongs to that stream, as under
``torch.cuda.stream(stream)``; its inputs have to be ready there.
"""
import collections

from . import _lib
from . import Fp8Rows, _call, _empty, _raw_stream, _torch

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
LAYOUTS = {"kn": 0, "nk": 1}


class Routing(collections.namedtuple("Routing", "ids weights offsets order position")):
    """Where each token goes: ids [T, k] int32 (-1: no expert), weights [T, k]
    float32, and the (token, choice) pairs sorted by expert: offsets [E + 1],
    order [T k], position [T, k], int32 (``route`` and ``dispatch`` write them)."""

    __slots__ = ()   # its tensors and nothing else: copies and pickles stand for themselves


def _code(table, value, what):
    code = table.get(value) if isinstance(value, str) else None
    if code is None:
        raise ValueError("%s must be one of %s" % (what, sorted(table)))
    return code


def _check(t, name, index, dtype=None):
    """A contiguous tensor on CUDA device `index` (of `dtype`); its address."""
    if t.get_device() != index:
        raise ValueError("%s must be a CUDA tensor on the first argument's device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _first(t, name, dtype=None):
    """The CUDA device of the first argument; checks it as the others."""
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    _check(t, name, index, dtype)
    return index


def _workspace(workspace, index):
    if workspace is None:
        return None, 0
    return _check(workspace, "workspace", index), workspace.numel() * workspace.element_size()


def _out(torch, out, shape, dtype, index, device, stream):
    if out is None:
        return _empty(torch, shape, dtype, device, stream)
    _check(out, "out", index)
    if out.shape != shape or out.dtype is not dtype:
        raise ValueError("out must be a contiguous %s tensor of %s" % (shape, dtype))
    return out


def linear(x, w, bias=None, residual=None, activation="none", out=None, out_dtype=None,
           workspace=None, stream=None, layout="kn"):
    """y = act(x @ w + bias) + residual.

    x [M, K] and w [K, N] (layout "kn") or [N, K] ("nk", torch.nn.Linear.weight)
    are contiguous bfloat16 CUDA tensors, K a multiple of 8; bias [N] is
    bfloat16 or float32; activation one of "none", "relu", "silu", "gelu" (error
    function), "gelu_tanh".  The result [M, N] is ``out_dtype`` (bfloat16, the
    default, or float32); residual has its type and may be ``out``.
    """
    torch = _torch()
    bf16 = torch.bfloat16
    index = _first(x, "x", bf16)
    pw = _check(w, "w", index, bf16)
    lay = _code(LAYOUTS, layout, "layout")
    act = _code(ACTIVATIONS, activation, "activation")
    if x.dim() != 2 or w.dim() != 2 or w.shape[lay] != x.shape[1]:
        raise ValueError("expected x [M, K] and w [K, N] (kn) or [N, K] (nk)")
    M, K = x.shape
    N = w.shape[1 - lay]
    if out_dtype is None:
        out_dtype = bf16 if out is None else out.dtype
    if out_dtype is not bf16 and out_dtype is not torch.float32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    pb, bias_code = None, _lib.BF16
    if bias is not None:
        pb = _check(bias, "bias", index)
        if bias.dim() != 1 or bias.shape[0] != N:
            raise ValueError("bias must be [N] = [%d]" % N)
        if bias.dtype is not bf16:
            bias_code = _lib.F32
            if bias.dtype is not torch.float32:
                raise TypeError("bias must be bfloat16 or float32")
    pr = None
    if residual is not None:
        pr = _check(residual, "residual", index)
        if residual.shape != (M, N) or residual.dtype is not out_dtype:
            raise ValueError("residual must be [M, N] of the result's dtype")
    out = _out(torch, out, (M, N), out_dtype, index, x.device, stream)
    ws, nws = _workspace(workspace, index)
    _call(index, _lib.load().swiglu_linear, x.data_ptr(), pw, pb, pr, out.data_ptr(), M, K, N, act,
          bias_code, _lib.BF16 if out_dtype is bf16 else _lib.F32, lay, ws, nws,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return out


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=None, group_score="max",
          renormalize=True, scale=1.0, stream=None):
    """Choose k of E experts for every token; returns a Routing.

    logits [T, E] (float32 or bfloat16), score "softmax" or "sigmoid", bias [E]
    float32 (a balance bias: it moves the choice, not the weights).  With
    ``groups`` > 1 only the experts of the ``topk_groups`` best groups are
    candidates (``group_score`` "max", or "top2" for the sum of a group's two
    best).  Ties go to the lowest index.  Experts whose logit is -inf or NaN are
    masked; missing choices are id -1 with weight 0.
    """
    torch = _torch()
    index = _first(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("expected logits [T, E]")
    f32 = torch.float32
    dt = _lib.F32
    if logits.dtype is not f32:
        dt = _lib.BF16
        if logits.dtype is not torch.bfloat16:
            raise TypeError("logits must be float32 or bfloat16, got %s" % logits.dtype)
    T, E = logits.shape
    pb = None
    if bias is not None:
        pb = _check(bias, "bias", index)
        if bias.dim() != 1 or bias.shape[0] != E or bias.dtype is not f32:
            raise ValueError("bias must be a float32 [E] = [%d] tensor" % E)
    sc = _code(SCORES, score, "score")
    gs = _code(GROUP_SCORES, group_score, "group_score")
    if k < 0:
        raise ValueError("k must not be negative")
    dev, i32 = logits.device, torch.int32
    ids = _empty(torch, (T, k), i32, dev, stream)
    weights = _empty(torch, (T, k), f32, dev, stream)
    offsets = _empty(torch, (E + 1,), i32, dev, stream)
    order = _empty(torch, (T * k,), i32, dev, stream)
    position = _empty(torch, (T, k), i32, dev, stream)
    _call(index, _lib.load().swiglu_route, logits.data_ptr(), pb, ids.data_ptr(),
          weights.data_ptr(), offsets.data_ptr(), order.data_ptr(), position.data_ptr(), T, E, k,
          dt, sc, groups, groups if topk_groups is None else topk_groups, gs,
          1 if renormalize else 0, scale,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return Routing(ids, weights, offsets, order, position)


def dispatch(ids, n_experts, weights=None, stream=None):
    """A Routing from chosen experts ids [T, k] (int32; values outside
    0 ... n_experts - 1 are dropped) and their weights [T, k] (float32)."""
    torch = _torch()
    index = _first(ids, "ids")
    if ids.dim() != 2 or ids.dtype is not torch.int32:
        raise ValueError("expected int32 ids [T, k]")
    T, k = ids.shape
    if weights is not None:
        _check(weights, "weights", index)
        if weights.shape != ids.shape or weights.dtype is not torch.float32:
            raise ValueError("weights must be float32 of ids' shape")
    if n_experts < 1:
        raise ValueError("n_experts must be positive")
    dev, i32 = ids.device, torch.int32
    offsets = _empty(torch, (n_experts + 1,), i32, dev, stream)
    order = _empty(torch, (T * k,), i32, dev, stream)
    position = _empty(torch, (T, k), i32, dev, stream)
    _call(index, _lib.load().swiglu_dispatch, ids.data_ptr(), offsets.data_ptr(), order.data_ptr(),
          position.data_ptr(), T, k, n_experts,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return Routing(ids, weights, offsets, order, position)


def _routing_of(r, E, index):
    """(T, k, address of offsets) of a routing over E experts on device `index`.
    Every call reads the tensors anew (and checks those that it uses): their
    storage and sizes can change between two calls."""
    shape = r.position.shape
    if len(shape) != 2 or r.offsets.dim() != 1:
        raise ValueError("expected position [T, k] and offsets [E + 1] in the routing")
    po = _check(r.offsets, "routing.offsets", index, _torch().int32)
    if r.offsets.numel() != E + 1:
        raise ValueError("the routing is of %d experts, not %d" % (r.offsets.numel() - 1, E))
    return shape[0], shape[1], po


def experts_up(x, w_gate, w_up, routing, out=None, layout="kn", workspace=None, stream=None):
    """h[r] = silu(x[t] @ w_gate[e]) * (x[t] @ w_up[e]) for every (token t,
    expert e) pair r of ``routing``, in its sorted order: h [T k, d_ff].

    x [T, d]; w_gate, w_up [E, d, d_ff] ("kn") or [E, d_ff, d] ("nk"); all
    contiguous bfloat16.  Rows of dropped choices (at the end) are zero.
    """
    torch = _torch()
    bf16 = torch.bfloat16
    index = _first(x, "x", bf16)
    pg = _check(w_gate, "w_gate", index, bf16)
    pu = _check(w_up, "w_up", index, bf16)
    lay = _code(LAYOUTS, layout, "layout")
    if x.dim() != 2 or w_gate.dim() != 3 or w_up.shape != w_gate.shape \
            or w_gate.shape[1 + lay] != x.shape[1]:
        raise ValueError("expected x [T, d] and w_gate, w_up [E, d, d_ff] or [E, d_ff, d]")
    T, d = x.shape
    E, d_ff = w_gate.shape[0], w_gate.shape[2 - lay]
    rT, k, po = _routing_of(routing, E, index)
    if rT != T:
        raise ValueError("the routing is of %d tokens, not %d" % (rT, T))
    order = routing.order
    pr = _check(order, "routing.order", index, torch.int32)
    if order.dim() != 1 or order.numel() != T * k:
        raise ValueError("expected order [T k] = [%d] in the routing" % (T * k))
    out = _out(torch, out, (T * k, d_ff), bf16, index, x.device, stream)
    ws, nws = _workspace(workspace, index)
    _call(index, _lib.load().swiglu_experts_up, x.data_ptr(), pg, pu, po, pr, out.data_ptr(), T, k,
          E, d, d_ff, lay, ws, nws,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return out


def experts_down(h, w_down, routing, residual=None, out=None, layout="kn", workspace=None,
                 stream=None):
    """y[t] = residual[t] + sum_j weights[t, j] h[r(t, j)] @ w_down[e(t, j)].

    h [T k, d_ff] in the routing's sorted order; w_down [E, d_ff, d] ("kn") or
    [E, d, d_ff] ("nk"); residual [T, d] (may be ``out``) or None; all
    contiguous bfloat16.  Returns y [T, d].
    """
    torch = _torch()
    bf16 = torch.bfloat16
    index = _first(h, "h", bf16)
    pw = _check(w_down, "w_down", index, bf16)
    lay = _code(LAYOUTS, layout, "layout")
    if h.dim() != 2 or w_down.dim() != 3 or w_down.shape[1 + lay] != h.shape[1]:
        raise ValueError("expected h [T k, d_ff] and w_down [E, d_ff, d] or [E, d, d_ff]")
    d_ff = h.shape[1]
    E, d = w_down.shape[0], w_down.shape[2 - lay]
    T, k, po = _routing_of(routing, E, index)
    pp = _check(routing.position, "routing.position", index, torch.int32)
    weights, pt = routing.weights, None
    if weights is not None:
        pt = _check(weights, "routing.weights", index, torch.float32)
        if weights.shape != routing.position.shape:
            raise ValueError("expected weights [T, k] in the routing")
    elif T * k > 0:
        raise ValueError("the routing needs weights")
    if h.shape[0] != T * k:
        raise ValueError("h has %d rows, the routing %d" % (h.shape[0], T * k))
    pr = None
    if residual is not None:
        pr = _check(residual, "residual", index, bf16)
        if residual.shape != (T, d):
            raise ValueError("residual must be [T, d] = [%d, %d]" % (T, d))
    out = _out(torch, out, (T, d), bf16, index, h.device, stream)
    ws, nws = _workspace(workspace, index)
    _call(index, _lib.load().swiglu_experts_down, h.data_ptr(), pw, po, pp, pt, pr, out.data_ptr(),
          T, k, E, d_ff, d, lay, ws, nws,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return out


def swiglu_moe(x, w_router, w_gate, w_up, w_down, k, router_bias=None, residual=None, out=None,
               layout="kn", stream=None, **routing):
    """The mixture-of-experts MLP: router logits (float32), ``route`` (further
    keyword arguments go to it), the experts' up and down projections.

    x [T, d], w_router [d, E], w_gate, w_up [E, d, d_ff], w_down [E, d_ff, d]
    ("kn"; each with its last two dimensions exchanged for "nk"); router_bias
    [E] is added to the logits.  Returns (y [T, d], the Routing).
    """
    torch = _torch()
    logits = linear(x, w_router, bias=router_bias, out_dtype=torch.float32, layout=layout,
                    stream=stream)
    r = route(logits, k, stream=stream, **routing)
    h = experts_up(x, w_gate, w_up, r, layout=layout, stream=stream)
    return experts_down(h, w_down, r, residual=residual, out=out, layout=layout, stream=stream), r


def _sorted_of(r, index):
    """(T, k, E, address of position, address of offsets) of a routing, read anew
    as in _routing_of."""
    i32 = _torch().int32
    shape = r.position.shape
    if len(shape) != 2 or r.offsets.dim() != 1 or r.offsets.numel() < 2:
        raise ValueError("expected position [T, k] and offsets [E + 1] in the routing")
    return (shape[0], shape[1], r.offsets.numel() - 1,
            _check(r.position, "routing.position", index, i32),
            _check(r.offsets, "routing.offsets", index, i32))


def _weights_of(r, index):
    """Address of a routing's weights [T, k] (0 where it has no pair)."""
    w = r.weights
    if w is None:
        if r.position.numel():
            raise ValueError("the routing needs weights")
        return None
    p = _check(w, "routing.weights", index, _torch().float32)
    if w.shape != r.position.shape:
        raise ValueError("expected weights [T, k] in the routing")
    return p


def _row_code(torch, t, name):
    if t.dtype is torch.bfloat16:
        return _lib.BF16
    if t.dtype is torch.float32:
        return _lib.F32
    raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def permute(x, routing, out=None, stream=None):
    """The rows of x at their sorted places: result[r] = x[t] for every (token t,
    expert e) pair r of ``routing``, in its sorted order; rows of dropped
    choices (at the end) are zero.

    x [T, d] is a contiguous bfloat16 or float32 tensor, or an Fp8Rows (the
    result is one too: the scales go along).  Returns [T k, d] of x's kind
    (``out`` if given).
    """
    torch = _torch()
    fp8 = isinstance(x, Fp8Rows)
    x, scales = x if fp8 else (x, None)
    index = _first(x, "codes" if fp8 else "x", torch.uint8 if fp8 else None)
    dt = _lib.E4M3 if fp8 else _row_code(torch, x, "x")
    if x.dim() != 2:
        raise ValueError("expected x [T, d]")
    T, d = x.shape
    rT, k, E, pp, po = _sorted_of(routing, index)
    if rT != T:
        raise ValueError("the routing is of %d tokens, not %d" % (rT, T))
    ps = pt = None
    new, new_scales = out if fp8 and out is not None else (out, None)
    new = _out(torch, new, (T * k, d), x.dtype, index, x.device, stream)
    if fp8:
        ps = _check(scales, "scales", index, torch.float32)
        if scales.dim() != 1 or scales.shape[0] != T:
            raise ValueError("expected scales [T] = [%d]" % T)
        new_scales = _out(torch, new_scales, (T * k,), torch.float32, index, x.device, stream)
        pt = new_scales.data_ptr()
    _call(index, _lib.load().swiglu_permute, x.data_ptr(), ps, pp, po, new.data_ptr(), pt, T, k, E,
          d, dt, stream.cuda_stream if stream is not None else _raw_stream(index))
    return Fp8Rows(new, new_scales) if fp8 else new


def _unpermute(z, routing, name, weighted, residual, out, stream):
    torch = _torch()
    index = _first(z, name)
    dt = _row_code(torch, z, name)
    T, k, _, pp, _ = _sorted_of(routing, index)
    if z.dim() != 2 or z.shape[0] != T * k:
        raise ValueError("expected %s [T k, d] with T k = %d" % (name, T * k))
    d = z.shape[1]
    pw = _weights_of(routing, index) if weighted else None
    pr = None
    if residual is not None:
        pr = _check(residual, "residual", index, z.dtype)
        if residual.shape != (T, d):
            raise ValueError("residual must be [T, d] = [%d, %d]" % (T, d))
    out = _out(torch, out, (T, d), z.dtype, index, z.device, stream)
    _call(index, _lib.load().swiglu_unpermute, z.data_ptr(), pp, pw, pr, out.data_ptr(), T, k, d,
          dt, stream.cuda_stream if stream is not None else _raw_stream(index))
    return out


def unpermute(z, routing, residual=None, out=None, stream=None):
    """y[t] = residual[t] + sum_j weights[t, j] z[r(t, j)], summed in float32 in
    the order of j and rounded once.

    z [T k, d], in the routing's sorted order, is a contiguous bfloat16 or
    float32 tensor; residual [T, d] of its dtype (may be ``out``) or None.
    Returns y [T, d].
    """
    return _unpermute(z, routing, "z", True, residual, out, stream)


def permute_backward(dout, routing, residual=None, out=None, stream=None):
    """The gradient of ``permute``'s x: dx[t] = residual[t] + sum_j dout[r(t, j)],
    residual being a gradient that reaches x another way, or None."""
    return _unpermute(dout, routing, "dout", False, residual, out, stream)


def unpermute_backward(dy, z, routing, out=None, stream=None):
    """The gradients of ``unpermute``: (dz [T k, d], dweights [T, k]).

    dy [T, d] and z [T k, d] are of one dtype, which dz has too (``out`` if
    given); dweights is float32.  The residual's gradient is dy itself.  Rows of
    dz that no choice has are zero, as are dweights of dropped choices.
    """
    torch = _torch()
    index = _first(dy, "dy")
    dt = _row_code(torch, dy, "dy")
    pz = _check(z, "z", index, dy.dtype)
    T, k, E, pp, po = _sorted_of(routing, index)
    if dy.dim() != 2 or dy.shape[0] != T or z.dim() != 2 or z.shape != (T * k, dy.shape[1]):
        raise ValueError("expected dy [T, d] and z [T k, d] of the routing's T = %d, k = %d"
                         % (T, k))
    d = dy.shape[1]
    pw = _weights_of(routing, index)
    dz = _out(torch, out, (T * k, d), dy.dtype, index, dy.device, stream)
    dw = _empty(torch, (T, k), torch.float32, dy.device, stream)
    _call(index, _lib.load().swiglu_unpermute_backward, dy.data_ptr(), pz, pp, po, pw, dz.data_ptr(),
          dw.data_ptr(), T, k, E, d, dt,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return dz, dw


def linear_workspace_bytes(M, K, N):
    """Workspace bytes ``linear`` needs on the current device."""
    return _bytes(_lib.load().swiglu_linear_workspace_bytes(M, K, N))


def experts_up_workspace_bytes(T, k, E, d, d_ff):
    """Workspace bytes ``experts_up`` needs on the current device."""
    return _bytes(_lib.load().swiglu_experts_up_workspace_bytes(T, k, E, d, d_ff))


def experts_down_workspace_bytes(T, k, E, d_ff, d):
    """Workspace bytes ``experts_down`` needs on the current device."""
    return _bytes(_lib.load().swiglu_experts_down_workspace_bytes(T, k, E, d_ff, d))


def _bytes(n):
    if n == 0:
        _lib.check(1)   # invalid sizes or no device (detail in the library's error string)
    return int(n)
