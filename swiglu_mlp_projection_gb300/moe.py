"""The mixture-of-experts MLP and the general linear product (see
``include/swiglu.h`` for the exact definitions): ``linear``, ``route``,
``dispatch``, ``experts_up``, ``experts_down``, and ``swiglu_moe``, which runs
them in turn.

As the rest of the binding, these only marshal torch tensors into the C ABI;
calls are asynchronous on torch's current stream (or ``stream``).
"""
import collections

from . import _lib
from . import _call, _check_cuda, _raw_stream

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
LAYOUTS = {"kn": 0, "nk": 1}

Routing = collections.namedtuple("Routing", "ids weights offsets order position")
Routing.__doc__ = """Where each token goes: ids [T, k] int32 (-1: no expert), weights [T, k]
float32, and the (token, choice) pairs sorted by expert: offsets [E + 1],
order [T k], position [T, k], int32 (``route`` and ``dispatch`` write them)."""


def _code(table, value, what):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s" % (what, sorted(table))) from None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace):
    if workspace is None:
        return None, 0
    _check_cuda(workspace=workspace)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _same_device(index, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s must be on the same device as the first argument" % name)


def _bf16(**tensors):
    import torch
    for name, t in tensors.items():
        if t is not None and t.dtype != torch.bfloat16:
            raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))


def _out(out, shape, dtype, like):
    import torch
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _check_cuda(out=out)
    _same_device(like.get_device(), out=out)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError("out must be a contiguous %s tensor of %s" % (tuple(shape), dtype))
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
    import torch
    _check_cuda(x=x, w=w, bias=bias, residual=residual)
    _bf16(x=x, w=w)
    lay = _code(LAYOUTS, layout, "layout")
    act = _code(ACTIVATIONS, activation, "activation")
    if x.dim() != 2 or w.dim() != 2 or w.shape[lay] != x.shape[1]:
        raise ValueError("expected x [M, K] and w [K, N] (kn) or [N, K] (nk)")
    M, K = x.shape
    N = w.shape[1 - lay]
    index = x.get_device()
    _same_device(index, w=w, bias=bias, residual=residual)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    bias_code = _lib.BF16
    if bias is not None:
        if bias.shape != (N,):
            raise ValueError("bias must be [N] = [%d]" % N)
        if bias.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("bias must be bfloat16 or float32")
        bias_code = _lib.BF16 if bias.dtype == torch.bfloat16 else _lib.F32
    if residual is not None and (residual.shape != (M, N) or residual.dtype != out_dtype):
        raise ValueError("residual must be [M, N] of the result's dtype")
    out = _out(out, (M, N), out_dtype, x)
    ws, nws = _workspace(workspace)
    _call(index, _lib.load().swiglu_linear, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual),
          out.data_ptr(), M, K, N, act, bias_code,
          _lib.BF16 if out_dtype == torch.bfloat16 else _lib.F32, lay, ws, nws,
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
    import torch
    _check_cuda(logits=logits, bias=bias)
    if logits.dim() != 2:
        raise ValueError("expected logits [T, E]")
    if logits.dtype == torch.float32:
        dt = _lib.F32
    elif logits.dtype == torch.bfloat16:
        dt = _lib.BF16
    else:
        raise TypeError("logits must be float32 or bfloat16, got %s" % logits.dtype)
    T, E = logits.shape
    index = logits.get_device()
    if bias is not None:
        _same_device(index, bias=bias)
        if bias.shape != (E,) or bias.dtype != torch.float32:
            raise ValueError("bias must be a float32 [E] = [%d] tensor" % E)
    sc = _code(SCORES, score, "score")
    gs = _code(GROUP_SCORES, group_score, "group_score")
    if topk_groups is None:
        topk_groups = groups
    dev = logits.device
    if k < 0:
        raise ValueError("k must not be negative")
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order = torch.empty(T * k, dtype=torch.int32, device=dev)
    position = torch.empty((T, k), dtype=torch.int32, device=dev)
    _call(index, _lib.load().swiglu_route, logits.data_ptr(), _ptr(bias), ids.data_ptr(),
          weights.data_ptr(), offsets.data_ptr(), order.data_ptr(), position.data_ptr(), T, E, k,
          dt, sc, groups, topk_groups, gs, 1 if renormalize else 0, float(scale),
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return Routing(ids, weights, offsets, order, position)


def dispatch(ids, n_experts, weights=None, stream=None):
    """A Routing from chosen experts ids [T, k] (int32; values outside
    0 ... n_experts - 1 are dropped) and their weights [T, k] (float32)."""
    import torch
    _check_cuda(ids=ids, weights=weights)
    if ids.dim() != 2 or ids.dtype != torch.int32:
        raise ValueError("expected int32 ids [T, k]")
    T, k = ids.shape
    index = ids.get_device()
    if weights is not None:
        _same_device(index, weights=weights)
        if weights.shape != ids.shape or weights.dtype != torch.float32:
            raise ValueError("weights must be float32 of ids' shape")
    dev = ids.device
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    order = torch.empty(T * k, dtype=torch.int32, device=dev)
    position = torch.empty((T, k), dtype=torch.int32, device=dev)
    _call(index, _lib.load().swiglu_dispatch, ids.data_ptr(), offsets.data_ptr(), order.data_ptr(),
          position.data_ptr(), T, k, n_experts,
          stream.cuda_stream if stream is not None else _raw_stream(index))
    return Routing(ids, weights, offsets, order, position)


def _check_routing(routing, T, E, index, weights):
    import torch
    T2, k = routing.position.shape
    if T2 != T:
        raise ValueError("the routing is of %d tokens, not %d" % (T2, T))
    if routing.offsets.shape != (E + 1,) or routing.order.shape != (T * k,):
        raise ValueError("the routing is not one of %d experts" % E)
    for name in ("offsets", "order", "position"):
        if getattr(routing, name).dtype != torch.int32:
            raise TypeError("routing.%s must be int32" % name)
    _check_cuda(offsets=routing.offsets, order=routing.order, position=routing.position)
    _same_device(index, offsets=routing.offsets, order=routing.order, position=routing.position)
    if weights:
        w = routing.weights
        if w is None or w.shape != (T, k) or w.dtype != torch.float32:
            raise ValueError("the routing needs float32 weights [T, k]")
        _check_cuda(weights=w)
        _same_device(index, weights=w)
    return k


def experts_up(x, w_gate, w_up, routing, out=None, layout="kn", workspace=None, stream=None):
    """h[r] = silu(x[t] @ w_gate[e]) * (x[t] @ w_up[e]) for every (token t,
    expert e) pair r of ``routing``, in its sorted order: h [T k, d_ff].

    x [T, d]; w_gate, w_up [E, d, d_ff] ("kn") or [E, d_ff, d] ("nk"); all
    contiguous bfloat16.  Rows of dropped choices (at the end) are zero.
    """
    import torch
    _check_cuda(x=x, w_gate=w_gate, w_up=w_up)
    _bf16(x=x, w_gate=w_gate, w_up=w_up)
    lay = _code(LAYOUTS, layout, "layout")
    if x.dim() != 2 or w_gate.dim() != 3 or w_up.shape != w_gate.shape \
            or w_gate.shape[1 + lay] != x.shape[1]:
        raise ValueError("expected x [T, d] and w_gate, w_up [E, d, d_ff] or [E, d_ff, d]")
    T, d = x.shape
    E, d_ff = w_gate.shape[0], w_gate.shape[2 - lay]
    index = x.get_device()
    _same_device(index, w_gate=w_gate, w_up=w_up)
    k = _check_routing(routing, T, E, index, False)
    out = _out(out, (T * k, d_ff), torch.bfloat16, x)
    ws, nws = _workspace(workspace)
    _call(index, _lib.load().swiglu_experts_up, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
          routing.offsets.data_ptr(), routing.order.data_ptr(), out.data_ptr(), T, k, E, d, d_ff,
          lay, ws, nws, stream.cuda_stream if stream is not None else _raw_stream(index))
    return out


def experts_down(h, w_down, routing, residual=None, out=None, layout="kn", workspace=None,
                 stream=None):
    """y[t] = residual[t] + sum_j weights[t, j] h[r(t, j)] @ w_down[e(t, j)].

    h [T k, d_ff] in the routing's sorted order; w_down [E, d_ff, d] ("kn") or
    [E, d, d_ff] ("nk"); residual [T, d] (may be ``out``) or None; all
    contiguous bfloat16.  Returns y [T, d].
    """
    import torch
    _check_cuda(h=h, w_down=w_down, residual=residual)
    _bf16(h=h, w_down=w_down, residual=residual)
    lay = _code(LAYOUTS, layout, "layout")
    if h.dim() != 2 or w_down.dim() != 3 or w_down.shape[1 + lay] != h.shape[1]:
        raise ValueError("expected h [T k, d_ff] and w_down [E, d_ff, d] or [E, d, d_ff]")
    d_ff = h.shape[1]
    E, d = w_down.shape[0], w_down.shape[2 - lay]
    index = h.get_device()
    _same_device(index, w_down=w_down, residual=residual)
    T = routing.position.shape[0]
    k = _check_routing(routing, T, E, index, True)
    if h.shape[0] != T * k:
        raise ValueError("h has %d rows, the routing %d" % (h.shape[0], T * k))
    if residual is not None and residual.shape != (T, d):
        raise ValueError("residual must be [T, d] = [%d, %d]" % (T, d))
    out = _out(out, (T, d), torch.bfloat16, h)
    ws, nws = _workspace(workspace)
    _call(index, _lib.load().swiglu_experts_down, h.data_ptr(), w_down.data_ptr(),
          routing.offsets.data_ptr(), routing.position.data_ptr(), routing.weights.data_ptr(),
          _ptr(residual), out.data_ptr(), T, k, E, d_ff, d, lay, ws, nws,
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
    import torch
    logits = linear(x, w_router, bias=router_bias, out_dtype=torch.float32, layout=layout,
                    stream=stream)
    r = route(logits, k, stream=stream, **routing)
    h = experts_up(x, w_gate, w_up, r, layout=layout, stream=stream)
    return experts_down(h, w_down, r, residual=residual, out=out, layout=layout, stream=stream), r


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
