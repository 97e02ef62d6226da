"""Expert layers: routing, grouped products and the AdamW step.

Argument marshalling for the entry points of ``include/dpg.h`` of the same
names, in the manner of the package's projections: torch tensors in, outputs
allocated on the call's stream where the caller gives none, errors raised
before any launch.  A training step of an expert layer is

    r  = dpg_route(logits, top_k)
    xs = dpg_dispatch(x, r.positions, r.offsets)
    ys = dpg_grouped_forward(xs, w, r.offsets)
    y  = dpg_combine(ys, r.positions, r.offsets, r.weights)

with the gradients by ``dpg_combine_dgrad``, ``dpg_grouped_dgrad``,
``dpg_grouped_wgrad``, ``dpg_combine`` without weights (of dispatch) and
``dpg_route_dgrad``, and ``dpg_adamw`` on the FP32 weight gradients.
"""
import collections
import ctypes

import torch

from . import (DpgError, _check_in, _check_out, _check_same_device, _check_workspace, _code, _i64, _ci, _ld, _lib,
               _on_device, _on_stream, _stream, _sz, _vp, F32)

E4M3 = 2
ADAMW_BLOCK = 256  # elements that share one scale of an 8-bit moment

Route = collections.namedtuple("Route", "experts weights offsets rows positions")
Route.__doc__ = "What dpg_route returns: int32 experts, offsets, rows, positions and FP32 weights."


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("grad", _vp), ("exp_avg", _vp), ("exp_avg_sq", _vp), ("avg_scale", _vp),
                ("sq_scale", _vp), ("copy", _vp), ("numel", _i64)]


class _AdamwOptions(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", _i64), ("grad_scale", _vp),
                ("grad_dtype", _ci), ("state_dtype", _ci), ("seed", ctypes.c_uint32)]


_SIGNATURES = {
    "dpg_grouped_forward": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _ci, _vp, _i64, _i64, _i64, _i64, _vp],
    "dpg_grouped_dgrad": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _ci, _vp, _i64, _i64, _i64, _i64, _vp],
    "dpg_grouped_wgrad": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _ci, _vp, _i64, _i64, _i64, _i64, _vp],
    "dpg_route": [_vp, _i64, _i64, _i64, _i64, _ci, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "dpg_route_dgrad": [_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _ci, _vp],
    "dpg_dispatch": [_vp, _i64, _vp, _vp, _vp, _i64, _ci, _i64, _i64, _i64, _i64, _i64, _vp],
    "dpg_combine": [_vp, _i64, _ci, _vp, _vp, _vp, _vp, _i64, _ci, _i64, _i64, _i64, _i64, _i64, _vp],
    "dpg_combine_dgrad": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _ci, _i64, _i64, _i64, _i64, _i64,
                          _vp],
    "dpg_adamw": [ctypes.POINTER(_AdamwTensor), _i64, ctypes.POINTER(_AdamwOptions), _vp],
}
for _name, _args in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci
_lib.dpg_route_workspace_size.argtypes = [_i64, _i64, _i64]
_lib.dpg_route_workspace_size.restype = _sz


def _raise_on(status, name):
    if status:
        raise DpgError(status, name)


def _ints(t, name, shape=None):
    """A contiguous int32 device tensor, of `shape` where given."""
    _check_in(t, torch.int32, name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _offsets(offsets, experts=None):
    _ints(offsets, "offsets")
    if offsets.dim() != 1 or offsets.shape[0] < 1 or (experts is not None and offsets.shape[0] != experts + 1):
        raise ValueError("offsets must be [E + 1]%s, got %s" % ("" if experts is None else " with E = %d" % experts,
                                                               tuple(offsets.shape)))
    return offsets.shape[0] - 1


def _floats(t, name, shape):
    """A contiguous FP32 device tensor of `shape`."""
    _check_in(t, torch.float32, name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _groups(t, name):
    """(group stride, row stride) of an [E, N, K] matrix per group."""
    if t.dim() != 3:
        raise ValueError("%s must be [E, N, K]" % name)
    e, rows, cols = t.shape
    packed = (cols + 7) // 8 * 8
    if t.numel() == 0:
        return rows * packed, packed
    if cols > 1 and t.stride(2) != 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return (t.stride(0) if e > 1 else 0), (t.stride(1) if rows > 1 else packed)


# ------------------------------------------------------- grouped products --
def _rows_2d(t, name):
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return t.shape


def _grouped(name, a, w, offsets, out, out_dtype, out_cols, R, N, K, stream):
    E = w.shape[0]
    _offsets(offsets, E)
    _check_same_device(("a", a), ("w", w), ("offsets", offsets))
    dev = a.device
    if out is None:
        with _on_stream(stream, dev):
            out = torch.empty((R, out_cols), dtype=out_dtype, device=dev)
    _check_out(out, (R, out_cols), dev)
    stride_w, ldw = _groups(w, "w")
    with _on_device(dev):
        st = getattr(_lib, name)(a.data_ptr(), _ld(a, "a"), w.data_ptr(), ldw, stride_w, out.data_ptr(),
                                 _ld(out, "out"), _code(out.dtype), offsets.data_ptr(), E, R, N, K,
                                 _stream(stream, dev))
    _raise_on(st, name)
    return out


def dpg_grouped_forward(x, w, offsets, out=None, out_dtype=torch.bfloat16, stream=None):
    """y[r] = x[r] w[e]^T for the rows r of group e, offsets[e] <= r <
    offsets[e + 1]: x [R, K] BF16 sorted by group, w [E, N, K] BF16, offsets
    int32 [E + 1] on the device.  Rows from offsets[E] on give zeros."""
    _check_in(x, torch.bfloat16, "x")
    _check_in(w, torch.bfloat16, "w")
    R, K = _rows_2d(x, "x")
    if w.dim() != 3 or w.shape[2] != K:
        raise ValueError("w must be [E, N, K]")
    return _grouped("dpg_grouped_forward", x, w, offsets, out, out_dtype, w.shape[1], R, w.shape[1], K, stream)


def dpg_grouped_dgrad(dy, w, offsets, out=None, out_dtype=torch.bfloat16, stream=None):
    """dx[r] = dy[r] w[e] for the rows r of group e: dy [R, N], w [E, N, K]."""
    _check_in(dy, torch.bfloat16, "dy")
    _check_in(w, torch.bfloat16, "w")
    R, N = _rows_2d(dy, "dy")
    if w.dim() != 3 or w.shape[1] != N:
        raise ValueError("w must be [E, N, K]")
    return _grouped("dpg_grouped_dgrad", dy, w, offsets, out, out_dtype, w.shape[2], R, N, w.shape[2], stream)


def dpg_grouped_wgrad(dy, x, offsets, out=None, out_dtype=torch.bfloat16, stream=None):
    """dw[e] = sum over the rows r of group e of dy[r]^T x[r], as [E, N, K]: dy
    [R, N], x [R, K].  A group without rows gives zeros."""
    _check_in(dy, torch.bfloat16, "dy")
    _check_in(x, torch.bfloat16, "x")
    R, N = _rows_2d(dy, "dy")
    if _rows_2d(x, "x")[0] != R:
        raise ValueError("x must be [R, K]")
    K = x.shape[1]
    E = _offsets(offsets)
    _check_same_device(("dy", dy), ("x", x), ("offsets", offsets))
    dev = dy.device
    if out is None:
        with _on_stream(stream, dev):
            out = torch.empty((E, N, K), dtype=out_dtype, device=dev)
    _check_out(out, (E, N, K), dev)
    stride, ld = _groups(out, "out")
    with _on_device(dev):
        st = _lib.dpg_grouped_wgrad(dy.data_ptr(), _ld(dy, "dy"), x.data_ptr(), _ld(x, "x"), out.data_ptr(), ld,
                                    stride, _code(out.dtype), offsets.data_ptr(), E, R, N, K, _stream(stream, dev))
    _raise_on(st, "dpg_grouped_wgrad")
    return out


# ---------------------------------------------------------------- routing --
def _logits(logits):
    _check_in(logits, torch.float32, "logits")
    T, E = _rows_2d(logits, "logits")
    if E > 1 and T > 0 and logits.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    return T, E, (logits.stride(0) if T > 1 else E)


def dpg_route(logits, top_k, renormalize=True, workspace=None, stream=None):
    """The top_k experts of every token and the stable order of the (token,
    slot) pairs by expert, from FP32 logits [T, E]; a Route of experts [T,
    top_k] (-1: none left), weights [T, top_k] (softmax over the chosen
    experts, or over all with renormalize=False), offsets [E + 1], rows
    [T * top_k] and positions [T, top_k].  A logit of -inf masks its expert."""
    T, E, ld = _logits(logits)
    dev = logits.device
    need = _lib.dpg_route_workspace_size(T, E, top_k)
    if need == ctypes.c_size_t(-1).value:
        raise DpgError(2 if 1 <= top_k <= E else 1, "dpg_route")
    _check_workspace(workspace, dev)
    with _on_device(dev):
        with _on_stream(stream, dev):
            # one block of memory: an allocation costs about what a launch does
            n = T * top_k
            words = torch.empty(4 * n + E + 1, dtype=torch.int32, device=dev)
            if workspace is None and need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        experts, weights, rows, positions, offsets = words.split((n, n, n, n, E + 1))
        weights = weights.view(torch.float32).view(T, top_k)
        st = _lib.dpg_route(logits.data_ptr(), ld, T, E, top_k, int(bool(renormalize)), experts.data_ptr(),
                            weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), positions.data_ptr(),
                            workspace.data_ptr() if need else None,
                            workspace.numel() * workspace.element_size() if need else 0, _stream(stream, dev))
    _raise_on(st, "dpg_route")
    return Route(experts.view(T, top_k), weights, offsets, rows, positions.view(T, top_k))


def dpg_route_dgrad(logits, experts, weights, dweights, renormalize=True, out=None, stream=None):
    """Gradient of dpg_route's weights by the logits, FP32 [T, E]."""
    T, E, ld = _logits(logits)
    dev = logits.device
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must be [T, top_k]")
    k = experts.shape[1]
    _ints(experts, "experts")
    _floats(weights, "weights", (T, k))
    _floats(dweights, "dweights", (T, k))
    _check_same_device(("logits", logits), ("experts", experts), ("weights", weights), ("dweights", dweights))
    if out is None:
        with _on_stream(stream, dev):
            out = torch.empty((T, E), dtype=torch.float32, device=dev)
    _check_in(out, torch.float32, "out")
    _check_out(out, (T, E), dev)
    if E > 1 and T > 0 and out.stride(1) != 1:
        raise ValueError("out must have unit column stride")
    with _on_device(dev):
        st = _lib.dpg_route_dgrad(logits.data_ptr(), ld, experts.data_ptr(), weights.data_ptr(), dweights.data_ptr(),
                                  out.data_ptr(), out.stride(0) if T > 1 else E, T, E, k, int(bool(renormalize)),
                                  _stream(stream, dev))
    _raise_on(st, "dpg_route_dgrad")
    return out


def _row_code(t, name):
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("%s must be torch.bfloat16 or torch.float32" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return _code(t.dtype)


def _slots(positions):
    _ints(positions, "positions")
    if positions.dim() != 2 or positions.shape[1] < 1:
        raise ValueError("positions must be [T, top_k]")
    return positions.shape


def dpg_dispatch(x, positions, offsets, out=None, stream=None):
    """xs[positions[t, j]] = x[t] for every slot, zeros from row offsets[E] on:
    x [T, H] BF16 or FP32, xs [T * top_k, H] of the same type."""
    code = _row_code(x, "x")
    T, k = _slots(positions)
    if _rows_2d(x, "x")[0] != T:
        raise ValueError("x must be [T, H]")
    H = x.shape[1]
    E = _offsets(offsets)
    _check_same_device(("x", x), ("positions", positions), ("offsets", offsets))
    dev = x.device
    if out is None:
        with _on_stream(stream, dev):
            out = torch.empty((T * k, H), dtype=x.dtype, device=dev)
    _check_in(out, x.dtype, "out")
    _check_out(out, (T * k, H), dev)
    with _on_device(dev):
        st = _lib.dpg_dispatch(x.data_ptr(), _ld(x, "x"), positions.data_ptr(), offsets.data_ptr(), out.data_ptr(),
                               _ld(out, "out"), code, T, T * k, H, E, k, _stream(stream, dev))
    _raise_on(st, "dpg_dispatch")
    return out


def dpg_combine(ys, positions, offsets, weights=None, out=None, out_dtype=None, stream=None):
    """y[t] = sum_j weights[t, j] ys[positions[t, j]] over the used slots, in
    FP32 and ascending j: ys [T * top_k, H], y [T, H] of ys's type unless
    out_dtype says otherwise.  Without weights the rows are summed, which is
    the gradient of dpg_dispatch."""
    code = _row_code(ys, "ys")
    T, k = _slots(positions)
    R, H = _rows_2d(ys, "ys")
    if R != T * k:
        raise ValueError("ys must be [T * top_k, H]")
    E = _offsets(offsets)
    named = [("ys", ys), ("positions", positions), ("offsets", offsets)]
    if weights is not None:
        _floats(weights, "weights", (T, k))
        named.append(("weights", weights))
    _check_same_device(*named)
    dev = ys.device
    if out is None:
        with _on_stream(stream, dev):
            out = torch.empty((T, H), dtype=out_dtype or ys.dtype, device=dev)
    _check_out(out, (T, H), dev)
    with _on_device(dev):
        st = _lib.dpg_combine(ys.data_ptr(), _ld(ys, "ys"), code, positions.data_ptr(), offsets.data_ptr(),
                              weights.data_ptr() if weights is not None else None, out.data_ptr(), _ld(out, "out"),
                              _code(out.dtype), T, R, H, E, k, _stream(stream, dev))
    _raise_on(st, "dpg_combine")
    return out


def dpg_combine_dgrad(dy, ys, positions, offsets, weights, stream=None):
    """Gradients of dpg_combine by ys and the weights: dys[positions[t, j]] =
    weights[t, j] dy[t] (zeros from row offsets[E] on) and dweights[t, j] =
    <dy[t], ys[positions[t, j]]>; dy and ys of one type."""
    code = _row_code(dy, "dy")
    _check_in(ys, dy.dtype, "ys")
    T, k = _slots(positions)
    if _rows_2d(dy, "dy")[0] != T or tuple(ys.shape) != (T * k, dy.shape[1]):
        raise ValueError("dy must be [T, H] and ys [T * top_k, H]")
    H = dy.shape[1]
    E = _offsets(offsets)
    _floats(weights, "weights", (T, k))
    _check_same_device(("dy", dy), ("ys", ys), ("positions", positions), ("offsets", offsets), ("weights", weights))
    dev = dy.device
    with _on_stream(stream, dev):
        dys = torch.empty((T * k, H), dtype=ys.dtype, device=dev)
        dweights = torch.empty((T, k), dtype=torch.float32, device=dev)
    with _on_device(dev):
        st = _lib.dpg_combine_dgrad(dy.data_ptr(), _ld(dy, "dy"), ys.data_ptr(), _ld(ys, "ys"), positions.data_ptr(),
                                    offsets.data_ptr(), weights.data_ptr(), dys.data_ptr(), _ld(dys, "dys"),
                                    dweights.data_ptr(), code, T, T * k, H, E, k, _stream(stream, dev))
    _raise_on(st, "dpg_combine_dgrad")
    return dys, dweights


# ------------------------------------------------------------------ AdamW --
def _adamw_pointers(tensors, name, dtype, sizes, device):
    """Data pointers of a list of contiguous tensors, one per parameter."""
    if tensors is None:
        return [None] * len(sizes)
    if len(tensors) != len(sizes):
        raise ValueError("%s must hold one tensor per parameter" % name)
    pointers = []
    for t, n in zip(tensors, sizes):
        if t.dtype is not dtype:
            raise TypeError("%s must be %s" % (name, dtype))
        if t.device != device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
        if t.numel() != n:
            raise ValueError("%s: %d elements, expected %d" % (name, t.numel(), n))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        pointers.append(t.data_ptr())
    return pointers


def dpg_adamw(params, grads, exp_avgs, exp_avg_sqs, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1,
              copies=None, avg_scales=None, sq_scales=None, grad_scale=None, seed=0, stream=None):
    """One AdamW step over lists of tensors, in place: FP32 params, BF16 or
    FP32 grads, moments all in FP32 (m and v) or all in float8_e4m3fn (m and
    sqrt(v), with avg_scales and sq_scales of ceil(numel / 256) FP32 powers of
    two each).  copies, BF16, receive the rounded parameters.  grad_scale, a
    device FP32 scalar, multiplies the gradients.  8-bit moments are rounded at
    random from `seed`, which the caller changes from step to step."""
    if not params:
        return
    dev = params[0].device
    if dev.type != "cuda":
        raise ValueError("params must be device tensors")
    sizes = [t.numel() for t in params]
    grad_dtype = grads[0].dtype if len(grads) else torch.float32
    state_dtype = exp_avgs[0].dtype if len(exp_avgs) else torch.float32
    e4m3 = state_dtype == torch.float8_e4m3fn
    if not e4m3 and state_dtype != torch.float32:
        raise TypeError("moments must be torch.float32 or torch.float8_e4m3fn")
    if e4m3 and (avg_scales is None or sq_scales is None):
        raise ValueError("8-bit moments need avg_scales and sq_scales")
    blocks = [-(-n // ADAMW_BLOCK) for n in sizes]
    columns = (_adamw_pointers(params, "params", torch.float32, sizes, dev),
               _adamw_pointers(grads, "grads", grad_dtype, sizes, dev),
               _adamw_pointers(exp_avgs, "exp_avgs", state_dtype, sizes, dev),
               _adamw_pointers(exp_avg_sqs, "exp_avg_sqs", state_dtype, sizes, dev),
               _adamw_pointers(avg_scales if e4m3 else None, "avg_scales", torch.float32, blocks, dev),
               _adamw_pointers(sq_scales if e4m3 else None, "sq_scales", torch.float32, blocks, dev),
               _adamw_pointers(copies, "copies", torch.bfloat16, sizes, dev), sizes)
    table = (_AdamwTensor * len(sizes))(*zip(*columns))
    if grad_scale is not None:
        _floats(grad_scale.reshape(-1), "grad_scale", (1,))
        _check_same_device(("params", params[0]), ("grad_scale", grad_scale))
    options = _AdamwOptions(lr, beta1, beta2, eps, weight_decay, step,
                            grad_scale.data_ptr() if grad_scale is not None else None, _code(grad_dtype),
                            E4M3 if e4m3 else F32, seed & 0xFFFFFFFF)
    with _on_device(dev):
        st = _lib.dpg_adamw(table, len(sizes), ctypes.byref(options), _stream(stream, dev))
    _raise_on(st, "dpg_adamw")
