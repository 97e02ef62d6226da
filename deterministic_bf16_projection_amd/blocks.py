"""Between the projections of a residual block: layer norm, dropout and a gated
linear recurrence.

The entry points of ``include/dpg.h`` of the same names, in the manner of the
package's others: torch tensors in, outputs allocated on the call's stream where
the caller gives none, errors raised before any launch.  A pre-norm block whose
rows are mixed along the sequence is

    n = dpg_add_layer_norm(y, stream, weight, bias, p=p, seed=seed, step=step)
    r = dpg_recurrence(dpg_forward(n.y, w_gate), dpg_forward(n.y, w_in))   # as [B, T, D]
    y = dpg_forward(r.h, w_out)

where n.sum is the stream that goes on, with the gradients by
``dpg_add_layer_norm_dgrad``, ``dpg_recurrence_dgrad`` and the projections' own.
"""
import collections

import torch

from . import _binding
from .experts import _on

LayerNorm = collections.namedtuple("LayerNorm", "y mean rstd sum")
LayerNorm.__doc__ = "What a layer norm returns: y, FP32 mean and rstd, and the sum that was normalised (or None)."
LayerNormGrad = collections.namedtuple("LayerNormGrad", "dx dresidual dweight dbias")
LayerNormGrad.__doc__ = "Gradients of a layer norm; dresidual is None where there was no residual."
Recurrence = collections.namedtuple("Recurrence", "h state carries")
Recurrence.__doc__ = "What dpg_recurrence returns: h, the FP32 state after each sequence, and carries (or None)."
RecurrenceGrad = collections.namedtuple("RecurrenceGrad", "dgate dx dstate")
RecurrenceGrad.__doc__ = "Gradients of dpg_recurrence; dstate is None where there was no state."


def dpg_dropout(x, p, seed, step=None, residual=None, out=None, out_dtype=None, stream=None):
    """y = keep x / (1 - p) [+ residual] for x [T, H], BF16 or FP32: the mask is a
    function of `seed`, `step` (a device int64 scalar, which a captured call
    reads at each replay) and an element's place.  y has residual's type, or
    x's unless out_dtype says otherwise.  The gradient is the same call on dy."""
    if stream is None:
        return _binding.dropout(x, p, seed, step, residual, out, out_dtype)
    return _on(stream, x, _binding.dropout, x, p, seed, step, residual, out, out_dtype)


def dpg_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=None, stream=None):
    """y = (x - mean) rstd weight + bias over the columns of x [T, H], BF16 or
    FP32, with FP32 weight and bias [H] (None: ones, zeros); y of x's type
    unless out_dtype says otherwise."""
    if stream is None:
        return LayerNorm(*_binding.layer_norm(x, weight, bias, eps, out, out_dtype), None)
    return LayerNorm(*_on(stream, x, _binding.layer_norm, x, weight, bias, eps, out, out_dtype), None)


def dpg_add_layer_norm(x, residual, weight=None, bias=None, eps=1e-5, p=0.0, seed=0, step=None, out=None, sum=None,
                       out_dtype=None, stream=None):
    """The layer norm of sum = residual + dropout(x), and the sum, of residual's
    type (`sum` may be residual itself); p, seed and step as for dpg_dropout; y
    of x's type unless out_dtype says otherwise."""
    args = (x, residual, weight, bias, eps, p, seed, step, out, sum, out_dtype)
    if stream is None:
        return LayerNorm._make(_binding.add_layer_norm(*args))
    return LayerNorm._make(_on(stream, x, _binding.add_layer_norm, *args))


def dpg_layer_norm_dgrad(dy, x, mean, rstd, weight=None, weight_grads=True, workspace=None, stream=None):
    """Gradients of dpg_layer_norm by x (of x's type), weight and bias (FP32; None
    with weight_grads=False), from what the call read and returned."""
    args = (dy, x, mean, rstd, weight, weight_grads, workspace)
    dx, dw, db = _binding.layer_norm_dgrad(*args) if stream is None else _on(stream, dy, _binding.layer_norm_dgrad,
                                                                             *args)
    return LayerNormGrad(dx, None, dw, db)


def dpg_add_layer_norm_dgrad(dy, sum, mean, rstd, weight=None, dsum=None, p=0.0, seed=0, step=None, x_dtype=None,
                             weight_grads=True, workspace=None, stream=None):
    """Gradients of dpg_add_layer_norm by x (of type x_dtype, dy's unless given),
    residual (of sum's type), weight and bias, from the sum that the call
    returned and its dropout's p, seed and step.  dsum: the gradient that
    reaches the sum from elsewhere."""
    args = (dy, sum, mean, rstd, weight, dsum, p, seed, step, x_dtype, weight_grads, workspace)
    if stream is None:
        return LayerNormGrad._make(_binding.add_layer_norm_dgrad(*args))
    return LayerNormGrad._make(_on(stream, dy, _binding.add_layer_norm_dgrad, *args))


def dpg_recurrence(gate, x, offsets=None, state=None, coupled=True, carries=False, out=None, state_out=None,
                   workspace=None, stream=None):
    """h[t] = f h[t - 1] + w x[t] with f = sigmoid(gate[t]) and w = 1 - f (coupled)
    or 1, along the sequences of x and gate [B, T, D], or [R, D] with int32
    offsets [S + 1] on the device; BF16 or FP32.  state [B, D], FP32, is h
    before the first rows; the state returned (into state_out, which may be
    `state`) is h after the last.  With carries=True the call keeps what
    dpg_recurrence_dgrad needs."""
    args = (x, gate, offsets, state, coupled, carries, out, state_out, workspace)
    if stream is None:
        return Recurrence._make(_binding.recurrence(*args))
    return Recurrence._make(_on(stream, x, _binding.recurrence, *args))


def dpg_recurrence_dgrad(dh, gate, x, carries, offsets=None, state=None, dstate=None, coupled=True, workspace=None,
                         stream=None):
    """Gradients of dpg_recurrence by gate, x and state, from dh, the gradient of
    h, and dstate, that of the state returned (None: zeros)."""
    args = (dh, gate, x, carries, offsets, state, dstate, coupled, workspace)
    if stream is None:
        return RecurrenceGrad._make(_binding.recurrence_dgrad(*args))
    return RecurrenceGrad._make(_on(stream, x, _binding.recurrence_dgrad, *args))
