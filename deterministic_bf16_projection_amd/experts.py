"""Expert layers: routing, grouped products and the AdamW step.

The entry points of ``include/dpg.h`` of the same names, in the manner of the
package's projections: torch tensors in, outputs allocated on the call's stream
where the caller gives none, errors raised before any launch.  What a call
writes in place (an ``out``, the optimizer's tensors) counts as modified for
autograd.  The compiled module ``_binding`` checks and marshals the arguments; called through ctypes
like the projections, it would take longer than the kernels of small calls.  A
training step of an expert layer is

    r  = dpg_route(logits, top_k)
    xs = dpg_dispatch(x, r.positions, r.offsets)
    ys = dpg_grouped_forward(xs, w, r.offsets)
    y  = dpg_combine(ys, r.positions, r.offsets, r.weights)

with the gradients by ``dpg_combine_dgrad``, ``dpg_grouped_dgrad``,
``dpg_grouped_wgrad``, ``dpg_combine`` without weights (of dispatch) and
``dpg_route_dgrad``, and ``dpg_adamw`` on the FP32 weight gradients.
"""
import collections

import torch

from . import DpgError, _binding, _on_device, _on_stream

ADAMW_BLOCK = 256  # elements that share one scale of an 8-bit moment

Route = collections.namedtuple("Route", "experts weights offsets rows positions")
Route.__doc__ = "What dpg_route returns: int32 experts, offsets, rows, positions and FP32 weights."

_binding.set_error(DpgError)


def _on(stream, tensor, fn, *args):
    """fn(*args) with `stream` as the current stream: the binding launches and
    allocates on that one."""
    with _on_device(tensor.device), _on_stream(stream, tensor.device):
        return fn(*args)


# ------------------------------------------------------- grouped products --
def dpg_grouped_forward(x, w, offsets, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """y[r] = x[r] w[e]^T for the rows r of group e, offsets[e] <= r <
    offsets[e + 1]: x [R, K] BF16 sorted by group, w [E, N, K] BF16, offsets
    int32 [E + 1] on the device.  Rows from offsets[E] on give zeros."""
    if stream is None:
        return _binding.grouped_forward(x, w, offsets, out, out_dtype, workspace)
    return _on(stream, x, _binding.grouped_forward, x, w, offsets, out, out_dtype, workspace)


def dpg_grouped_dgrad(dy, w, offsets, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """dx[r] = dy[r] w[e] for the rows r of group e: dy [R, N], w [E, N, K]."""
    if stream is None:
        return _binding.grouped_dgrad(dy, w, offsets, out, out_dtype, workspace)
    return _on(stream, dy, _binding.grouped_dgrad, dy, w, offsets, out, out_dtype, workspace)


def dpg_grouped_wgrad(dy, x, offsets, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """dw[e] = sum over the rows r of group e of dy[r]^T x[r], as [E, N, K]: dy
    [R, N], x [R, K].  A group without rows gives zeros."""
    if stream is None:
        return _binding.grouped_wgrad(dy, x, offsets, out, out_dtype, workspace)
    return _on(stream, dy, _binding.grouped_wgrad, dy, x, offsets, out, out_dtype, workspace)


# ---------------------------------------------------------------- routing --
def dpg_route(logits, top_k, renormalize=True, workspace=None, stream=None):
    """The top_k experts of every token and the stable order of the (token,
    slot) pairs by expert, from FP32 logits [T, E]; a Route of experts [T,
    top_k] (-1: none left), weights [T, top_k] (softmax over the chosen
    experts, or over all with renormalize=False), offsets [E + 1], rows
    [T * top_k] and positions [T, top_k].  A logit of -inf masks its expert."""
    if stream is None:
        return Route._make(_binding.route(logits, top_k, renormalize, workspace))
    return Route._make(_on(stream, logits, _binding.route, logits, top_k, renormalize, workspace))


def dpg_route_dgrad(logits, experts, weights, dweights, renormalize=True, out=None, stream=None):
    """Gradient of dpg_route's weights by the logits, FP32 [T, E]."""
    if stream is None:
        return _binding.route_dgrad(logits, experts, weights, dweights, renormalize, out)
    return _on(stream, logits, _binding.route_dgrad, logits, experts, weights, dweights, renormalize, out)


def dpg_dispatch(x, positions, offsets, out=None, stream=None):
    """xs[positions[t, j]] = x[t] for every slot, zeros from row offsets[E] on:
    x [T, H] BF16 or FP32, xs [T * top_k, H] of the same type."""
    if stream is None:
        return _binding.dispatch(x, positions, offsets, out)
    return _on(stream, x, _binding.dispatch, x, positions, offsets, out)


def dpg_combine(ys, positions, offsets, weights=None, out=None, out_dtype=None, stream=None):
    """y[t] = sum_j weights[t, j] ys[positions[t, j]] over the used slots, in
    FP32 and ascending j: ys [T * top_k, H], y [T, H] of ys's type unless
    out_dtype says otherwise.  Without weights the rows are summed, which is
    the gradient of dpg_dispatch."""
    if stream is None:
        return _binding.combine(ys, positions, offsets, weights, out, out_dtype)
    return _on(stream, ys, _binding.combine, ys, positions, offsets, weights, out, out_dtype)


def dpg_combine_dgrad(dy, ys, positions, offsets, weights, stream=None):
    """Gradients of dpg_combine by ys and the weights: dys[positions[t, j]] =
    weights[t, j] dy[t] (zeros from row offsets[E] on) and dweights[t, j] =
    <dy[t], ys[positions[t, j]]>; dy and ys of one type."""
    if stream is None:
        return _binding.combine_dgrad(dy, ys, positions, offsets, weights)
    return _on(stream, dy, _binding.combine_dgrad, dy, ys, positions, offsets, weights)


# ------------------------------------------------------------------ AdamW --
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
    if stream is None:
        _binding.adamw(params, grads, exp_avgs, exp_avg_sqs, copies, avg_scales, sq_scales, grad_scale, lr, beta1,
                       beta2, eps, weight_decay, step, seed & 0xFFFFFFFF)
    else:
        _on(stream, params[0], _binding.adamw, params, grads, exp_avgs, exp_avg_sqs, copies, avg_scales, sq_scales,
            grad_scale, lr, beta1, beta2, eps, weight_decay, step, seed & 0xFFFFFFFF)
