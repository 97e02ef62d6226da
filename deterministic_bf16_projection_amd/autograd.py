"""Training wrappers over the C ABI.

``projection(x, w)`` and ``router_gating(x, w)`` are torch autograd functions:
the forward calls ``dpg_forward`` / ``dpg_router_forward`` and saves only its
inputs; the backward calls the input-gradient and weight-gradient entry points
on the incoming gradient.  ``CheckpointedStep`` prepares the launches of one
checkpointed training step of a projection (forward, recomputed forward, input
gradient, weight gradient) with static buffers and captures them in one HIP
graph, so a replay costs no host work per kernel.

``route``, ``dispatch``, ``grouped_projection`` and ``combine`` are the same for
the expert layer's entry points; an expert layer is

    r = route(router_gating(x32, w_router), top_k)
    h = grouped_projection(dispatch(x, r), w_experts, r.offsets)
    y = combine(h, r)

``layer_norm``, ``add_layer_norm``, ``dropout`` and ``recurrence`` are what stands
between the projections of a residual block:

    h, stream = add_layer_norm(y, stream, w_norm, b_norm, p=p, seed=seed, step=step)
    m, state = recurrence(projection(h, w_gate), projection(h, w_in))
    y = projection(m, w_out)

Their gradients have no gradients: differentiating twice raises.

Argument marshalling only, as in the rest of the package: every product runs
in the library's kernels.  ``deterministic=False`` asks for the fast plans; when
``torch.use_deterministic_algorithms(True)`` is in force the deterministic
plans are used instead and a warning is given once.
"""
import warnings

import torch
from torch.autograd.function import once_differentiable

from . import (Route, dpg_combine, dpg_combine_dgrad, dpg_dispatch, dpg_grouped_dgrad, dpg_grouped_forward,
               dpg_grouped_wgrad, dpg_route, dpg_route_dgrad)
from . import (dpg_add_layer_norm, dpg_add_layer_norm_dgrad, dpg_dropout, dpg_layer_norm, dpg_layer_norm_dgrad,
               dpg_recurrence, dpg_recurrence_dgrad)
from . import (dpg_dgrad, dpg_forward, dpg_router_dgrad, dpg_router_forward, dpg_router_wgrad, dpg_wgrad,
               workspace_size, PASS_FORWARD, PASS_DGRAD, PASS_WGRAD)

_warned = [False]


def resolve_deterministic(deterministic):
    """The plan family a call runs: deterministic if asked for, or if torch's
    deterministic-algorithms switch is on (then warns once)."""
    if deterministic:
        return True
    if torch.are_deterministic_algorithms_enabled():
        if not _warned[0]:
            warnings.warn("torch.use_deterministic_algorithms(True) is set: the projection GEMMs run their "
                          "deterministic plans", stacklevel=3)
            _warned[0] = True
        return True
    return False


def _packed(t):
    """t itself where it is contiguous and starts at a multiple of 16 bytes, as the
    library takes it, else a copy: a gradient may be a view of a larger one."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _rows(t):
    """[..., C] as a contiguous [R, C] view (the library takes unit column stride)."""
    return _packed(t.reshape(-1, t.shape[-1]))


class _Projection(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, deterministic, out_dtype, round_grad):
        x2 = _rows(x)
        y = dpg_forward(x2, w, out_dtype=out_dtype, deterministic=deterministic)
        ctx.save_for_backward(x2, w)
        ctx.deterministic = deterministic
        ctx.round_grad = round_grad
        ctx.x_shape = x.shape
        return y.reshape(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, dy):
        x2, w = ctx.saved_tensors
        # the library's gradient passes take a BF16 dY; any other incoming
        # gradient is rounded (nearest even) only when the caller asked for it
        if dy.dtype != torch.bfloat16:
            if not ctx.round_grad:
                raise TypeError("projection: the incoming gradient is %s, but the gradient GEMMs take BF16; "
                                "pass round_grad_to_bf16=True to round it to BF16 explicitly" % dy.dtype)
            dy = dy.to(torch.bfloat16)
        dy2 = _rows(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = dpg_dgrad(dy2, w, out_dtype=torch.bfloat16, deterministic=ctx.deterministic).reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            dw = dpg_wgrad(dy2, x2, out_dtype=torch.bfloat16, deterministic=ctx.deterministic)
        return dx, dw, None, None, None


class _Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, deterministic):
        x2 = _rows(x)
        y = dpg_router_forward(x2, w, deterministic=deterministic)
        ctx.save_for_backward(x2, w)
        ctx.deterministic = deterministic
        ctx.x_shape = x.shape
        return y.reshape(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, dy):
        x2, w = ctx.saved_tensors
        dy2 = _rows(dy if dy.dtype == torch.float32 else dy.to(torch.float32))
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = dpg_router_dgrad(dy2, w, deterministic=ctx.deterministic).reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            dw = dpg_router_wgrad(dy2, x2, deterministic=ctx.deterministic)
        return dx, dw, None


def projection(x, w, deterministic=True, out_dtype=torch.bfloat16, round_grad_to_bf16=False):
    """y[..., N] = x[..., K] w[N, K]^T with BF16 operands and FP32 accumulation;
    differentiable in x and w (gradients in BF16).

    The gradient GEMMs take a BF16 incoming gradient.  With ``out_dtype=float32``
    the incoming gradient is FP32: backward then raises unless
    ``round_grad_to_bf16=True``, which rounds it to BF16 (nearest even) first."""
    return _Projection.apply(x, w, resolve_deterministic(deterministic), out_dtype, bool(round_grad_to_bf16))


def router_gating(x, w, deterministic=True):
    """FP32 router logits y[..., E] = x[..., H] w[E, H]^T by BF16x3;
    differentiable in x and w (FP32 gradients)."""
    return _Router.apply(x, w, resolve_deterministic(deterministic))


def _matrix(t):
    """[..., C] as a 2-D matrix that the library takes: rows that do not overlap,
    unit column stride; copied only where it is not one already."""
    t2 = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    rows, cols = t2.shape
    return t2 if (cols <= 1 or t2.stride(1) == 1) and (rows <= 1 or t2.stride(0) >= cols) else t2.contiguous()


def _slots(t):
    """[..., top_k] as [T, top_k]."""
    return t if t.dim() == 2 else t.reshape(-1, t.shape[-1])


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, renormalize):
        matrix = _matrix(logits)
        r = dpg_route(matrix, top_k, renormalize=renormalize)
        if logits.dim() != 2:
            lead = logits.shape[:-1]
            r = r._replace(experts=r.experts.view(*lead, top_k), weights=r.weights.view(*lead, top_k),
                           positions=r.positions.view(*lead, top_k))
        ctx.save_for_backward(matrix, r.experts, r.weights)
        ctx.renormalize = renormalize
        ctx.shape = logits.shape
        ctx.mark_non_differentiable(r.experts, r.offsets, r.rows, r.positions)
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, _experts, dweights, _offsets, _rows_, _positions):
        matrix, experts, weights = ctx.saved_tensors
        dlogits = dpg_route_dgrad(matrix, _slots(experts), _slots(weights), _slots(dweights).contiguous(),
                                  renormalize=ctx.renormalize)
        return dlogits.reshape(ctx.shape), None, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, offsets):
        ctx.save_for_backward(positions, offsets)
        ctx.shape = x.shape
        return dpg_dispatch(_matrix(x), _slots(positions), offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        positions, offsets = ctx.saved_tensors
        return dpg_combine(_rows(dxs), _slots(positions), offsets).reshape(ctx.shape), None, None


class _Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return dpg_grouped_forward(x, w, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = _rows(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = dpg_grouped_dgrad(dy, w, offsets)
        if ctx.needs_input_grad[1]:
            dw = dpg_grouped_wgrad(dy, x, offsets)
        return dx, dw, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, positions, offsets):
        ctx.save_for_backward(ys, weights, positions, offsets)
        y = dpg_combine(ys, _slots(positions), offsets, _slots(weights))
        return y if positions.dim() == 2 else y.view(*positions.shape[:-1], ys.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weights, positions, offsets = ctx.saved_tensors
        dys, dweights = dpg_combine_dgrad(_rows(dy), ys, _slots(positions), offsets, _slots(weights))
        return dys, dweights.view(weights.shape), None, None


def route(logits, top_k, renormalize=True):
    """dpg_route on logits [..., E], differentiable from its weights to the logits
    (the choice of experts is held): experts, weights and positions are [...,
    top_k], the tokens numbered in the order of the leading dimensions."""
    return Route._make(_Route.apply(logits, top_k, bool(renormalize)))


def dispatch(x, r):
    """x [..., H] into the order of the route r, [T * top_k, H]; differentiable in x."""
    return _Dispatch.apply(x, r.positions, r.offsets)


def grouped_projection(x, w, offsets):
    """y[r] = x[r] w[e]^T for the rows r of group e (BF16); differentiable in x and
    w.  Use dpg_grouped_wgrad with out_dtype=torch.float32 for FP32 gradients."""
    return _Grouped.apply(x, w, offsets)


def combine(ys, r):
    """y[t] = sum_j weights[t, j] ys[positions[t, j]], as [..., H] with the leading
    dimensions of the route r; differentiable in ys and in the route's weights."""
    return _Combine.apply(ys, r.weights, r.positions, r.offsets)


def _aligned(t, pitch):
    """Whether t and its rows, `pitch` elements apart, start at multiples of 16 bytes."""
    return t.data_ptr() % 16 == 0 and pitch * t.element_size() % 16 == 0


def _operand(t):
    """_matrix(t), copied where its rows are not aligned."""
    t2 = _matrix(t)
    return t2 if _aligned(t2, t2.stride(0) if t2.shape[0] > 1 else 0) else t2.clone(memory_format=torch.contiguous_format)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        matrix = _operand(x)
        n = dpg_layer_norm(matrix, weight, bias, eps=eps, out_dtype=out_dtype)
        ctx.save_for_backward(matrix, weight, n.mean, n.rstd)
        ctx.shape = x.shape
        return n.y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        matrix, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        d = dpg_layer_norm_dgrad(_rows(dy), matrix, mean, rstd, weight, weight_grads=need[1] or need[2])
        return (d.dx.view(ctx.shape) if need[0] else None, d.dweight if need[1] else None,
                d.dbias if need[2] else None, None, None)


def _same_shape(x, residual):
    # the matrices that the library sees could still agree, the gradients' shapes not
    if residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")


def _mask_step(p, step):
    """The step that the backward pass needs: saved, so that counting it up before
    then is an error that its version shows; none where nothing is left out."""
    return step if p > 0 else None


class _AddLayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, p, seed, step, out_dtype):
        _same_shape(x, residual)
        n = dpg_add_layer_norm(_operand(x), _operand(residual), weight, bias, eps=eps, p=p, seed=seed, step=step,
                               out_dtype=out_dtype)
        total = n.sum.view(x.shape)
        ctx.save_for_backward(total, weight, n.mean, n.rstd, _mask_step(p, step))
        ctx.drop, ctx.x_dtype = (p, seed), x.dtype
        ctx.set_materialize_grads(False)
        return n.y.view(x.shape), total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum):
        total, weight, mean, rstd, step = ctx.saved_tensors
        need, (p, seed), shape = ctx.needs_input_grad, ctx.drop, total.shape
        if dy is None and dsum is None:
            return (None,) * 9
        if dy is None:
            # nothing came through the norm
            dx = dpg_dropout(_rows(dsum), p, seed, step=step, out_dtype=ctx.x_dtype).view(shape) if need[0] else None
            return (dx, dsum if need[1] else None) + (None,) * 7
        d = dpg_add_layer_norm_dgrad(_rows(dy), _rows(total), mean, rstd, weight,
                                     dsum=None if dsum is None else _rows(dsum), p=p, seed=seed, step=step,
                                     x_dtype=ctx.x_dtype, weight_grads=need[2] or need[3])
        return (d.dx.view(shape) if need[0] else None, d.dresidual.view(shape) if need[1] else None,
                d.dweight if need[2] else None, d.dbias if need[3] else None) + (None,) * 5


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, step, residual):
        if residual is not None:
            _same_shape(x, residual)
        ctx.save_for_backward(_mask_step(p, step))
        ctx.drop, ctx.x_dtype = (p, seed), x.dtype
        y = dpg_dropout(_operand(x), p, seed, step=step, residual=None if residual is None else _operand(residual))
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (step,) = ctx.saved_tensors
        dx = None
        if ctx.needs_input_grad[0]:
            dx = dpg_dropout(_rows(dy), *ctx.drop, step=step, out_dtype=ctx.x_dtype).view(dy.shape)
        return dx, None, None, None, dy if ctx.needs_input_grad[4] else None


def _sequences(t):
    """t itself where all its rows are aligned and one stride apart, else a copy."""
    if t.dim() == 2:
        return _operand(t)
    b, n, d = t.shape
    last = d <= 1 or t.stride(2) == 1
    even = n <= 1 or (t.stride(1) >= d and (b <= 1 or t.stride(0) == n * t.stride(1)))
    taken = last and even and (n > 1 or b <= 1 or t.stride(0) >= d)
    taken = taken and _aligned(t, t.stride(1) if n > 1 else t.stride(0) if b > 1 else 0)
    return t if taken else t.clone(memory_format=torch.contiguous_format)


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, offsets, state, coupled):
        gate, x = _sequences(gate), _sequences(x)
        r = dpg_recurrence(gate, x, offsets=offsets, state=state, coupled=coupled, carries=any(ctx.needs_input_grad))
        ctx.save_for_backward(gate, x, r.carries, offsets, state)
        ctx.coupled = coupled
        ctx.set_materialize_grads(False)
        return r.h, r.state

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dstate):
        gate, x, carries, offsets, state = ctx.saved_tensors
        if dh is None and dstate is None:
            return (None,) * 5
        dh = torch.zeros_like(x) if dh is None else _sequences(dh)
        d = dpg_recurrence_dgrad(dh, gate, x, carries, offsets=offsets, state=state,
                                 dstate=None if dstate is None else _packed(dstate), coupled=ctx.coupled)
        return d.dgate, d.dx, None, d.dstate, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=None):
    """dpg_layer_norm over the last dimension of x [..., H]; differentiable in x
    (gradient of x's type), weight and bias (FP32)."""
    return _LayerNorm.apply(x, weight, bias, eps, out_dtype)


def add_layer_norm(x, residual, weight=None, bias=None, eps=1e-5, p=0.0, seed=0, step=None, out_dtype=None):
    """(y, sum) of dpg_add_layer_norm on [..., H]: the residual stream that goes on
    and its norm; differentiable in x, residual, weight and bias.  Pass p=0 in
    evaluation."""
    return _AddLayerNorm.apply(x, residual, weight, bias, eps, p, seed, step, out_dtype)


def dropout(x, p, seed, step=None, residual=None):
    """dpg_dropout on [..., H]; differentiable in x and residual."""
    return _Dropout.apply(x, p, seed, step, residual)


def recurrence(gate, x, offsets=None, state=None, coupled=True):
    """(h, state) of dpg_recurrence on [B, T, D], or [R, D] with offsets;
    differentiable in gate, x and state."""
    return _Recurrence.apply(gate, x, offsets, state, bool(coupled))


class CheckpointedStep:
    """One checkpointed training step of a projection with prepared launches:
    forward, recomputed forward, input gradient and weight gradient of
    x[T, K], w[N, K] and the incoming gradient dy[T, N], into static outputs
    (y, y_recomputed, dx, dw) of dtype ``out_dtype``, captured in one HIP
    graph on first use.  The caller refreshes the inputs in place (copy_) and
    calls ``replay()``; ``eager()`` issues the same launches without the graph.
    """

    def __init__(self, x, w, dy, out_dtype=torch.float32, deterministic=True):
        self.x, self.w, self.dy = x, w, dy
        T, K = x.shape
        N = w.shape[0]
        dev = x.device
        self.deterministic = resolve_deterministic(deterministic)
        self.y = torch.empty((T, N), dtype=out_dtype, device=dev)
        self.y2 = torch.empty((T, N), dtype=out_dtype, device=dev)
        self.dx = torch.empty((T, K), dtype=out_dtype, device=dev)
        self.dw = torch.empty((N, K), dtype=out_dtype, device=dev)

        def ws(pass_):
            n = workspace_size(pass_, T, N, K, out_dtype, self.deterministic, 0)
            return torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        # the two forwards run back to back on one stream and may share a workspace
        self.ws = {PASS_FORWARD: ws(PASS_FORWARD), PASS_DGRAD: ws(PASS_DGRAD), PASS_WGRAD: ws(PASS_WGRAD)}
        self.graph = None

    def eager(self):
        d = self.deterministic
        dpg_forward(self.x, self.w, out=self.y, deterministic=d, workspace=self.ws[PASS_FORWARD])
        dpg_forward(self.x, self.w, out=self.y2, deterministic=d, workspace=self.ws[PASS_FORWARD])
        dpg_dgrad(self.dy, self.w, out=self.dx, deterministic=d, workspace=self.ws[PASS_DGRAD])
        dpg_wgrad(self.dy, self.x, out=self.dw, deterministic=d, workspace=self.ws[PASS_WGRAD])
        return self.y, self.y2, self.dx, self.dw

    def replay(self):
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.eager()  # plans resolved and cached before capture
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.eager()
        self.graph.replay()
        return self.y, self.y2, self.dx, self.dw
