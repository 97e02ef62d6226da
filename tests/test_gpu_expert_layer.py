"""The expert-layer operators together: autograd wrappers, the whole layer's
gradients against 64-bit autograd with the routing held, and the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _inputs(T, E, H, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(E, N, H, generator=g) * H ** -0.5).to(torch.bfloat16).cuda()
    dy = torch.randn(T, N, generator=g).to(torch.bfloat16).cuda()
    return logits, x, w, dy


@pytest.mark.parametrize("renormalize", [True, False])
def test_autograd_equals_the_entry_points(renormalize):
    T, E, H, N, k = 70, 9, 128, 72, 3
    logits, x, w, dy = _inputs(T, E, H, N)
    logits[3] = -float("inf")
    for t in (logits, x, w):
        t.requires_grad_(True)
    r = dag.route(logits, k, renormalize)
    xs = dag.dispatch(x, r)
    ys = dag.grouped_projection(xs, w, r.offsets)
    y = dag.combine(ys, r)
    y.backward(dy)
    assert not (r.experts.requires_grad or r.offsets.requires_grad or r.positions.requires_grad)
    with torch.no_grad():
        q = dpg.dpg_route(logits, k, renormalize=renormalize)
        qs = dpg.dpg_dispatch(x, q.positions, q.offsets)
        zs = dpg.dpg_grouped_forward(qs, w, q.offsets)
        assert torch.equal(y, dpg.dpg_combine(zs, q.positions, q.offsets, q.weights))
        dys, dweights = dpg.dpg_combine_dgrad(dy, zs, q.positions, q.offsets, q.weights)
        assert torch.equal(w.grad, dpg.dpg_grouped_wgrad(dys, qs, q.offsets))
        assert torch.equal(x.grad, dpg.dpg_combine(dpg.dpg_grouped_dgrad(dys, w, q.offsets), q.positions, q.offsets))
        assert torch.equal(logits.grad, dpg.dpg_route_dgrad(logits, q.experts, q.weights, dweights,
                                                            renormalize=renormalize))
    assert bool((logits.grad[3] == 0).all()) and bool((x.grad[3] == 0).all())


def test_an_expanded_gradient():
    """sum().backward() hands over a gradient without strides of its own."""
    logits, x, w, _ = _inputs(20, 4, 64, 64)
    r = dpg.dpg_route(logits, 2)
    w.requires_grad_(True)
    y = dag.combine(dag.grouped_projection(dag.dispatch(x, r), w, r.offsets), r)
    y.sum().backward()
    ones = torch.ones(20, 64, dtype=torch.bfloat16, device="cuda")
    dys, _ = dpg.dpg_combine_dgrad(ones, torch.zeros(40, 64, dtype=torch.bfloat16, device="cuda"), r.positions,
                                   r.offsets, r.weights)
    assert torch.equal(w.grad, dpg.dpg_grouped_wgrad(dys, dpg.dpg_dispatch(x, r.positions, r.offsets), r.offsets))


def test_layer_gradients_against_64_bits():
    """One expert layer without activation.  Values rounded to BF16 on the way
    (each off by 2^-8 of its size at most): xs exact, ys once, y once; backward
    dys once, dx's terms and dx once each, dw once.  FP32 sums add less than
    2^-15 of the magnitudes (128 terms of 2^-24 each, twice)."""
    T, E, H, N, k = 96, 6, 128, 64, 3
    logits, x, w, dy = _inputs(T, E, H, N, seed=2)
    r = dpg.dpg_route(logits, k)
    lg, xx, ww = (t.double().cpu().requires_grad_(True) for t in (logits, x, w))
    ex = r.experts.long().cpu()
    q = torch.softmax(torch.gather(lg, 1, ex), 1)
    terms = torch.einsum("tjnh,th->tjn", ww[ex], xx)
    (terms * q[..., None]).sum(1).backward(dy.double().cpu())
    for t in (logits, x, w):
        t.requires_grad_(True)
    r = dag.route(logits, k)
    y = dag.combine(dag.grouped_projection(dag.dispatch(x, r), w, r.offsets), r)
    y.backward(dy)
    with torch.no_grad():
        d = dy.double().cpu()
        h, small = 2.0 ** -8, 2.0 ** -15
        # sums of magnitudes: what each rounding is a part of
        mag_w = torch.zeros(E, N, H, dtype=torch.float64)
        mag_x = torch.zeros(T, H, dtype=torch.float64)
        part_x = torch.zeros(T, H, dtype=torch.float64)
        for j in range(k):
            dj = d.abs() * q[:, j:j + 1]
            mag_w.index_add_(0, ex[:, j], dj[:, :, None] * xx.abs()[:, None, :])
            mag_x += torch.einsum("tn,tnh->th", dj, ww[ex[:, j]].abs())
            part_x += torch.einsum("tn,tnh->th", d * q[:, j:j + 1], ww[ex[:, j]]).abs()
        limit_w = (h + small) * mag_w + h * (ww.grad.abs() + h * mag_w)
        assert bool(((w.grad.double().cpu() - ww.grad).abs() <= limit_w).all())
        limit_x = (h + small) * mag_x + h * (part_x + h * mag_x) + 2 * h * (xx.grad.abs() + 2 * h * mag_x)
        assert bool(((x.grad.double().cpu() - xx.grad).abs() <= limit_x).all())
        # dweights: ys once, then an FP32 sum; dlogits = q (dw - sum q dw)
        dw_err = ((h + small) * (terms.abs() * d.abs()[:, None]).sum(2)).max(1, keepdim=True).values
        limit_l = 2.0 * dw_err * (1 + 2.0 ** -12) + 2.0 ** -18 * (terms.abs() * d.abs()[:, None]).sum(2).max(1, keepdim=True).values
        assert bool(((logits.grad.double().cpu() - lg.grad).abs() <= limit_l).all())


@pytest.mark.parametrize("pass_", ["x", "w"])
def test_grouped_gradients_against_differences(pass_):
    """The products are linear: with whole numbers the difference of <y, dy> over
    a step of one is the gradient exactly."""
    g = np.random.default_rng(3)
    counts, N, K = [5, 0, 40, 3], 24, 40
    R = sum(counts)
    ints = lambda *s: torch.from_numpy(g.integers(-4, 5, s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    x, w, dy = ints(R, K), ints(4, N, K), ints(R, N)
    off = torch.tensor([0, 5, 5, 45, 48], dtype=torch.int32, device="cuda")
    value = lambda: float((dpg.dpg_grouped_forward(x, w, off, out_dtype=torch.float32).double() * dy.double()).sum())  # noqa: E731
    if pass_ == "x":
        grad, t, places = dpg.dpg_grouped_dgrad(dy, w, off, out_dtype=torch.float32), x, [(0, 0), (7, 39), (47, 11)]
    else:
        grad, t, places = dpg.dpg_grouped_wgrad(dy, x, off, out_dtype=torch.float32), w, [(0, 3, 2), (2, 23, 39), (3, 0, 0), (1, 1, 1)]
    base = value()
    for at in places:
        old = t[at].clone()
        t[at] += 1
        assert value() - base == float(grad[at])
        t[at] = old


def test_example_trains():
    spec = importlib.util.spec_from_file_location("expert_layer_example", os.path.join(ROOT, "examples", "expert_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.main(steps=40, tokens=256, experts=8, hidden=128, inner=256, top_k=2)
    assert np.isfinite(losses).all() and losses[-1] < 0.7 * losses[0]
    # the same run gives the same bits
    assert example.main(steps=6, tokens=256, experts=8, hidden=128, inner=256, top_k=2) == losses[:6]
