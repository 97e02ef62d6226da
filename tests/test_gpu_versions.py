"""Writes of the expert-layer entry points into a caller's tensors are seen by
autograd: their versions go up, and a backward pass that saved one raises."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402


def _adamw(n, e4m3, copies):
    zeros = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    s = {"params": [zeros(n)], "exp_avgs": [zeros(n)], "exp_avg_sqs": [zeros(n)]}
    if e4m3:
        for name in ("exp_avgs", "exp_avg_sqs"):
            s[name] = [t.to(torch.float8_e4m3fn) for t in s[name]]
        s["avg_scales"], s["sq_scales"] = [zeros(-(-n // 256)) + 1], [zeros(-(-n // 256)) + 1]
    if copies:
        s["copies"] = [zeros(n).to(torch.bfloat16)]
    return s


@pytest.mark.parametrize("e4m3,copies", [(False, False), (False, True), (True, True)])
def test_a_step_raises_the_versions_of_what_it_writes(e4m3, copies):
    s = _adamw(300, e4m3, copies)
    grad = torch.ones(300, device="cuda")
    before = {k: v[0]._version for k, v in s.items()}, grad._version
    dpg.dpg_adamw(grads=[grad], lr=1e-3, **s)
    assert {k: v[0]._version - before[0][k] for k, v in s.items()} == {k: 1 for k in s}
    assert grad._version == before[1]


def test_a_refused_step_raises_no_version():
    s = _adamw(300, False, True)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_adamw(grads=[torch.ones(300, device="cuda")], lr=1e-3, step=0, **s)
    assert all(v[0]._version == 0 for v in s.values())


def test_a_backward_pass_after_a_step_on_its_weights_raises():
    x = torch.randn(20, 64, device="cuda").to(torch.bfloat16).requires_grad_(True)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    s = _adamw(64 * 64, False, True)
    w = s["copies"][0].view(1, 64, 64)
    y = dag.grouped_projection(x, w, off)
    dpg.dpg_adamw(grads=[torch.ones(64 * 64, device="cuda")], lr=1e-3, **s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(torch.ones_like(y))


def test_given_outputs():
    lg = torch.randn(10, 4, device="cuda")
    r = dpg.dpg_route(lg, 2)
    x = torch.randn(10, 64, device="cuda").to(torch.bfloat16)
    w = torch.randn(4, 64, 64, device="cuda").to(torch.bfloat16)
    xs = dpg.dpg_dispatch(x, r.positions, r.offsets)
    for call, shape, dtype in (
            (lambda out: dpg.dpg_grouped_forward(xs, w, r.offsets, out=out), (20, 64), torch.bfloat16),
            (lambda out: dpg.dpg_grouped_dgrad(xs, w, r.offsets, out=out), (20, 64), torch.float32),
            (lambda out: dpg.dpg_grouped_wgrad(xs, xs, r.offsets, out=out), (4, 64, 64), torch.float32),
            (lambda out: dpg.dpg_dispatch(x, r.positions, r.offsets, out=out), (20, 64), torch.bfloat16),
            (lambda out: dpg.dpg_combine(xs, r.positions, r.offsets, r.weights, out=out), (10, 64), torch.float32),
            (lambda out: dpg.dpg_route_dgrad(lg, r.experts, r.weights, r.weights, out=out), (10, 4), torch.float32)):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        assert call(out) is out and out._version == 1
        with torch.inference_mode():
            out = torch.empty(shape, dtype=dtype, device="cuda")
        call(out)  # has no version: written all the same
    assert all(t._version == 0 for t in (xs, x, w, lg, *r))
