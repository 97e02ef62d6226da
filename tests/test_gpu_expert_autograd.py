"""What autograd makes of the expert-layer functions beyond one backward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402


def _bf16(*shape):
    return torch.randn(*shape, device="cuda").to(torch.bfloat16).requires_grad_(True)


@pytest.mark.parametrize("name", ["route", "dispatch", "grouped_projection", "combine"])
def test_a_second_derivative_raises(name):
    """The gradients come from kernels that autograd does not see: as constants
    they would give wrong second derivatives without a word."""
    logits = torch.randn(12, 4, device="cuda", requires_grad=True)
    r = dpg.dpg_route(logits.detach(), 2)
    if name == "route":
        leaf, out = logits, dag.route(logits, 2).weights
    elif name == "dispatch":
        leaf = _bf16(12, 64)
        out = dag.dispatch(leaf, r)
    elif name == "grouped_projection":
        leaf = _bf16(24, 64)
        out = dag.grouped_projection(leaf, _bf16(4, 64, 64), r.offsets)
    else:
        leaf = _bf16(24, 64)
        out = dag.combine(leaf, r._replace(weights=r.weights.requires_grad_(True)))
    grad, = torch.autograd.grad(out.float().square().sum(), leaf, create_graph=True)
    assert bool(torch.isfinite(grad).all())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (out.float().sum() + grad.float().square().sum()).backward()  # a penalty on the gradient
