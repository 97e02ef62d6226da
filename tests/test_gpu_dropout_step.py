"""A dropout's step and its backward pass: needed where there is a mask, and only
there."""
import pytest
import torch

pytestmark = pytest.mark.gpu

pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402

CALLS = {"dropout": lambda x, p, step: dag.dropout(x, p, 1, step=step),
         "dropout, residual": lambda x, p, step: dag.dropout(x, p, 1, step=step, residual=x),
         "sum": lambda x, p, step: dag.add_layer_norm(x, x, p=p, seed=1, step=step)[0],
         "sum alone": lambda x, p, step: dag.add_layer_norm(x, x, p=p, seed=1, step=step)[1]}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_step_counted_up_between_the_passes(name):
    """Two forward passes with the step counted up, then their backward passes:
    with p = 0 no mask depends on it."""
    x = torch.randn(4, 16, generator=torch.Generator().manual_seed(1)).cuda().requires_grad_(True)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    dy = torch.randn(4, 16, generator=torch.Generator().manual_seed(2)).cuda()
    (want,) = torch.autograd.grad(CALLS[name](x, 0.0, None), x, dy)
    losses = []
    for _ in range(2):
        losses.append(CALLS[name](x, 0.0, step))
        step += 1
    for y in losses:
        (got,) = torch.autograd.grad(y, x, dy)
        assert torch.equal(got, want)
    y = CALLS[name](x, 0.5, step)
    step += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.backward(dy)
