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


def _layer(logits, x, w, k):
    r = dag.route(logits, k)
    y = dag.combine(dag.grouped_projection(dag.dispatch(x, r), w, r.offsets), r)
    return r, y


@pytest.mark.parametrize("lead", [(2, 3, 5), (4, 1, 9), (1,), (), (0, 3)])
def test_leading_dimensions(lead):
    """Any leading shape, as the projections take: the same bits as for the
    tokens in one row of them, gradients in the inputs' shapes."""
    T, E, H, N, k = int(torch.tensor(lead).prod()) if lead else 1, 4, 64, 72, 3
    flat = [torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda").to(torch.bfloat16),
            torch.randn(E, N, H, device="cuda").to(torch.bfloat16)]
    shaped = [flat[0].reshape(*lead, E).clone(), flat[1].reshape(*lead, H).clone(), flat[2].clone()]
    for t in flat + shaped:
        t.requires_grad_(True)
    r, y = _layer(*flat, k)
    q, z = _layer(*shaped, k)
    assert z.shape == (*lead, N)
    assert q.experts.shape == q.weights.shape == q.positions.shape == (*lead, k)
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(q, r)) and torch.equal(z.reshape(T, N), y)
    dy = torch.randn(T, N, device="cuda").to(torch.bfloat16)
    y.backward(dy)
    z.backward(dy.reshape(z.shape))
    for a, b in zip(shaped, flat):
        assert a.grad.shape == a.shape and torch.equal(a.grad.reshape(b.shape), b.grad)


def test_expanded_and_transposed_inputs():
    """One row of logits for all tokens, and tokens that are columns in memory: the
    gradients are those of a copy, summed over the broadcast tokens."""
    T, E, H, N, k = 10, 4, 64, 72, 2
    row = torch.randn(1, E, device="cuda", requires_grad=True)
    cols = torch.randn(H, T, device="cuda").to(torch.bfloat16).requires_grad_(True)
    w = torch.randn(E, N, H, device="cuda").to(torch.bfloat16)
    dy = torch.randn(T, N, device="cuda").to(torch.bfloat16)
    _, y = _layer(row.expand(T, E), cols.t(), w, k)
    y.backward(dy)
    logits = row.detach().expand(T, E).contiguous().requires_grad_(True)
    x = cols.detach().t().contiguous().requires_grad_(True)
    _, z = _layer(logits, x, w, k)
    z.backward(dy)
    assert torch.equal(y, z) and torch.equal(cols.grad, x.grad.t())
    assert torch.equal(row.grad, logits.grad.sum(0, keepdim=True))
