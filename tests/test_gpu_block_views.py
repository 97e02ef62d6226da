"""The training wrappers of layer norm, dropout and the recurrence on views: inputs
and gradients that start, or whose rows start, at no multiple of 16 bytes, as a
part of a concatenation does.  The bits are those of aligned copies."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
B, T, D = 3, 11, 24


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def _odd(t, how):
    """The values of t as a view with other strides, or another start."""
    if how == "wide":        # rows 4 elements too long
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 4, dtype=t.dtype, device="cuda")
        at = wide[..., :t.shape[-1]]
    elif how == "inside":    # and from the fourth element on
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 8, dtype=t.dtype, device="cuda")
        at = wide[..., 2:t.shape[-1] + 2]
    else:                    # contiguous, from the first element of a vector on
        at = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    at.copy_(t)
    return at


CALLS = {
    "layer norm": (lambda x, r, w: (dag.layer_norm(x, w),), 1),
    "sum": (lambda x, r, w: dag.add_layer_norm(x, r, w, p=0.25, seed=3), 2),
    "dropout": (lambda x, r, w: (dag.dropout(x, 0.25, 3, residual=r),), 1),
    "recurrence": (lambda x, r, w: dag.recurrence(x, r, state=w.expand(B, D).contiguous()), 2),
}


def _inputs(dtype, shape):
    g = torch.Generator().manual_seed(1)
    return _randn(g, *shape, dtype=dtype), _randn(g, *shape, dtype=dtype), 1 + _randn(g, shape[-1])


def _gradients(call, leaves, views, seeds):
    outs = call(*views)
    torch.autograd.backward(outs, seeds(outs))
    return [o.detach() for o in outs] + [v.grad for v in leaves]


@pytest.mark.parametrize("how", ["wide", "inside", "start"])
@pytest.mark.parametrize("shape", [(B, T, D), (B, 1, D), (1, T, D)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(CALLS))
def test_views_as_inputs_and_gradients(name, dtype, shape, how):
    call, outputs = CALLS[name]
    if name == "recurrence":
        call = lambda x, r, w: dag.recurrence(x, r, state=w.expand(shape[0], D).contiguous())  # noqa: E731
    values = _inputs(dtype, shape)
    g = torch.Generator().manual_seed(2)
    plain = [v.clone().requires_grad_(True) for v in values]
    given = []

    def seeds(outs):
        given.extend(_randn(g, *o.shape, dtype=o.dtype) for o in outs)
        return tuple(given)
    want = _gradients(call, plain, plain, seeds)
    assert len(given) == outputs
    odd = [_odd(v, how).requires_grad_(True) for v in values[:2]] + [values[2].clone().requires_grad_(True)]
    got = _gradients(call, odd, odd, lambda outs: tuple(_odd(v, how) for v in given))
    assert all((a is None) == (b is None) and (a is None or torch.equal(a, b)) for a, b in zip(want, got))


def test_outputs_in_a_concatenation():
    """What torch hands back for parts of one vector, and of one matrix."""
    x, r, w = _inputs(BF16, (B, T, D))
    x.requires_grad_(True)
    h, state = dag.recurrence(x, r)
    beside = torch.cat([torch.ones(B, T, 4, dtype=BF16, device="cuda"), h], 2)
    behind = torch.cat([torch.ones(1, device="cuda"), state.flatten()])
    dh, ds = torch.randn_like(beside), torch.randn_like(behind)
    torch.autograd.backward((beside, behind), (dh, ds))
    k = dpg.dpg_recurrence(x.detach(), r, carries=True)
    d = dpg.dpg_recurrence_dgrad(dh[..., 4:].contiguous(), x.detach(), r, k.carries, dstate=ds[1:].clone().view(B, D))
    assert torch.equal(x.grad, d.dgate)
    y = dag.projection(x.detach(), torch.ones(8, D, dtype=BF16, device="cuda", requires_grad=True))
    torch.cat([torch.ones(1, dtype=BF16, device="cuda"), y.flatten()]).sum().backward()
