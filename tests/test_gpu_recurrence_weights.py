"""The recurrence's weights where FP32 ends: gates whose forget weight is below the
normal numbers.

Tolerances: the bounds of block_reference plus the rounding to the output's type,
and what a test's comment adds to them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_recurrence import BF16, F32, _compare, _run  # noqa: E402

LOW = [-86 - 0.5 * i for i in range(9)]


def _uniform(g, *shape, dtype=F32):
    return (torch.rand(*shape, generator=g) - 0.5).to(dtype).cuda()


@pytest.mark.parametrize("T", [1, 40, 700], ids=["steps", "short", "spans"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
def test_gates_from_86_to_90_below_zero(coupled, dtype, T):
    """Half of the rows have such a gate, the others one of -3 to 1.  f counts as 0
    where it is below the smallest normal number, 1.2e-38; states, gradients and
    inputs of at most a half stay below 2 (f up to 0.74), so that this moves
    nothing by more than the 1e-37 that _check allows."""
    B, D = 5, 72
    g = torch.Generator().manual_seed(T)
    gate = torch.rand(B * T, D, generator=g) * 4 - 3
    low = torch.tensor(LOW)[torch.randint(len(LOW), (B * T, D), generator=g)]
    gate = torch.where(torch.rand(B * T, D, generator=g) < 0.5, low, gate)
    assert all(bool((gate == v).any()) for v in LOW)
    d = {"gate": gate.to(dtype).cuda(), "state": _uniform(g, B, D), "dstate": _uniform(g, B, D)}
    d.update({k: _uniform(g, B * T, D, dtype=dtype) for k in ("x", "dh")})
    offsets = [T * i for i in range(B + 1)]
    _compare(d, offsets, coupled, *_run(d, offsets, coupled, (B, T, D)))
    _compare(d, offsets, coupled, *_run(d, offsets, coupled))
