"""The recurrence's weights and their products where FP32 ends: gates whose forget
weight is below the normal numbers, and large finite states across runs of rows
whose product of weights is.

Tolerances: the bounds of block_reference plus the rounding to the output's type,
and what a test's comment adds to them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_reference as ref  # noqa: E402
from test_gpu_recurrence import BF16, F32, _check, _compare, _run  # noqa: E402

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


@pytest.mark.parametrize("T, at, n", [(40, 8, 8), (768, 8, 8), (768, 128, 8), (768, 128, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
def test_a_large_state_does_not_outlive_its_weights(coupled, dtype, T, at, n):
    """A state of 1e37 that `at` rows hold, then n rows of gate -20, eight of which
    have a product of 10^-70; and the same from the end for the gradient.  Products of
    weights are FP32 numbers: every one of at most T multiplications and minima is off
    by 2^-149 below the normal numbers, and what it multiplies, by that part of 1e37."""
    D, big = 24, 1e37
    g = torch.Generator().manual_seed(3)
    gate = torch.rand(T, D, generator=g) + 6
    gate[:at] = gate[T - at:] = 20
    gate[at:at + n] = gate[T - at - n:T - at] = -20
    d = {"gate": gate.to(dtype).cuda(), "x": _uniform(g, T, D, dtype=dtype), "dh": _uniform(g, T, D, dtype=dtype)}
    for k in ("state", "dstate"):
        d[k] = torch.full((1, D), big, device="cuda")
    r, b = _run(d, [0, T], coupled)
    h = {k: ref.host(v) for k, v in d.items()}
    want = ref.recurrence(h["gate"], h["x"], [0, T], h["state"], coupled, h["dh"], h["dstate"])
    leak = big * T * 2.0 ** -149
    _check("h", r.h, want["h"], want["e_h"] + leak, dtype)
    _check("state", r.state, want["state"], want["e_state"] + leak, F32)
    _check("dx", b.dx, want["dx"], want["e_dx"] + leak, dtype)
    _check("dstate", b.dstate, want["dstate"], want["e_dstate"] + leak, F32)
    # between both: r off by the leak, times h and x, and h off by it, times r, all below 50, times f (1 - f)
    inside = slice(at + n, T - at - n)
    _check("dgate", b.dgate[inside], want["dgate"][inside], want["e_dgate"][inside] + 25 * leak, dtype)
    assert leak < 2e-5 and np.abs(want["h"][inside]).max() < 49 and (coupled or np.abs(want["dx"][inside]).max() < 50)
