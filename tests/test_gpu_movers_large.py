"""Routing, row movement and AdamW at the sizes of mover_cases.py, where the
kernels of large calls run: the checks of test_gpu_route.py and test_gpu_adamw.py,
with their bounds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import mover_cases  # noqa: E402
import test_gpu_adamw as adamw  # noqa: E402
import test_gpu_route as route  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", mover_cases.ROUTES)
def test_choice_and_order(T, E, k, renorm):
    """Real values, and among them rows with ties, masks, NaN and lowest values:
    at the start, around the border of two blocks and at the end."""
    g = torch.Generator().manual_seed(E)
    lg = torch.randn(T, E, generator=g) * 2
    lg[::5] = torch.randint(-2, 3, (len(lg[::5]), E), generator=g).float()
    for t in (0, 60, T - 8):
        lg[t] = -INF                                       # nothing left
        lg[t + 1, 3:] = -INF                               # three left
        lg[t + 2] = torch.finfo(torch.float32).min         # the lowest value masks nothing
        lg[t + 3, E // 2] = NAN
        lg[t + 4] = NAN
        lg[t + 5] = -INF
        lg[t + 5, E - 1] = -3.0
        lg[t + 6] = 0.0
        lg[t + 6, ::2] = -0.0
        lg[t + 7] = -INF
        lg[t + 7, 2] = NAN
    r = route._check_route(lg.cuda(), k, renorm)
    for t in (0, 60, T - 8):
        assert r.experts[t].tolist() == [-1] * k and r.experts[t + 2].tolist() == list(range(k))


@pytest.mark.parametrize("renorm", [True, False])
def test_ties_masks_and_strange_values(renorm):
    route.test_ties_masks_and_strange_values(1500, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,masked", [(1100, 100, 10, 0.2), (1030, 300, 17, 0.9)])
def test_route_gradient(T, E, k, masked, renorm):
    route.test_route_gradient(T, E, k, masked, renorm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H,pad", mover_cases.STREAMED)
def test_streamed_rows_there_and_back(T, k, H, pad, dtype):
    """Rows that pass the caches by; a part of the slots has no expert."""
    route.test_rows_there_and_back(T, k, H, 64, pad, dtype)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 3])
def test_adamw_of_many_elements(monkeypatch, e4m3, grad_dtype, shift):
    """Aligned tensors and ones that start three elements into a buffer."""
    monkeypatch.setattr(adamw, "SIZES", mover_cases.ADAMW)
    adamw.test_step(e4m3, grad_dtype, 7, shift)
