"""Workspaces that the expert-layer entry points refuse: views whose bytes do not
follow each other.  Every call here is refused before a launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)


@pytest.mark.parametrize("view", ["expanded", "columns"])
def test_workspaces_with_overlaps_or_gaps(view):
    off = torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    dy = torch.zeros(3000, 264, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(3000, 136, dtype=torch.bfloat16, device="cuda")
    if view == "expanded":
        ws = torch.zeros(16, dtype=torch.uint8, device="cuda")[:1].expand(1 << 24)
    else:
        ws = torch.zeros(1 << 12, 1 << 13, dtype=torch.uint8, device="cuda")[:, :1 << 12]
    calls = [lambda: dpg.dpg_grouped_wgrad(dy, x, off, workspace=ws),
             lambda: dpg.dpg_grouped_forward(x, torch.zeros(1, 264, 136, dtype=torch.bfloat16, device="cuda"), off,
                                             workspace=ws),
             lambda: dpg.dpg_route(torch.zeros(3000, 16, device="cuda"), 2, workspace=ws)]
    for call in calls:
        with pytest.raises(ValueError, match="contiguous"):
            call()
