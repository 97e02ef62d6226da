"""The grouped products' large tiles on the GPU: whole numbers whose sums are exact
in FP32, compared bit for bit, as in test_gpu_grouped.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)


@pytest.mark.parametrize("N,out_dtype", [(1 << 24, torch.float32), (1 << 25, torch.bfloat16), (8454144 + 8, torch.float32),
                                         ((1 << 29) + 1032, torch.float32), ((1 << 30) + 1032, torch.bfloat16)])
def test_one_row_of_very_many_columns(N, out_dtype):
    """The 32-bit offsets of the tile's rows past the only one pass 2^32 from 8.45
    million FP32 columns on, the columns to the right 2^31 bytes from 2^29 on."""
    value = torch.arange(N, dtype=torch.int32, device="cuda").remainder_(251).to(torch.bfloat16)
    w = torch.zeros(1, N, 8, dtype=torch.bfloat16, device="cuda")
    w[0, :, 3] = value
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 3] = 1
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = torch.full((1, N), 7.0, dtype=out_dtype, device="cuda")
    dpg.dpg_grouped_forward(x, w, off, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[0].to(torch.bfloat16), value)  # at most 250: exact in both types
