"""AdamW's 8-bit moments on the GPU: what one element that is not finite does to
the block of 256 whose scale it shares."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _state(n, seed):
    g = torch.Generator().manual_seed(seed)
    blocks = -(-n // 256)
    return {"params": [torch.randn(n, generator=g).cuda()],
            "exp_avgs": [(torch.randn(n, generator=g) * 50).to(torch.float8_e4m3fn).cuda()],
            "exp_avg_sqs": [(torch.rand(n, generator=g) * 200 + 1).to(torch.float8_e4m3fn).cuda()],
            "avg_scales": [torch.full((blocks,), 2.0 ** -14, device="cuda")],
            "sq_scales": [torch.full((blocks,), 2.0 ** -14, device="cuda")]}


def _bits(s, name):
    return s[name][0].view(torch.uint8)


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("strange", [float("inf"), -float("inf"), float("nan")])
def test_a_strange_gradient_is_lost_alone(strange, grad_dtype):
    """Three steps beside a run whose element has a gradient of zero and empty
    moments: every other element, its codes and the scales are the same bits."""
    n, bad = 700, 300
    g = torch.Generator().manual_seed(1)
    grads = [(torch.randn(n, generator=g) * 0.01).to(grad_dtype).cuda() for _ in range(3)]
    a, b = _state(n, 2), _state(n, 2)
    for s in (a, b):
        _bits(s, "exp_avgs")[bad] = _bits(s, "exp_avg_sqs")[bad] = 0
    others = torch.arange(n, device="cuda") != bad
    for step, grad in enumerate(grads, 1):
        plain, hit = grad.clone(), grad.clone()
        plain[bad] = 0
        if step == 1:
            hit[bad] = strange
        dpg.dpg_adamw(grads=[hit], step=step, seed=step, **a, **HYPER)
        dpg.dpg_adamw(grads=[plain], step=step, seed=step, **b, **HYPER)
        for name in ("avg_scales", "sq_scales"):
            assert torch.equal(a[name][0], b[name][0]), (step, name)
        for name in ("exp_avgs", "exp_avg_sqs"):
            assert torch.equal(_bits(a, name)[others], _bits(b, name)[others]), (step, name)
            assert int(_bits(a, name)[bad]) & 127 == 127
        assert torch.equal(a["params"][0][others], b["params"][0][others]), step
        assert bool(torch.isfinite(a["params"][0][others]).all())


def test_a_square_past_fp32_leaves_the_other_roots():
    """A finite gradient of 1e20, whose square is infinite in FP32: the block's
    roots and their scale are those of a run without it."""
    n, bad = 512, 17
    g = torch.Generator().manual_seed(3)
    a, b = _state(n, 4), _state(n, 4)
    for s in (a, b):
        _bits(s, "exp_avgs")[bad] = _bits(s, "exp_avg_sqs")[bad] = 0
    others = torch.arange(n, device="cuda") != bad
    for step in (1, 2, 3):
        plain = (torch.randn(n, generator=g) * 0.01).cuda()
        plain[bad] = 0
        hit = plain.clone()
        if step == 1:
            hit[bad] = 1e20
        dpg.dpg_adamw(grads=[hit], step=step, seed=step, **a, **HYPER)
        dpg.dpg_adamw(grads=[plain], step=step, seed=step, **b, **HYPER)
        assert torch.equal(a["sq_scales"][0], b["sq_scales"][0])
        assert torch.equal(_bits(a, "exp_avg_sqs")[others], _bits(b, "exp_avg_sqs")[others])
        assert bool(torch.isfinite(a["params"][0][others]).all())
