"""AdamW on the GPU against the definition in 64 bits, in both moment types."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

EPS32 = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 3, 255, 256, 257, 0, 4096, 4097, 1000, 70001]


def _lists(sizes, grad_dtype, e4m3, seed=0, shift=0):
    """Tensors of the given sizes, each `shift` elements into its own buffer."""
    g = torch.Generator().manual_seed(seed)

    def make(scale, dtype=torch.float32, positive=False):
        out = []
        for n in sizes:
            v = torch.randn(n + shift, generator=g) * scale
            out.append((v.abs() if positive else v).to(dtype).cuda()[shift:])
        return out
    s = {"params": make(0.5), "grads": make(0.01, grad_dtype), "copies": make(1.0, torch.bfloat16)}
    if e4m3:
        s["exp_avgs"] = [t.clamp(-448, 448).to(torch.float8_e4m3fn) for t in make(100.0)]
        s["exp_avg_sqs"] = [t.clamp(0.002, 448).to(torch.float8_e4m3fn) for t in make(100.0, positive=True)]
        for name in ("avg_scales", "sq_scales"):
            s[name] = [torch.exp2(torch.randint(-18, -14, (-(-n // 256),), generator=g).float()).cuda() for n in sizes]
    else:
        s["exp_avgs"], s["exp_avg_sqs"] = make(0.003), make(1e-4, positive=True)
    return s


def _grow(codes, scale):
    return codes.float().double() * scale.double().repeat_interleave(256)[:codes.numel()]


def _expected(s, i, step, grad_scale, e4m3, lr, beta1, beta2, eps, weight_decay):
    p, g = s["params"][i].double(), s["grads"][i].double() * grad_scale
    m, v = s["exp_avgs"][i], s["exp_avg_sqs"][i]
    if e4m3:
        m, v = _grow(m, s["avg_scales"][i]), _grow(v, s["sq_scales"][i]) ** 2
    m = beta1 * m.double() + (1 - beta1) * g
    v = beta2 * v.double() + (1 - beta2) * g * g
    upd = lr * (m / (1 - beta1 ** step)) / (torch.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - upd, m, v, upd


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step,shift", [(1, 0), (7, 0), (7, 3)])
def test_step(e4m3, grad_dtype, step, shift):
    s = _lists(SIZES, grad_dtype, e4m3, shift=shift)
    scale = torch.tensor([0.75], device="cuda")
    want = [_expected(s, i, step, 0.75, e4m3, **HYPER) for i in range(len(SIZES))]
    before = {k: [t.clone() for t in v] for k, v in s.items()}
    dpg.dpg_adamw(**s, step=step, grad_scale=scale, seed=5, **HYPER)
    torch.cuda.synchronize()
    for i, (p, m, v, upd) in enumerate(want):
        # m, v: three or four FP32 roundings of terms no larger than the two that are added
        g = before["grads"][i].double() * 0.75
        size_m = m.abs() + 2 * 0.1 * g.abs()
        # the update: m's error over the root, and some ten roundings of its own
        m_err = 6 * EPS32 * size_m
        u_err = upd.abs() * 24 * EPS32 + HYPER["lr"] * m_err / (1 - 0.9 ** step) / (torch.sqrt(v / (1 - 0.95 ** step)) + 1e-8)
        got = s["params"][i].double()
        assert bool(((got - p).abs() <= 4 * EPS32 * p.abs() + 4 * EPS32 * before["params"][i].double().abs() + u_err).all()), i
        assert torch.equal(s["copies"][i], s["params"][i].to(torch.bfloat16))
        assert torch.equal(s["grads"][i], before["grads"][i])
        if not e4m3:
            assert bool(((s["exp_avgs"][i].double() - m).abs() <= m_err).all())
            assert bool(((s["exp_avg_sqs"][i].double() - v).abs() <= 8 * EPS32 * v).all())
        else:
            # stored values: between the neighbouring codes of the moment, in a block scaled to (224, 448]
            for name, sc, val in (("exp_avgs", "avg_scales", m), ("exp_avg_sqs", "sq_scales", torch.sqrt(v))):
                n = val.numel()
                if n == 0:
                    continue
                top = torch.nn.functional.pad(val.abs(), (0, -n % 256)).view(-1, 256).amax(1)
                assert bool(((top / s[sc][i].double() <= 448 * (1 + 1e-6)) & (top / s[sc][i].double() > 224 * (1 - 1e-6))).all())
                mant, _ = torch.frexp(s[sc][i])
                assert bool((mant == 0.5).all())  # powers of two
                unit = s[sc][i].double().repeat_interleave(256)[:n]
                off = (_grow(s[name][i], s[sc][i]) - val).abs() / unit
                mag = val.abs() / unit
                gap = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
                assert bool((off <= gap * (1 + 1e-4)).all())


def test_all_codes_are_read_as_e4m3():
    """A step with beta1 = 0 for the gradient part: lr = 0, m keeps beta1 times its value."""
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8).cuda()
    m = codes.view(torch.float8_e4m3fn).clone()
    n = m.numel()
    value = m.float().double()
    p = torch.zeros(n, device="cuda")
    # beta2 = 0 and a gradient of 1 make the root 1, so that p = -lr beta1 m (step large: no correction)
    one = torch.ones(1, device="cuda")
    v = torch.zeros(n, device="cuda").to(torch.float8_e4m3fn)
    dpg.dpg_adamw([p], [torch.zeros(n, device="cuda")], [m], [v], lr=1.0, beta1=0.5, beta2=0.5, eps=1.0,
                  weight_decay=0.0, step=60, avg_scales=[one.clone()], sq_scales=[one.clone()])
    assert torch.equal(p.double(), -0.5 * value)  # powers of two: exact


def test_random_rounding_is_unbiased():
    """The mean of many stored values is the moment: within 6 standard errors
    (the spread of one value is at most half a gap)."""
    n = 1 << 16
    target = 0.3137 * 256
    g = torch.full((n,), target, device="cuda")
    g[::256] = 448.0  # every block's largest
    total = 0.0
    for seed in range(4):
        m, v = (torch.zeros(n, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        sc = [torch.ones(n // 256, device="cuda") for _ in range(2)]
        dpg.dpg_adamw([torch.zeros(n, device="cuda")], [g], [m], [v], lr=0.0, beta1=0.0, beta2=0.0, step=1,
                      avg_scales=[sc[0]], sq_scales=[sc[1]], seed=seed)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[::256] = False
        vals, roots = _grow(m, sc[0])[keep], _grow(v, sc[1])[keep]
        assert set(vals.unique().tolist()) == {80.0, 88.0} == set(roots.unique().tolist())
        total += float(vals.mean()) / 4
        # the two moments' random bits are not the same
        assert 0.1 < float(((vals == 88) == (roots == 88)).double().mean()) < 0.99
    assert abs(total - target) <= 6 * 4.0 / math.sqrt(4 * n)


def test_small_roots_are_not_stored_as_zero_and_zeros_stay():
    n = 512
    g = torch.full((n,), 1e-12, device="cuda")
    g[0] = g[256] = 1.0
    g[1] = 0.0
    m, v = (torch.zeros(n, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    sc = [torch.ones(2, device="cuda") for _ in range(2)]
    p = torch.zeros(n, device="cuda")
    dpg.dpg_adamw([p], [g], [m], [v], lr=1e-3, beta1=0.9, beta2=0.999, step=1, avg_scales=[sc[0]], sq_scales=[sc[1]])
    v = v.float()
    assert float(v[1]) == 0 and float(p[1]) == 0
    assert bool((v[2:256] == 2.0 ** -9).all())


def test_blocks_of_zeros_and_strange_gradients():
    for e4m3 in (False, True):
        s = _lists([600], torch.float32, e4m3)
        s["grads"][0][:] = 0
        s["exp_avgs"][0].view(torch.uint8).zero_()
        s["exp_avg_sqs"][0].view(torch.uint8).zero_()
        p = s["params"][0].clone()
        s["grads"][0][300] = float("nan")
        s["grads"][0][301] = float("inf")
        dpg.dpg_adamw(**s, step=1, **HYPER)
        got = s["params"][0]
        ok = torch.ones(600, dtype=torch.bool, device="cuda")
        ok[300:302] = False
        assert bool(torch.isfinite(got[ok]).all()) and not bool(torch.isfinite(got[300:302]).any())
        assert bool(((got[ok] - p[ok] * (1 - 3e-4)).abs() <= 2 * EPS32 * p[ok].abs()).all())
        if e4m3:
            assert s["exp_avgs"][0].view(torch.uint8)[300:302].tolist() == [127, 127]
            assert float(s["avg_scales"][0][0]) == 1.0  # a block of zeros


@pytest.mark.parametrize("count", [1, 48, 49, 130])
def test_many_tensors_and_their_places(count):
    """Across the launches' borders; equal tensors at different places take different random bits, the same call
    the same ones."""
    sizes = [700 + 13 * (i % 7) for i in range(count)]
    a, b = _lists(sizes, torch.float32, True, seed=1), _lists(sizes, torch.float32, True, seed=1)
    want = [_expected(a, i, 3, 1.0, True, **HYPER)[0] for i in range(count)]
    dpg.dpg_adamw(**a, step=3, seed=9, **HYPER)
    dpg.dpg_adamw(**b, step=3, seed=9, **HYPER)
    for k in a:
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for i in range(count):
        assert float((a["params"][i].double() - want[i]).abs().max()) < 1e-6
    same = _lists([5000], torch.float32, True)
    twice = {k: [v[0].clone(), v[0].clone()] for k, v in same.items()}
    dpg.dpg_adamw(**twice, step=3, seed=9, **HYPER)
    assert not torch.equal(twice["exp_avgs"][0].view(torch.uint8), twice["exp_avgs"][1].view(torch.uint8))
    assert torch.equal(twice["params"][0], twice["params"][1])


def test_several_steps_follow_the_64_bit_run():
    """Ten steps with FP32 moments stay within ten times a step's error; with 8-bit moments a quadratic still descends."""
    g = torch.Generator().manual_seed(2)
    p64 = torch.randn(3000, generator=g).double()
    p = p64.float().cuda()
    m64 = v64 = torch.zeros(3000, dtype=torch.float64)
    p64 = p.double().cpu()
    m, v = torch.zeros(3000, device="cuda"), torch.zeros(3000, device="cuda")
    for step in range(1, 11):
        grad = p.clone()
        g64 = grad.double().cpu()
        dpg.dpg_adamw([p], [grad], [m], [v], step=step, **HYPER)
        m64, v64 = 0.9 * m64 + 0.1 * g64, 0.95 * v64 + 0.05 * g64 ** 2
        p64 = p64 * (1 - 3e-4) - 3e-3 * m64 / (1 - 0.9 ** step) / ((v64 / (1 - 0.95 ** step)).sqrt() + 1e-8)
        assert float((p.double().cpu() - p64).abs().max()) <= step * 8 * EPS32 * 4
    q = torch.randn(3000, generator=g).cuda()
    start = float(q.square().mean())
    m, v = (torch.zeros(3000, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    sc = [torch.ones(12, device="cuda") for _ in range(2)]
    for step in range(1, 201):
        dpg.dpg_adamw([q], [q.clone()], [m], [v], lr=1e-2, beta1=0.9, beta2=0.95, weight_decay=0.0, step=step,
                      avg_scales=[sc[0]], sq_scales=[sc[1]], seed=step)
    assert float(q.square().mean()) < 0.15 * start


def test_on_a_side_stream_and_in_a_graph():
    a, b = _lists(SIZES, torch.float32, True), _lists(SIZES, torch.float32, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dpg.dpg_adamw(**a, step=2, seed=1, stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    dpg.dpg_adamw(**b, step=2, seed=1, **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dpg.dpg_adamw(**a, step=3, seed=2, **HYPER)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        dpg.dpg_adamw(**b, step=3, seed=2, **HYPER)
        for k in a:
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k


def test_refusals():
    s = _lists([100, 200], torch.float32, False)

    def bad(error, **change):
        with pytest.raises(error):
            dpg.dpg_adamw(**{**s, **HYPER, "step": 1, **change})
    bad(dpg.DpgError, step=0)
    bad(dpg.DpgError, beta1=1.0)
    bad(dpg.DpgError, beta2=-0.1)
    bad(dpg.DpgError, lr=float("nan"))
    bad(dpg.DpgError, eps=-1.0)
    bad(ValueError, grads=s["grads"][:1])
    bad(ValueError, grads=s["grads"][::-1])
    bad(TypeError, grads=[s["grads"][0], s["grads"][1].to(torch.bfloat16)])
    bad(TypeError, params=[t.to(torch.bfloat16) for t in s["params"]])
    bad(TypeError, exp_avgs=[t.half() for t in s["exp_avgs"]])
    bad(ValueError, copies=[t.cpu() for t in s["copies"]])
    bad(ValueError, grads=[torch.zeros(200, device="cuda")[::2], s["grads"][1]])
    bad(ValueError, exp_avgs=[t.to(torch.float8_e4m3fn) for t in s["exp_avgs"]],
        exp_avg_sqs=[t.to(torch.float8_e4m3fn) for t in s["exp_avg_sqs"]])
    assert dpg.dpg_adamw([], [], [], [], lr=1.0) is None
