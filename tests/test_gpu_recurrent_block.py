"""Layer norm, dropout, recurrence and projections together: the autograd
wrappers, a block captured in a graph, and the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_reference as ref  # noqa: E402
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32


def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _block(B, T, H, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = {"y": _randn(g, B, T, H, dtype=BF16), "stream": _randn(g, B, T, H), "w": 1 + _randn(g, H, scale=0.2),
         "b": _randn(g, H, scale=0.2), "w_gate": _randn(g, N, H, dtype=BF16, scale=H ** -0.5),
         "w_in": _randn(g, N, H, dtype=BF16, scale=H ** -0.5), "w_out": _randn(g, H, N, dtype=BF16, scale=N ** -0.5),
         "state": _randn(g, B, N)}
    grads = {"out": _randn(g, B, T, H, dtype=BF16), "stream": _randn(g, B, T, H), "state": _randn(g, B, N)}
    return t, grads


P, SEED = 0.25, 99


def _by_hand(t, grads, step):
    """The block and its gradients through the entry points alone."""
    B, T, H = t["y"].shape
    N = t["w_gate"].shape[0]
    rows = lambda v: v.reshape(B * T, -1)  # noqa: E731
    seqs = lambda v: v.view(B, T, -1)  # noqa: E731
    n = dpg.dpg_add_layer_norm(rows(t["y"]), rows(t["stream"]), t["w"], t["b"], p=P, seed=SEED, step=step)
    gate, v = dpg.dpg_forward(n.y, t["w_gate"]), dpg.dpg_forward(n.y, t["w_in"])
    r = dpg.dpg_recurrence(seqs(gate), seqs(v), state=t["state"], carries=True)
    out = dpg.dpg_forward(rows(r.h), t["w_out"])
    dout = rows(grads["out"])
    d = {"w_out": dpg.dpg_wgrad(dout, rows(r.h))}
    dh = dpg.dpg_dgrad(dout, t["w_out"])
    b = dpg.dpg_recurrence_dgrad(seqs(dh), seqs(gate), seqs(v), r.carries, state=t["state"], dstate=grads["state"])
    d["w_gate"], d["w_in"] = dpg.dpg_wgrad(rows(b.dgate), n.y), dpg.dpg_wgrad(rows(b.dx), n.y)
    dn = dpg.dpg_dgrad(rows(b.dgate), t["w_gate"]) + dpg.dpg_dgrad(rows(b.dx), t["w_in"])
    e = dpg.dpg_add_layer_norm_dgrad(dn, n.sum, n.mean, n.rstd, t["w"], dsum=rows(grads["stream"]), p=P, seed=SEED,
                                     step=step, x_dtype=BF16)
    d.update(y=seqs(e.dx), stream=seqs(e.dresidual), w=e.dweight, b=e.dbias, state=b.dstate)
    assert gate.shape[1] == N
    return seqs(out), seqs(n.sum), r.state, d


def _by_autograd(t, step):
    n, stream = dag.add_layer_norm(t["y"], t["stream"], t["w"], t["b"], p=P, seed=SEED, step=step)
    h, state = dag.recurrence(dag.projection(n, t["w_gate"]), dag.projection(n, t["w_in"]), state=t["state"])
    return dag.projection(h, t["w_out"]), stream, state


def test_autograd_equals_the_entry_points():
    t, grads = _block(3, 70, 72, 136)
    step = torch.tensor([3], device="cuda")
    out, stream, state, d = _by_hand(t, grads, step)
    leaves = {k: v.clone().requires_grad_(True) for k, v in t.items()}
    got = _by_autograd(leaves, step)
    for a, b in zip(got, (out, stream, state)):
        assert torch.equal(a, b)
    torch.autograd.backward(got, (grads["out"], grads["stream"], grads["state"]))
    for k, v in leaves.items():
        assert torch.equal(v.grad, d[k]), k


def test_each_wrapper_alone():
    g = torch.Generator().manual_seed(4)
    x, dy = _randn(g, 2, 9, 40, dtype=BF16), _randn(g, 2, 9, 40, dtype=BF16)
    w, b = 1 + _randn(g, 40, scale=0.1), _randn(g, 40)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, b)]
    y = dag.layer_norm(*leaves)
    y.backward(dy)
    n = dpg.dpg_layer_norm(x.view(18, 40), w, b)
    d = dpg.dpg_layer_norm_dgrad(dy.view(18, 40), x.view(18, 40), n.mean, n.rstd, w)
    assert torch.equal(y.view(18, 40), n.y) and torch.equal(leaves[0].grad.view(18, 40), d.dx)
    assert torch.equal(leaves[1].grad, d.dweight) and torch.equal(leaves[2].grad, d.dbias)
    r = _randn(g, 2, 9, 40).requires_grad_(True)
    v = x.clone().requires_grad_(True)
    dag.dropout(v, 0.5, 7, residual=r).backward(dy.float())
    assert torch.equal(r.grad, dy.float())
    assert torch.equal(v.grad.view(18, 40), dpg.dpg_dropout(dy.float().view(18, 40), 0.5, 7, out_dtype=BF16))
    # only the sum is used: its gradient goes past the norm
    v, r = x.clone().requires_grad_(True), _randn(g, 2, 9, 40).requires_grad_(True)
    _, total = dag.add_layer_norm(v, r, p=0.5, seed=8)
    total.sum().backward()
    assert bool((r.grad == 1).all())
    assert np.array_equal(ref.host(v.grad).reshape(18, 40), ref.dropped(np.ones((18, 40)), 0.5, 8))


def test_packed_sequences_and_views_through_autograd():
    g = torch.Generator().manual_seed(5)
    both = _randn(g, 50, 2 * 40, dtype=BF16)
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda")
    leaf = both.clone().requires_grad_(True)
    h, state = dag.recurrence(leaf[:, :40], leaf[:, 40:], offsets=off)
    dh = _randn(g, 50, 40, dtype=BF16)
    h.backward(dh)
    r = dpg.dpg_recurrence(both[:, :40], both[:, 40:], offsets=off, carries=True)
    d = dpg.dpg_recurrence_dgrad(dh, both[:, :40], both[:, 40:], r.carries, offsets=off)
    assert torch.equal(h, r.h) and torch.equal(state, r.state)
    assert torch.equal(leaf.grad, torch.cat([d.dgate, d.dx], 1))
    # steps of longer sequences: not one stride apart, copied
    t = _randn(g, 4, 30, 40, dtype=BF16)
    h2, _ = dag.recurrence(t[:, 5:20], t[:, 5:20])
    assert torch.equal(h2, dpg.dpg_recurrence(t[:, 5:20].contiguous(), t[:, 5:20].contiguous()).h)


def test_a_step_counted_up_before_the_backward_pass_is_an_error():
    x = torch.ones(4, 16, device="cuda", requires_grad=True)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    y = dag.dropout(x, 0.5, 1, step=step)
    step += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


def test_differentiating_twice_raises():
    x = torch.randn(2, 9, 16, device="cuda", requires_grad=True)
    for f in (lambda: dag.layer_norm(x), lambda: dag.add_layer_norm(x, x)[0], lambda: dag.dropout(x, 0.5, 1),
              lambda: dag.recurrence(x, x)[0]):
        (dx,) = torch.autograd.grad(f().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            dx.sum().backward()


def test_gradients_against_64_bits():
    """FP32 norm and recurrence of one leaf each, against 64-bit autograd: the
    reference formulas are torch's, not this library's.  The bound is that of
    block_reference on the same inputs, which the other tests derive."""
    g = torch.Generator().manual_seed(6)
    B, T, D = 2, 90, 16
    gate, x, dh, h0 = _randn(g, B, T, D), _randn(g, B, T, D), _randn(g, B, T, D), _randn(g, B, D)
    lg, lx, l0 = (v.double().cpu().requires_grad_(True) for v in (gate, x, h0))
    h, rows = l0, []
    f = torch.sigmoid(lg)
    for i in range(T):
        h = f[:, i] * h + (1 - f[:, i]) * lx[:, i]
        rows.append(h)
    torch.stack(rows, 1).backward(dh.double().cpu())
    want = ref.recurrence(ref.host(gate).reshape(-1, D), ref.host(x).reshape(-1, D), [0, T, 2 * T], ref.host(h0), True,
                          ref.host(dh).reshape(-1, D))
    for name, leaf in (("dgate", lg), ("dx", lx), ("dstate", l0)):
        assert np.abs(want[name] - leaf.grad.numpy().reshape(want[name].shape)).max() < 1e-12
    leaves = [v.clone().requires_grad_(True) for v in (gate, x, h0)]
    dag.recurrence(leaves[0], leaves[1], state=leaves[2])[0].backward(dh)
    for name, leaf in zip(("dgate", "dx", "dstate"), leaves):
        got, w = ref.host(leaf.grad).reshape(want[name].shape), want[name]
        assert bool((np.abs(got - w) <= want["e_" + name] * 1.01 + ref.U * np.abs(w)).all()), name


def test_block_in_a_graph():
    """Forward and gradients captured once, replayed with new inputs and steps, the
    eager block between the replays."""
    t, grads = _block(2, 300, 64, 128, seed=7)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _by_hand(t, grads, step)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, stream, state, d = _by_hand(t, grads, step)
    for i in range(4):
        fresh, _ = _block(2, 300, 64, 128, seed=20 + i)
        for k, v in t.items():
            v.copy_(fresh[k])
        step.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        a, b, c, e = _by_hand(t, grads, step)
        assert torch.equal(out, a) and torch.equal(stream, b) and torch.equal(state, c)
        assert all(torch.equal(d[k], e[k]) for k in e)


def test_example_runs_and_its_gradients():
    spec = importlib.util.spec_from_file_location("recurrent_block_example",
                                                  os.path.join(ROOT, "examples", "recurrent_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    small = dict(batch=2, length=64, layers=2, hidden=64, inner=64)
    losses = example.main(steps=6, **small)
    assert np.isfinite(losses).all()
    assert example.main(steps=3, **small) == losses[:3]  # the same run gives the same bits
    # without dropout the last norm's bias enters the output linearly
    model = example.RecurrentBlocks(2, 64, 64, p=0.0)
    g = torch.Generator().manual_seed(2)
    x = _randn(g, 2, 64, 64, dtype=BF16)
    weight = torch.randint(-3, 4, (2, 64, 64), generator=g).float().cuda()
    leaves = model.leaves()
    grads = torch.autograd.grad((model.forward(x, leaves) * weight).sum(), leaves)
    assert all(bool(torch.isfinite(v).all()) for v in grads)
    assert torch.equal(grads[-1].double(), weight.double().sum((0, 1)))
