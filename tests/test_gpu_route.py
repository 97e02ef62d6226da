"""Routing on the GPU against a 64-bit statement of the definitions: the choice
and the order are whole numbers and equal, the weights and gradients within
bounds counted from their roundings."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

INF, NAN = float("inf"), float("nan")
# weights: exp (within 2 units in the last place of FP32, and its argument off by
# half a step of a difference of at most 20: 20 * 2^-24), up to 512 added terms
# and a quotient: 2 * (2 + 20 + 2 + 10) * 2^-24 covers both sides of the quotient
W_TOL = 80 * 2.0 ** -24


def _choice(lg, k, renorm):
    """experts, weights, offsets, rows, positions in numpy, one token at a time."""
    lg = np.asarray(lg, dtype=np.float64)
    T, E = lg.shape
    experts, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if lg[t, e] > -INF), key=lambda e: (-lg[t, e], e))[:k]
        if not order:
            continue
        experts[t, :len(order)] = order
        pool = order if renorm else [e for e in range(E) if lg[t, e] > -INF]
        top = lg[t, order[0]]
        total = sum(math.exp(lg[t, e] - top) for e in pool)
        weights[t, :len(order)] = [math.exp(lg[t, e] - top) / total for e in order]
        if np.isnan(lg[t]).any():
            weights[t, :len(order)] = NAN
    key = np.where(experts < 0, E, experts).reshape(-1)
    rows = np.argsort(key, kind="stable")
    positions = np.argsort(rows, kind="stable").reshape(T, k)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return experts, weights, offsets, rows, positions


def _check_route(lg, k, renorm):
    r = dpg.dpg_route(lg, k, renormalize=renorm)
    torch.cuda.synchronize()
    ref = _choice(lg.double().cpu().numpy(), k, renorm)
    for name, want in zip(("experts", "offsets", "rows", "positions"), (ref[0], ref[2], ref[3], ref[4])):
        got = getattr(r, name).cpu().numpy()
        assert got.shape == want.shape and np.array_equal(got, want), name
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref[1]))
    assert np.nanmax(np.abs(got - ref[1]) - W_TOL * ref[1], initial=0.0) <= 2.0 ** -140
    return r


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 256, 8), (5, 3, 3), (64, 64, 6), (65, 64, 6), (200, 65, 1),
                                   (129, 512, 32), (1000, 256, 8), (777, 130, 5), (3000, 2, 2), (70, 128, 4)])
def test_choice_and_order(T, E, k, renorm):
    g = torch.Generator().manual_seed(T + E)
    _check_route(torch.randn(T, E, generator=g).cuda() * 2, k, renorm)


def test_many_tokens_per_block():
    """More than 64 * 512 tokens: blocks of more than 64 tokens."""
    g = torch.Generator().manual_seed(1)
    lg = torch.randn(40001, 16, generator=g).cuda()
    r = dpg.dpg_route(lg, 2)
    key = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(r.experts, key.int())
    rows = torch.sort(key.reshape(-1), stable=True).indices
    assert torch.equal(r.rows, rows.int())
    assert torch.equal(r.positions.reshape(-1)[rows], torch.arange(80002, device="cuda", dtype=torch.int32))
    assert torch.equal(r.offsets[1:], torch.cumsum(torch.bincount(key.reshape(-1), minlength=16), 0).int())


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [3, 300])
def test_ties_masks_and_strange_values(T, renorm):
    E, k = 70, 6
    g = torch.Generator().manual_seed(2)
    lg = torch.randint(-2, 3, (T, E), generator=g).float()       # many ties
    lg[0] = -INF                                                  # nothing left
    lg[1, 3:] = -INF                                              # three left
    lg[2] = torch.finfo(torch.float32).min                        # the lowest value masks nothing
    if T > 3:
        lg[3, 5] = NAN
        lg[4] = NAN
        lg[5, :] = -INF
        lg[5, 69] = -3.0
        lg[6, 10] = 0.0
        lg[6, 4] = -0.0
        lg[7] = -INF
        lg[7, 2] = NAN
        lg[8] *= 1e30
    r = _check_route(lg.cuda(), k, renorm)
    assert r.experts[0].tolist() == [-1] * k and r.weights[0].tolist() == [0.0] * k
    assert r.experts[2].tolist() == list(range(k))


def test_an_infinite_logit_is_chosen():
    lg = torch.zeros(1, 8, device="cuda")
    lg[0, 5] = INF
    r = dpg.dpg_route(lg, 2)
    assert r.experts.tolist() == [[5, 0]] and bool(torch.isnan(r.weights).all())


def test_strided_logits_and_streams():
    g = torch.Generator().manual_seed(3)
    wide = torch.full((90, 77), NAN, device="cuda")
    wide[:, :61] = torch.randn(90, 61, generator=g).cuda()
    a = _check_route(wide[:, :61], 4, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = dpg.dpg_route(wide[:, :61], 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,masked", [(1, 4, 2, 0.0), (33, 64, 6, 0.3), (50, 200, 8, 0.0), (20, 512, 32, 0.97)])
def test_route_gradient(T, E, k, masked, renorm):
    """Against the formula in 64 bits and against differences of the 64-bit weights."""
    g = torch.Generator().manual_seed(E)
    lg = torch.randn(T, E, generator=g)
    lg[torch.rand(T, E, generator=g) < masked] = -INF
    if masked:
        lg[T // 2] = -INF
    dw = torch.randn(T, k, generator=g)
    r = dpg.dpg_route(lg.cuda(), k, renormalize=renorm)
    got = dpg.dpg_route_dgrad(lg.cuda(), r.experts, r.weights, dw.cuda(), renormalize=renorm).double().cpu().numpy()
    experts, weights = _choice(lg.double().numpy(), k, renorm)[:2]
    d = dw.double().numpy()

    def value(l64, t):  # the scalar whose gradient is asked for, with the choice held
        e = experts[t][experts[t] >= 0]
        z = np.exp(l64 - l64.max())
        q = z / (z[e].sum() if renorm else z.sum())
        return float((q[e] * d[t, :len(e)]).sum())

    ref = np.zeros((T, E))
    for t in range(T):
        e = experts[t][experts[t] >= 0]
        if not len(e):
            continue
        row = lg[t].double().numpy()
        z = np.exp(row - row.max())
        q = np.zeros(E)
        if renorm:
            q[e] = z[e] / z[e].sum()
        else:
            q = z / z.sum()
        gf = np.zeros(E)
        gf[e] = d[t, :len(e)]
        ref[t] = q * (gf - (q * gf).sum())
        for i in (e[0], e[-1], int(np.argmax(np.where(np.isin(np.arange(E), e), -INF, row)))):
            if row[i] == -INF:
                continue
            up, dn = row.copy(), row.copy()
            up[i] += 1e-5
            dn[i] -= 1e-5
            assert abs((value(up, t) - value(dn, t)) / 2e-5 - ref[t, i]) < 1e-8
    # each factor is off by W_TOL, the inner sum by that of its terms' magnitudes
    mag = np.abs(d).max(1, keepdims=True) * 2
    assert (np.abs(got - ref) <= 2 * W_TOL * mag).all()
    assert (got[experts.max(1) < 0] == 0).all()


def _case(T, k, H, E, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(T, E, generator=g)
    lg[torch.rand(T, E, generator=g) < 0.4] = -INF
    r = dpg.dpg_route(lg.cuda(), k)

    def rows(n, fill=None):
        t = torch.randn(n, H + pad, generator=g).to(dtype).cuda()
        return t[:, :H]
    return r, rows


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H,E,pad", [(1, 1, 8, 1, 0), (3, 2, 24, 4, 8), (50, 6, 264, 9, 0), (130, 8, 4096, 64, 0),
                                         (7, 4, 10240, 8, 16), (40, 32, 128, 40, 0), (530, 8, 4104, 64, 0)])
def test_rows_there_and_back(T, k, H, E, pad, dtype):
    r, rows = _case(T, k, H, E, dtype, pad=pad)
    used, pos = int(r.offsets[-1]), r.positions.long()
    live = (pos < used)[..., None]
    x, ys, dy = rows(T), rows(T * k), rows(T)
    ys[used:] = NAN  # never read
    xs = dpg.dpg_dispatch(x, r.positions, r.offsets)
    want = x[(r.rows // k).long()].clone()
    want[used:] = 0
    assert torch.equal(xs, want)
    eps = 2.0 ** -24
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    picked = torch.where(live, ys[pos].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    w = r.weights.double()[..., None]
    # k products and additions in FP32, then the output's rounding
    ref, mag = (picked * w).sum(1), (picked.abs() * w).sum(1)
    limit = (k + 1) * eps * mag
    for out in (torch.bfloat16, torch.float32):
        got = dpg.dpg_combine(ys, r.positions, r.offsets, r.weights, out_dtype=out).double()
        h = 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24
        assert bool(((got - ref).abs() <= limit + h * (ref.abs() + limit)).all())
    # without weights: dispatch's gradient, and its transpose <dispatch(x), ys> = <x, combine(ys)>
    ref1, mag1 = picked.sum(1), picked.abs().sum(1)
    got = dpg.dpg_combine(ys, r.positions, r.offsets).double()
    assert bool(((got - ref1).abs() <= k * eps * mag1 + half * (ref1.abs() + mag1 * k * eps)).all())
    dys, dw = dpg.dpg_combine_dgrad(dy, ys, r.positions, r.offsets, r.weights)
    want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    want[pos.reshape(-1)] = torch.where(live, dy.double()[:, None] * w, torch.zeros_like(w)).reshape(T * k, H)
    assert bool(((dys.double() - want).abs() <= (half + eps) * want.abs()).all())
    ref2, mag2 = (picked * dy.double()[:, None]).sum(2), (picked * dy.double()[:, None]).abs().sum(2)
    assert bool(((dw.double() - ref2).abs() <= H * eps * mag2).all())


def test_combine_gradient_against_differences():
    r, rows = _case(9, 3, 16, 5, torch.float32, seed=4)
    ys, dy = rows(27), rows(9)
    dys, dw = dpg.dpg_combine_dgrad(dy, ys, r.positions, r.offsets, r.weights)
    used = int(r.offsets[-1])

    def f(y, w):
        got = dpg.dpg_combine(y.float(), r.positions, r.offsets, w.float()).double()
        return float((got * dy.double()).sum())
    for i, j in ((0, 0), (used - 1, 15), (used // 2, 7)):
        up, dn = ys.clone(), ys.clone()
        up[i, j] += 0.5
        dn[i, j] -= 0.5
        # the function is linear: the difference is the gradient, up to FP32 sums of about 10 in size
        assert abs(f(up, r.weights) - f(dn, r.weights) - float(dys[i, j])) < 1e-4
    t, s = [int(v) for v in (r.positions < used).nonzero()[0]]
    up, dn = r.weights.clone(), r.weights.clone()
    up[t, s] += 0.5
    dn[t, s] -= 0.5
    assert abs(f(ys, up) - f(ys, dn) - float(dw[t, s])) < 1e-4


def test_positions_outside_the_matrix_are_left_out():
    r, rows = _case(6, 2, 32, 4, torch.bfloat16)
    bad = r.positions.clone()
    bad[0] = torch.tensor([-1, 2 ** 31 - 1], dtype=torch.int32)
    bad[1] = torch.tensor([12, -2 ** 31], dtype=torch.int32)
    off = r.offsets.clone()
    off[-1] = 2 ** 31 - 1
    x, ys = rows(6), rows(12)
    wide = torch.full((14, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    dpg.dpg_dispatch(x, bad, off, out=wide[1:13])
    y = dpg.dpg_combine(ys, bad, off, r.weights)
    dpg.dpg_combine_dgrad(x, ys, bad, off, r.weights)
    torch.cuda.synchronize()
    assert bool((wide[[0, 13]] == 7.0).all()) and bool((y[:2] == 0).all())


def test_graph_replays():
    """A captured route, dispatch and combine, replayed on changed inputs with eager work between."""
    g = torch.Generator().manual_seed(6)
    lg, x = torch.randn(300, 64, generator=g).cuda(), torch.randn(300, 256, generator=g).cuda().to(torch.bfloat16)

    def step():
        r = dpg.dpg_route(lg, 6)
        xs = dpg.dpg_dispatch(x, r.positions, r.offsets)
        return [*r, xs, dpg.dpg_combine(xs, r.positions, r.offsets, r.weights)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        lg.copy_(torch.randn(300, 64, generator=g).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_refusals():
    lg = torch.zeros(4, 16, device="cuda")
    for k in (0, 17, -1):
        with pytest.raises(dpg.DpgError):
            dpg.dpg_route(lg, k)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_route(torch.zeros(4, 513, device="cuda"), 2)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_route(torch.zeros(4, 64, device="cuda"), 33)
    with pytest.raises(TypeError):
        dpg.dpg_route(lg.to(torch.bfloat16), 2)
    r = dpg.dpg_route(lg, 2)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        dpg.dpg_dispatch(x[:3], r.positions, r.offsets)
    with pytest.raises(TypeError):
        dpg.dpg_dispatch(x.half(), r.positions, r.offsets)
    with pytest.raises(ValueError):
        dpg.dpg_combine(x, r.positions, r.offsets)
    with pytest.raises(ValueError):
        dpg.dpg_combine(x.repeat(2, 1), r.positions, r.offsets, r.weights[:3])
    with pytest.raises(TypeError):
        dpg.dpg_combine_dgrad(x, x.repeat(2, 1).float(), r.positions, r.offsets, r.weights)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_dispatch(x[:, :60].contiguous(), r.positions, r.offsets)  # 60 columns: no 16-byte rows
