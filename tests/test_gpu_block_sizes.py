"""Layer norm and dropout at the sizes of large calls (block_cases.py): several
rounds of rows, the rows at each round's ends against 64-bit references, and
dropout past the caches.

Tolerances: the bounds of block_reference plus the rounding to the output's type."""
import functools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_cases as cases  # noqa: E402
import block_reference as ref  # noqa: E402
from test_gpu_layer_norm import BF16, EPS, F32, TYPES, _check  # noqa: E402

KINDS = [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")]


@pytest.fixture(autouse=True)
def _additions_of_these_cuts(monkeypatch):
    """With eight groups of eight columns to a lane a value goes through up to 64
    additions in a lane, 6 over the lanes, 16 over the waves, and a few for the
    composition."""
    monkeypatch.setattr(ref, "ROW_SUM", 64 + 6 + 16 + 10)


def _rand(seed, *shape, dtype=F32, scale=1.0, mean=0.0):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.normal_(mean, scale, generator=torch.Generator(device="cuda").manual_seed(seed))


def _affine(H):
    return _rand(H + 1, H, scale=0.3, mean=1.0).abs().clamp(min=0.25), _rand(H + 2, H, scale=0.2)


def _rows(T, step):
    """Around the border of each round."""
    at = {0, 1, T - 2, T - 1}
    for border in range(step, T, step):
        at |= {border - 2, border - 1, border, border + 1}
    return sorted(t for t in at if 0 <= t < T)


def _kept(rows, H, p, seed, step):
    return np.concatenate([_row_kept(t, H, p, seed, step) for t in rows])


def _row_kept(t, H, p, seed, step):
    w = ref.philox(np.arange(t * (H // 8), (t + 1) * (H // 8)), seed, step)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 1).reshape(8, -1).T.reshape(1, H)
    return bits >= np.uint64(int(np.floor(p * 65536 + 0.5)))


@pytest.mark.parametrize("x, y", KINDS)
@pytest.mark.parametrize("case", cases.NORM, ids=str)
def test_norm_rounds(case, x, y):
    T, H = case
    v = _rand(H, T, H, dtype=TYPES[x], scale=2.0, mean=0.7)
    w, b = _affine(H)
    n = dpg.dpg_layer_norm(v, w, b, eps=EPS, out_dtype=TYPES[y])
    at = _rows(T, cases.norm_round(H, True, False))
    wy, wm, wr, ey, em, er = ref.layer_norm(ref.host(v[at]), ref.host(w), ref.host(b), EPS)
    _check("y", n.y[at], wy, ey, TYPES[y])
    _check("mean", n.mean[at], wm, em)
    _check("rstd", n.rstd[at], wr, er)
    # all the others: rows of mean 0 and unit spread, but for the weights.  z is off by 4 u (|z| + |b| / 0.25), which moves
    # the means by less than 1e-5; eps over a variance of 1 or more takes 1e-5 of it
    if y == "f32":
        z = (n.y - b) / w
        assert float((z.square().mean(1) - 1).abs().max()) < 1e-4 and float(z.mean(1).abs().max()) < 1e-4


@pytest.mark.parametrize("x, branch", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("case", cases.ADD_NORM, ids=str)
def test_sum_rounds(case, x, branch):
    T, H = case
    p, seed = 0.3, 0x123456789ABCDEF0 + H
    r, v = _rand(H, T, H, dtype=TYPES[x], scale=2.0), _rand(H + 3, T, H, dtype=TYPES[branch])
    w, b = _affine(H)
    step = torch.tensor([5], device="cuda")
    n = dpg.dpg_add_layer_norm(v, r, w, b, eps=EPS, p=p, seed=seed, step=step, out_dtype=BF16)
    at = _rows(T, cases.norm_round(H, True, True))
    part = np.where(_kept(at, H, p, seed, 5), ref.host(v[at]) * ref.keep_scale(p), 0.0)
    hr = ref.host(r[at])
    total = hr + part
    _check("sum", n.sum[at], total, ref.U * (2 * np.abs(part) + np.abs(total)), TYPES[x])
    wy, wm, wr, ey, em, _ = ref.layer_norm(total, ref.host(w), ref.host(b), EPS)
    # the sum's own error, at most 3 u of |r| + |part|, moves mean, differences and rstd as a change of the input
    big = 3 * ref.U * (np.abs(hr) + np.abs(part))
    move = big + big.mean(1, keepdims=True)
    unit = np.abs(total - wm[:, None]) * wr[:, None]
    shift = wr[:, None] * (move + unit * (move * unit).mean(1, keepdims=True))
    _check("y", n.y[at], wy, ey + 1.01 * np.abs(ref.host(w)) * shift, BF16)
    _check("mean", n.mean[at], wm, em + big.mean(1))
    # every row's sum is that of dpg_dropout, each with its own product, sum and rounding to the type
    other = dpg.dpg_dropout(v, p, seed, step=step, residual=r)
    limit = 2 * (ref.half_step(TYPES[x]) + 3 * ref.U) * (r.float().abs() + 1.5 * v.float().abs())
    assert bool(((n.sum.float() - other.float()).abs() <= limit).all())
    # and with the sum over the residual the same bits
    own = r.clone()
    m = dpg.dpg_add_layer_norm(v, own, w, b, eps=EPS, p=p, seed=seed, step=step, sum=own, out_dtype=BF16)
    assert torch.equal(own, n.sum) and torch.equal(m.y, n.y) and torch.equal(m.mean, n.mean) and torch.equal(m.rstd, n.rstd)


@pytest.mark.parametrize("x, dy", KINDS)
@pytest.mark.parametrize("add", [False, True], ids=["alone", "sum"])
@pytest.mark.parametrize("case", cases.NORM_GRADIENT, ids=str)
def test_gradient_rounds(case, add, x, dy):
    T, H = case
    v = _rand(H, T, H, dtype=TYPES[x], scale=2.0, mean=0.3)
    g = _rand(H + 5, T, H, dtype=TYPES[dy])
    w, _ = _affine(H)
    n = dpg.dpg_layer_norm(v, w, eps=EPS)
    at = _rows(T, cases.norm_gradient_round(H))
    p, seed = 0.3, 77 + H
    if add:
        more = _rand(H + 6, T, H, dtype=TYPES[x])
        d = dpg.dpg_add_layer_norm_dgrad(g, v, n.mean, n.rstd, w, dsum=more, p=p, seed=seed, x_dtype=BF16)
    else:
        d = dpg.dpg_layer_norm_dgrad(g, v, n.mean, n.rstd, w)
    dv, _, _, ev, _, _ = ref.layer_norm_dgrad(ref.host(g[at]), ref.host(v[at]), ref.host(n.mean[at]),
                                              ref.host(n.rstd[at]), ref.host(w))
    if add:
        dv = dv + ref.host(more[at])
        ev = ev + ref.U * np.abs(dv)
        _check("dresidual", d.dresidual[at], dv, ev, TYPES[x])
        keep = np.where(_kept(at, H, p, seed, 0), ref.keep_scale(p), 0.0)
        _check("dx", d.dx[at], keep * dv, keep * (ev + 2 * ref.U * np.abs(dv)), BF16)
    else:
        _check("dx", d.dx[at], dv, ev, TYPES[x])
    # over all rows, at some columns: each sum goes through no more additions than there are rows, and a few
    col = sorted({0, 1, 7, 8, 63, H // 2, H - 9, H - 2, H - 1})
    unit = (ref.host(v[:, col]) - ref.host(n.mean)[:, None]) * ref.host(n.rstd)[:, None]
    hg = ref.host(g[:, col])
    depth = (T + 8) * ref.U
    _check("dweight", d.dweight[col], (hg * unit).sum(0), depth * np.abs(hg * unit).sum(0))
    _check("dbias", d.dbias[col], hg.sum(0), depth * np.abs(hg).sum(0))


@pytest.mark.parametrize("T, H", [(1027, 1544), (4103, 2056), (4103, 4096), (1030, 8200)])
@pytest.mark.parametrize("x", list(TYPES))
def test_many_rows_of_a_wider_matrix(T, H, x):
    wide = {k: torch.full((T, H + 32), 7.0, dtype=TYPES[x], device="cuda") for k in "xyd"}
    cut = {k: t[:, 16:16 + H] for k, t in wide.items()}
    cut["x"].copy_(_rand(H, T, H, scale=2.0))
    cut["d"].copy_(_rand(H + 1, T, H))
    w, b = _affine(H)
    n = dpg.dpg_layer_norm(cut["x"], w, b, out=cut["y"])
    m = dpg.dpg_layer_norm(cut["x"].contiguous(), w, b)
    assert torch.equal(cut["y"], m.y) and torch.equal(n.mean, m.mean) and torch.equal(n.rstd, m.rstd)
    assert bool((wide["y"][:, :16] == 7).all()) and bool((wide["y"][:, 16 + H:] == 7).all())
    d = dpg.dpg_layer_norm_dgrad(cut["d"], cut["x"], n.mean, n.rstd, w)
    e = dpg.dpg_layer_norm_dgrad(cut["d"].contiguous(), cut["x"].contiguous(), n.mean, n.rstd, w)
    assert torch.equal(d.dx, e.dx) and torch.equal(d.dweight, e.dweight) and torch.equal(d.dbias, e.dbias)


@pytest.mark.parametrize("T, H", [(4103, 2048), (4103, 4096), (4103, 8192), (2051, 16384)])
def test_strange_rows_among_many(T, H):
    """Infinities and NaN stay in their rows, whatever rows share their workgroup."""
    x = _rand(H, T, H)
    want = dpg.dpg_layer_norm(x)
    step = cases.norm_round(H, True, False)
    strange = [0, 3, step - 1, step, step + 2, 2 * step + 1, T - 1]
    for i, t in enumerate(strange):
        x[t, (i * 977) % H] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    n = dpg.dpg_layer_norm(x)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[strange] = True
    assert bool(n.y[bad].isnan().all()) and torch.equal(n.y[~bad], want.y[~bad])
    assert torch.equal(n.mean[~bad], want.mean[~bad]) and torch.equal(n.rstd[~bad], want.rstd[~bad])
    dy = torch.ones_like(x)
    d = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd)
    e = dpg.dpg_layer_norm_dgrad(dy, x, want.mean, want.rstd)
    assert bool(d.dx[bad].isnan().all()) and torch.equal(d.dx[~bad], e.dx[~bad])


@functools.lru_cache(maxsize=1)
def _mask(T, H, p, seed, step):
    return ref.kept(T, H, p, seed, step)


@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
@pytest.mark.parametrize("case", cases.DROPOUT, ids=str)
def test_dropout_past_the_caches(case, residual, x):
    """The mask of every element, and its value."""
    kind, T, H, pad = case
    p, seed, at = 0.37, (1 << 63) + 12345, (7 << 32) + 3
    wide = lambda s, t: _rand(s, T, H + pad, dtype=t)[:, :H]  # noqa: E731
    v = wide(1, TYPES[x])
    r = wide(2, TYPES[kind]) if residual else None
    step = torch.tensor([at], device="cuda")
    out = torch.full((T, H + pad), 7.0, dtype=TYPES[kind], device="cuda")
    y = dpg.dpg_dropout(v, p, seed, step=step, residual=r, out=out[:, :H])
    assert y.data_ptr() == out.data_ptr() and bool((out[:, H:] == 7).all())
    kept = torch.from_numpy(_mask(T, H, p, seed, at)).cuda()
    part = torch.where(kept, v.double() * ref.keep_scale(p), torch.zeros((), dtype=torch.float64, device="cuda"))
    want = part + r.double() if residual else part
    bound = ref.U * (2 * part.abs() + want.abs())  # the scale, the product, the sum
    limit = bound * 1.01 + ref.half_step(TYPES[kind]) * (want.abs() + bound) + 1e-37
    assert bool(((y.double() - want).abs() <= limit).all())
    if not residual:
        assert torch.equal(y == 0, ~kept | (v == 0))
    # over the input, or over the residual
    own = r if residual else v if x == kind else None
    if own is not None:
        assert torch.equal(dpg.dpg_dropout(v, p, seed, step=step, residual=r, out=own), y)
