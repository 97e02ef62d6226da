"""Layer norm and dropout against 64-bit references: every cut of the row, types,
odd rows, strides, means far from zero, infinities and NaN, masks bit for bit.

Tolerances: the bounds of block_reference plus the rounding to the output's type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_reference as ref  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
TYPES = {"bf16": BF16, "f32": F32}


def _randn(g, *shape, dtype=F32, scale=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g) * scale + mean).to(dtype).cuda()


def _check(name, got, want, bound, dtype=F32):
    limit = bound * 1.01 + ref.half_step(dtype) * (np.abs(want) + bound) + 1e-37
    off = np.abs(ref.host(got) - want)
    assert got.dtype == dtype and bool((off <= limit).all()), (name, float((off / limit).max()))


def _affine(g, H):
    return _randn(g, H, scale=0.3, mean=1.0), _randn(g, H, scale=0.2)


# each number of waves to a row and groups to a lane, at its ends
WIDTHS = [8, 16, 64, 72, 128, 136, 256, 264, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144, 6152, 8192, 8200, 12288, 12296, 16384]


@pytest.mark.parametrize("y", list(TYPES))
@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("H", WIDTHS)
def test_forward_and_gradient(H, x, y):
    T = 37 if H < 4096 else 11
    g = torch.Generator().manual_seed(H)
    v = _randn(g, T, H, dtype=TYPES[x], scale=2.0, mean=0.7)
    w, b = _affine(g, H)
    n = dpg.dpg_layer_norm(v, w, b, eps=EPS, out_dtype=TYPES[y])
    hv, hw, hb = ref.host(v), ref.host(w), ref.host(b)
    wy, wm, wr, ey, em, er = ref.layer_norm(hv, hw, hb, EPS)
    _check("y", n.y, wy, ey, TYPES[y])
    _check("mean", n.mean, wm, em)
    _check("rstd", n.rstd, wr, er)
    assert n.sum is None
    dy = _randn(g, T, H, dtype=TYPES[y])
    d = dpg.dpg_layer_norm_dgrad(dy, v, n.mean, n.rstd, w)
    dx, dw, db, ex, ew, eb = ref.layer_norm_dgrad(ref.host(dy), hv, ref.host(n.mean), ref.host(n.rstd), hw)
    _check("dx", d.dx, dx, ex, TYPES[x])
    _check("dweight", d.dweight, dw, ew)
    _check("dbias", d.dbias, db, eb)
    assert d.dresidual is None
    d2 = dpg.dpg_layer_norm_dgrad(dy, v, n.mean, n.rstd, w, weight_grads=False)
    assert torch.equal(d2.dx, d.dx) and d2.dweight is None and d2.dbias is None


@pytest.mark.parametrize("branch", list(TYPES))
@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("H", [8, 56, 120, 256, 520, 1024, 2048, 4096, 6144, 8192, 12288, 16384])
def test_residual_sum(H, x, branch):
    T, p, seed = (29 if H < 4096 else 7), 0.3, 0x123456789ABCDEF0 + H
    g = torch.Generator().manual_seed(H + 1)
    r = _randn(g, T, H, dtype=TYPES[x], scale=2.0)
    v = _randn(g, T, H, dtype=TYPES[branch])
    w, b = _affine(g, H)
    step = torch.tensor([5], device="cuda")
    n = dpg.dpg_add_layer_norm(v, r, w, b, eps=EPS, p=p, seed=seed, step=step, out_dtype=BF16)
    part = ref.dropped(ref.host(v), p, seed, 5)
    total = ref.host(r) + part
    e_total = ref.U * (2 * np.abs(part) + np.abs(total))
    _check("sum", n.sum, total, e_total, TYPES[x])
    wy, wm, wr, ey, em, er = ref.layer_norm(total, ref.host(w), ref.host(b), EPS)
    # the sum's own error, at most u' = 3 u of |r| + |part|, moves mean, differences and rstd as a change of the input
    big = 3 * ref.U * (np.abs(ref.host(r)) + np.abs(part))
    move = big + big.mean(1, keepdims=True)
    unit = np.abs(total - wm[:, None]) * wr[:, None]
    shift = wr[:, None] * (move + unit * (move * unit).mean(1, keepdims=True))
    _check("y", n.y, wy, ey + 1.01 * np.abs(ref.host(w)) * shift, BF16)
    _check("mean", n.mean, wm, em + big.mean(1))
    dy, dsum = _randn(g, T, H, dtype=BF16), _randn(g, T, H, dtype=TYPES[x])
    for extra in (dsum, None):
        d = dpg.dpg_add_layer_norm_dgrad(dy, n.sum, n.mean, n.rstd, w, dsum=extra, p=p, seed=seed, step=step,
                                         x_dtype=TYPES[branch])
        dv, dw, db, ev, ew, eb = ref.layer_norm_dgrad(ref.host(dy), ref.host(n.sum), ref.host(n.mean),
                                                      ref.host(n.rstd), ref.host(w))
        if extra is not None:
            dv = dv + ref.host(dsum)
            ev = ev + ref.U * np.abs(dv)
        _check("dresidual", d.dresidual, dv, ev, TYPES[x])
        scale = ref.keep_scale(p)
        _check("dx", d.dx, ref.dropped(dv, p, seed, 5), scale * (ev + 2 * ref.U * np.abs(dv)), TYPES[branch])
        _check("dweight", d.dweight, dw, ew)
        _check("dbias", d.dbias, db, eb)


@pytest.mark.parametrize("y", list(TYPES))
@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("H", [8, 64, 104, 248, 520, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 12296, 16384])
def test_many_rows(H, x, y):
    """Enough rows for the cuts that give each as few waves as hold it; the last
    rows are no whole round."""
    T = 1025 + 8 * (H % 3)
    g = torch.Generator(device="cuda").manual_seed(H)
    v = torch.randn(T, H, generator=g, device="cuda").mul_(2).add_(0.7).to(TYPES[x])
    w, b = _affine(torch.Generator().manual_seed(H), H)
    n = dpg.dpg_layer_norm(v, w, b, eps=EPS, out_dtype=TYPES[y])
    hw, hb = ref.host(w), ref.host(b)
    for rows in (slice(0, 9), slice(T // 2, T // 2 + 9), slice(T - 9, T)):
        wy, wm, wr, ey, em, er = ref.layer_norm(ref.host(v[rows]), hw, hb, EPS)
        _check("y", n.y[rows], wy, ey, TYPES[y])
        _check("mean", n.mean[rows], wm, em)
        _check("rstd", n.rstd[rows], wr, er)
    few = dpg.dpg_layer_norm(v[:7], w, b, eps=EPS, out_dtype=TYPES[y])  # another cut: as near as both bounds
    _, _, _, ey, em, _ = ref.layer_norm(ref.host(v[:7]), hw, hb, EPS)
    assert bool((np.abs(ref.host(few.mean) - ref.host(n.mean[:7])) <= 2 * em + 2 * ref.U * np.abs(ref.host(few.mean))).all())


def test_without_dropout_the_sum_is_a_sum():
    g = torch.Generator().manual_seed(2)
    x, r = _randn(g, 33, 264, dtype=BF16), _randn(g, 33, 264)
    n = dpg.dpg_add_layer_norm(x, r)
    assert torch.equal(n.sum, x.float() + r)
    m = dpg.dpg_layer_norm(n.sum, out_dtype=BF16)
    assert torch.equal(n.y, m.y) and torch.equal(n.mean, m.mean) and torch.equal(n.rstd, m.rstd)
    same = r.clone()
    n2 = dpg.dpg_add_layer_norm(x, same, sum=same)
    assert n2.sum.data_ptr() == same.data_ptr() and torch.equal(same, n.sum) and torch.equal(n2.y, n.y)


@pytest.mark.parametrize("H", [264, 2048, 8192])
def test_fused_and_separate_masks_agree(H):
    """The fused sum's mask is dpg_dropout's, and its gradient's too."""
    g = torch.Generator().manual_seed(3)
    x, r = _randn(g, 21, H, dtype=BF16), _randn(g, 21, H)
    n = dpg.dpg_add_layer_norm(x, r, p=0.5, seed=77)
    zero = torch.zeros_like(x)
    assert torch.equal(n.sum, dpg.dpg_dropout(x, 0.5, 77, residual=r))
    d = dpg.dpg_add_layer_norm_dgrad(zero, n.sum, n.mean, n.rstd, dsum=torch.ones_like(r), p=0.5, seed=77)
    assert torch.equal(d.dx, dpg.dpg_dropout(torch.ones_like(r), 0.5, 77, out_dtype=BF16))
    assert torch.equal(d.dx != 0, torch.from_numpy(ref.kept(21, H, 0.5, 77)).cuda())


def test_a_mean_far_from_zero():
    """Squares of differences, not a difference of squares: 300 and a spread of 1."""
    g = torch.Generator().manual_seed(4)
    x = _randn(g, 9, 4096, mean=300.0)
    n = dpg.dpg_layer_norm(x, eps=0.0)
    wy, wm, wr, ey, em, er = ref.layer_norm(ref.host(x), np.ones(4096), np.zeros(4096), 0.0)
    _check("rstd", n.rstd, wr, er)
    _check("y", n.y, wy, ey)
    assert float(np.abs(ref.host(n.rstd) - wr).max() / wr.max()) < 1e-4


def test_constant_rows_and_strange_values():
    x = torch.full((6, 2056), 3.0, device="cuda")
    x[1, 5], x[2, 2000], x[3, 7], x[3, 1999] = float("nan"), float("inf"), float("inf"), -float("inf")
    bias = torch.arange(2056, dtype=F32, device="cuda")
    n = dpg.dpg_layer_norm(x, None, bias)
    for row in (0, 4, 5):
        assert torch.equal(n.y[row], bias) and float(n.mean[row]) == 3.0
        assert abs(float(n.rstd[row]) - EPS ** -0.5) < 1e-4 * EPS ** -0.5
    assert bool(n.y[1:4].isnan().all())
    dy = torch.ones_like(x)
    d = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd)
    assert bool(d.dx[1:4].isnan().all()) and bool((d.dx[[0, 4, 5]] == 0).all())
    assert bool((d.dbias == 6).all())


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 511, 513, 4095, 4097, 5000])
@pytest.mark.parametrize("H", [40, 128, 248, 1032])
def test_row_counts(T, H):
    """Whole numbers: dbias is exact, whatever the cut over workgroups."""
    g = torch.Generator().manual_seed(T)
    x = _randn(g, T, H, dtype=BF16)
    dy = torch.randint(-8, 9, (T, H), generator=g).to(BF16).cuda()
    n = dpg.dpg_layer_norm(x)
    d = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd)
    assert torch.equal(d.dbias.double(), dy.double().sum(0))
    _, dw, _, _, ew, _ = ref.layer_norm_dgrad(ref.host(dy), ref.host(x), ref.host(n.mean), ref.host(n.rstd), 1.0)
    _check("dweight", d.dweight, dw, ew)
    wy, _, _, ey, _, _ = ref.layer_norm(ref.host(x), 1.0, 0.0, EPS)
    _check("y", n.y, wy, ey, BF16)


def test_strides_and_untouched_columns():
    g = torch.Generator().manual_seed(6)
    T, H, W = 19, 520, 544
    base = {k: torch.full((T, W), 7.0, dtype=BF16, device="cuda") for k in ("x", "r", "y", "sum", "dy", "ds")}
    cut = {k: t[:, 8:8 + H] for k, t in base.items()}
    for k in ("x", "r", "dy", "ds"):
        cut[k].copy_(_randn(g, T, H, dtype=BF16))
    w, b = _affine(g, H)
    n = dpg.dpg_add_layer_norm(cut["x"], cut["r"], w, b, p=0.2, seed=3, out=cut["y"], sum=cut["sum"])
    m = dpg.dpg_add_layer_norm(cut["x"].contiguous(), cut["r"].contiguous(), w, b, p=0.2, seed=3)
    assert torch.equal(cut["y"], m.y) and torch.equal(cut["sum"], m.sum)
    for k in ("y", "sum"):
        assert bool((base[k][:, :8] == 7).all()) and bool((base[k][:, 8 + H:] == 7).all())
    d = dpg.dpg_add_layer_norm_dgrad(cut["dy"], cut["sum"], n.mean, n.rstd, w, dsum=cut["ds"], p=0.2, seed=3)
    e = dpg.dpg_add_layer_norm_dgrad(cut["dy"].contiguous(), m.sum, m.mean, m.rstd, w, dsum=cut["ds"].contiguous(),
                                     p=0.2, seed=3)
    assert all(torch.equal(a, c) for a, c in zip(d, e))
    a = dpg.dpg_dropout(cut["x"], 0.4, 9, residual=cut["r"], out=cut["y"])
    c = dpg.dpg_dropout(cut["x"].contiguous(), 0.4, 9, residual=cut["r"].contiguous())
    assert torch.equal(a, c) and bool((base["y"][:, :8] == 7).all()) and bool((base["y"][:, 8 + H:] == 7).all())


def test_empty():
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    n = dpg.dpg_layer_norm(x)
    assert n.y.shape == (0, 64) and n.mean.shape == (0,)
    d = dpg.dpg_layer_norm_dgrad(x, x, n.mean, n.rstd)
    assert d.dx.shape == (0, 64) and bool((d.dweight == 0).all()) and bool((d.dbias == 0).all())
    assert dpg.dpg_dropout(x, 0.5, 1).shape == (0, 64)
    y = torch.zeros(5, 0, dtype=BF16, device="cuda")
    assert dpg.dpg_layer_norm(y).y.shape == (5, 0) and dpg.dpg_dropout(y, 0.5, 1).shape == (5, 0)


def test_gradient_against_differences():
    """Central differences of <y, dy> along random directions; with t = 2^-6 the
    truncation is below t^2 / 6 times the third derivative, which for rows of
    unit spread is below 40 |direction|^3 rstd^3 |dy w| per element; the outputs'
    FP32 errors are divided by 2 t."""
    g = torch.Generator().manual_seed(7)
    T, H, t = 6, 264, 2.0 ** -6
    x, dy = _randn(g, T, H, scale=2.0), _randn(g, T, H)
    w, b = _affine(g, H)
    n = dpg.dpg_layer_norm(x, w, b)
    d = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd, w)
    direction = _randn(g, T, H).sign()
    value, fp = {}, 0.0
    for s in (t, -t):
        z = x + s * direction
        value[s] = (dpg.dpg_layer_norm(z, w, b).y.double() * dy.double()).sum(1)
        _, _, _, ey, _, _ = ref.layer_norm(ref.host(z), ref.host(w), ref.host(b), EPS)
        # the argument itself is rounded: u of z, times the slope
        fp = fp + ((ey + ref.U * np.abs(ref.host(n.y))) * np.abs(ref.host(dy))).sum(1)
        fp = fp + (ref.U * np.abs(ref.host(z)) * np.abs(ref.host(d.dx))).sum(1) * 2
    slope = (d.dx.double() * direction.double()).sum(1)
    third = 40 * ref.host(n.rstd) ** 3 * np.abs(ref.host(dy) * ref.host(w)).sum(1)
    limit = fp / (2 * t) + t * t / 6 * third
    assert bool((np.abs(ref.host((value[t] - value[-t]) / (2 * t) - slope)) <= limit).all())
    # the weight and the bias enter linearly
    for name, grad in (("w", d.dweight), ("b", d.dbias)):
        for col in (0, 100, 263):
            args = {"w": w.clone(), "b": b.clone()}
            args[name][col] += 1
            new = dpg.dpg_layer_norm(x, args["w"], args["b"]).y
            change = float(((new - n.y).double() * dy.double())[:, col].sum())
            mag = float((dy.double().abs() * (n.y.double().abs() + new.double().abs()))[:, col].sum())
            assert abs(change - float(grad[col])) <= 16 * ref.U * mag + 60 * ref.U * mag


@pytest.mark.parametrize("out", [None, "f32", "bf16"])
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 8), (3, 264), (1000, 16), (5, 20000)])
def test_dropout(shape, x, residual, out):
    if residual and out and out != residual:
        return
    T, H = shape
    g = torch.Generator().manual_seed(T)
    v = _randn(g, T, H, dtype=TYPES[x])
    r = _randn(g, T, H, dtype=TYPES[residual]) if residual else None
    p, seed = 0.37, (1 << 63) + 12345
    step = torch.tensor([(7 << 32) + 3], device="cuda")
    y = dpg.dpg_dropout(v, p, seed, step=step, residual=r, out_dtype=TYPES[out] if out else None)
    part = ref.dropped(ref.host(v), p, seed, (7 << 32) + 3)
    want = part + (ref.host(r) if residual else 0.0)
    kind = TYPES[out or residual or x]
    _check("y", y, want, ref.U * (2 * np.abs(part) + np.abs(want)), kind)
    if not residual:
        assert np.array_equal(ref.host(y) != 0, (part != 0))


def test_the_generator():
    """Known answers of Philox4x32 with ten rounds: counter and key of zeros, and
    of ones."""
    w = ref.philox([0], 0, 0)
    assert [int(v) for v in w[:, 0]] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = (1 << 64) - 1
    w = ref.philox([ones], ones, ones)
    assert [int(v) for v in w[:, 0]] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_shares_and_steps():
    x = torch.ones(512, 4096, device="cuda")
    seen = []
    for p in (0.0, 0.1, 0.5, 0.999, 1.0):
        y = dpg.dpg_dropout(x, p, 5)
        bar = int(np.floor(p * 65536 + 0.5))
        left = float((y == 0).double().mean())
        # a binomial share of 2^21 elements, five standard deviations
        assert abs(left - bar / 65536) <= 5 * (bar / 65536 * (1 - bar / 65536) / x.numel()) ** 0.5
        kept = y[y != 0]
        if kept.numel():
            assert bool((kept == np.float32(ref.keep_scale(p))).all())
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(3):
        seen.append(dpg.dpg_dropout(x, 0.5, 5, step=step) == 0)
        step += 1
    assert torch.equal(seen[0], dpg.dpg_dropout(x, 0.5, 5) == 0)
    for a, b in ((0, 1), (1, 2), (0, 2)):
        same = float((seen[a] == seen[b]).double().mean())
        assert abs(same - 0.5) <= 5 * 0.5 / x.numel() ** 0.5
    other = dpg.dpg_dropout(x, 0.5, 6) == 0
    assert abs(float((seen[0] == other).double().mean()) - 0.5) <= 5 * 0.5 / x.numel() ** 0.5


def test_what_is_left_out_counts_as_zero():
    x = torch.full((64, 1024), float("nan"), device="cuda")
    mask = torch.from_numpy(ref.kept(64, 1024, 0.5, 8)).cuda()
    r = torch.ones_like(x)
    y = dpg.dpg_dropout(x, 0.5, 8, residual=r)
    assert torch.equal(y.isnan(), mask) and bool((y[~mask] == 1).all())
    assert bool((dpg.dpg_dropout(x, 1.0, 8, residual=r) == 1).all())


def test_dropout_in_place_and_versions():
    g = torch.Generator().manual_seed(1)
    x = _randn(g, 100, 64, dtype=BF16)
    want = dpg.dpg_dropout(x, 0.25, 3)
    version = x._version
    y = dpg.dpg_dropout(x, 0.25, 3, out=x)
    assert torch.equal(y, want) and x._version > version


def test_a_captured_step_counts_up():
    x = torch.ones(64, 1024, device="cuda")
    r = torch.zeros_like(x)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, total = torch.empty_like(x), torch.empty_like(x)
    dpg.dpg_dropout(x, 0.5, 11, step=step, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dpg.dpg_dropout(x, 0.5, 11, step=step, out=out)
        n = dpg.dpg_add_layer_norm(x, r, p=0.5, seed=12, step=step, sum=total)
        step += 1
    step.zero_()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        at = torch.tensor([i], device="cuda")
        assert torch.equal(out, dpg.dpg_dropout(x, 0.5, 11, step=at))
        m = dpg.dpg_add_layer_norm(x, r, p=0.5, seed=12, step=at)
        assert torch.equal(total, m.sum) and torch.equal(n.y, m.y)


def test_reruns_give_the_same_bits():
    g = torch.Generator().manual_seed(9)
    x, dy = _randn(g, 3000, 1032, dtype=BF16), _randn(g, 3000, 1032, dtype=BF16)
    w, b = _affine(g, 1032)
    n = dpg.dpg_layer_norm(x, w, b)
    first = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd, w)
    for _ in range(5):
        torch.empty(1 << 27, dtype=torch.uint8, device="cuda").fill_(0xff)
        assert torch.equal(dpg.dpg_layer_norm(x, w, b).y, n.y)
        again = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd, w)
        assert torch.equal(again.dx, first.dx) and torch.equal(again.dweight, first.dweight)
        assert torch.equal(again.dbias, first.dbias)


def test_other_streams():
    g = torch.Generator().manual_seed(10)
    x = _randn(g, 500, 1024, dtype=BF16)
    want = dpg.dpg_layer_norm(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = dpg.dpg_layer_norm(x, stream=side)
    d = dpg.dpg_dropout(x, 0.5, 2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n.y, want.y) and torch.equal(d, dpg.dpg_dropout(x, 0.5, 2))


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    n = dpg.dpg_layer_norm(x)
    with pytest.raises(TypeError):
        dpg.dpg_layer_norm(x, w.to(BF16))
    with pytest.raises(ValueError):
        dpg.dpg_layer_norm(x, w[:32])
    with pytest.raises(ValueError):
        dpg.dpg_layer_norm(x.view(2, 2, 64))
    with pytest.raises(ValueError):
        dpg.dpg_add_layer_norm(x, x[:2])
    with pytest.raises(TypeError):
        dpg.dpg_add_layer_norm(x, x, sum=torch.zeros(4, 64, device="cuda"))
    with pytest.raises(TypeError):
        dpg.dpg_layer_norm(x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        dpg.dpg_layer_norm_dgrad(x, x, n.mean[:2], n.rstd)
    with pytest.raises(TypeError):
        dpg.dpg_add_layer_norm_dgrad(x, x, n.mean, n.rstd, dsum=torch.zeros(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        dpg.dpg_dropout(x, 0.1, 1, step=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        dpg.dpg_dropout(x, 0.1, 1, step=torch.zeros(1, device="cuda"))
    with pytest.raises(TypeError):
        dpg.dpg_dropout(x, 0.1, "seed")
    with pytest.raises(TypeError):
        dpg.dpg_dropout(x, 0.1, 1, residual=x, out_dtype=F32)
    for call, status in ((lambda: dpg.dpg_dropout(x, 1.5, 1), 1), (lambda: dpg.dpg_dropout(x, float("nan"), 1), 1),
                         (lambda: dpg.dpg_layer_norm(x, eps=-1.0), 1),
                         (lambda: dpg.dpg_layer_norm(x[:, :60]), 3),
                         (lambda: dpg.dpg_layer_norm(torch.zeros(1, 16392, device="cuda")), 2),
                         (lambda: dpg.dpg_layer_norm_dgrad(x, x, n.mean, n.rstd, workspace=w), 4)):
        with pytest.raises(dpg.DpgError) as e:
            call()
        assert e.value.status == status
