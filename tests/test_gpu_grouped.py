"""Grouped products on the GPU.  Integer inputs small enough that every sum is
exact in FP32 make the comparison with the 64-bit product bit for bit: FP32
outputs equal it, BF16 outputs are its nearest-even rounding.  Memory that a
call must not read holds NaN, memory that it must not write a sentinel."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

NAN = float("nan")


def _ints(g, *shape):
    return torch.from_numpy(g.integers(-4, 5, shape).astype(np.float32)).cuda().to(torch.bfloat16)


def _padded(t, pad, fill=NAN):
    """t as a view of wider rows (pad more elements), the padding filled."""
    if not pad:
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _ref(pass_, counts, R, a, b, E):
    a, b = a.double().cpu(), b.double().cpu()
    off = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    if pass_ == "wgrad":
        return torch.stack([a[i:j].T @ b[i:j] for i, j in zip(off, off[1:])]) if E else a.new_zeros(0, a.shape[1], b.shape[1])
    cols = b.shape[1] if pass_ == "forward" else b.shape[2]
    out = torch.zeros(R, cols, dtype=torch.float64)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        out[i:j] = a[i:j] @ (b[e].T if pass_ == "forward" else b[e])
    return out


def _check(pass_, counts, N, K, out_dtype, tail=0, pad=0, seed=0):
    g = np.random.default_rng(seed)
    E, R = len(counts), int(sum(counts)) + tail
    x, dy, w = _ints(g, R, K), _ints(g, R, N), _ints(g, E, N, K)
    if tail:  # rows of no group are not read
        x[R - tail:] = NAN
        dy[R - tail:] = NAN
    a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[pass_]
    ref = _ref(pass_, counts, R, a, b, E)
    shape = tuple(ref.shape)
    wide = torch.full((*shape[:-1], shape[-1] + pad), 7.0, dtype=out_dtype, device="cuda")
    out = wide[..., :shape[-1]]
    fn = getattr(dpg, "dpg_grouped_" + pass_)
    got = fn(_padded(a, pad), _padded(b, pad), _offsets(counts), out=out)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), ref.to(out_dtype)), (pass_, counts, N, K)
    assert bool((wide[..., shape[-1]:] == 7.0).all())


PASSES = ("forward", "dgrad", "wgrad")
COUNTS = {
    "one row": [1],
    "one of many": [0, 0, 1, 0, 0],
    "empty ends": [0, 17, 0, 130, 0],
    "tile edges": [255, 256, 257, 1, 127, 128, 129],
    "skewed": [700, 3, 0, 64, 65, 1, 1, 200],
    "hundred": [(7 * i) % 5 for i in range(100)],
}


@pytest.mark.parametrize("pass_", PASSES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_group_sizes(pass_, out_dtype, counts):
    _check(pass_, counts, 264, 328, out_dtype)


@pytest.mark.parametrize("pass_", PASSES)
@pytest.mark.parametrize("N,K", [(8, 8), (64, 64), (72, 200), (512, 8), (8, 1032), (256, 1024)])
@pytest.mark.parametrize("rows", [3, 300])
def test_odd_shapes(pass_, N, K, rows):
    _check(pass_, [rows, 0, 2 * rows + 1], N, K, torch.float32, seed=N + K)


@pytest.mark.parametrize("pass_", PASSES)
@pytest.mark.parametrize("tail", [1, 40, 600])
def test_rows_of_no_group_are_not_read_and_give_zeros(pass_, tail):
    _check(pass_, [5, 0, 90], 136, 72, torch.bfloat16, tail=tail)
    _check(pass_, [300, 280], 264, 136, torch.float32, tail=tail)


@pytest.mark.parametrize("pass_", PASSES)
@pytest.mark.parametrize("counts", [[3, 0, 20], [260, 500]])
def test_padded_strides(pass_, counts):
    _check(pass_, counts, 136, 200, torch.bfloat16, pad=24)
    _check(pass_, counts, 264, 264, torch.float32, tail=9, pad=8)


@pytest.mark.parametrize("pass_", PASSES)
def test_all_rows_in_no_group_and_no_rows(pass_):
    _check(pass_, [0, 0, 0], 64, 64, torch.float32, tail=33)
    _check(pass_, [0, 0], 64, 64, torch.bfloat16)


def test_no_groups():
    x = torch.full((50, 64), NAN, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(0, 128, 64, dtype=torch.bfloat16, device="cuda")
    off = _offsets([])
    assert float(dpg.dpg_grouped_forward(x, w, off).abs().sum()) == 0.0
    assert dpg.dpg_grouped_wgrad(torch.zeros(50, 128, dtype=torch.bfloat16, device="cuda"), x, off).shape == (0, 128, 64)


@pytest.mark.parametrize("pass_", PASSES)
def test_empty_reduction_writes_zeros(pass_):
    N, K = {"forward": (64, 0), "dgrad": (0, 64), "wgrad": (64, 64)}[pass_]
    _check(pass_, [0, 0] if pass_ == "wgrad" else [20, 300], N, K, torch.float32)


def test_one_group_equals_the_projection():
    """With one group the product is the plain projection: the same sums."""
    g = np.random.default_rng(5)
    x, w, dy = _ints(g, 777, 512), _ints(g, 1, 1024, 512), _ints(g, 777, 1024)
    off = _offsets([777])
    for got, ref in ((dpg.dpg_grouped_forward(x, w, off), dpg.dpg_forward(x, w[0])),
                     (dpg.dpg_grouped_dgrad(dy, w, off), dpg.dpg_dgrad(dy, w[0])),
                     (dpg.dpg_grouped_wgrad(dy, x, off)[0], dpg.dpg_wgrad(dy, x))):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("pass_", PASSES)
def test_shared_weight_and_side_by_side_gradients(pass_):
    """One weight for all groups (stride 0); gradients of the groups side by
    side in one wider matrix."""
    g = np.random.default_rng(6)
    counts, N, K = [40, 0, 100], 72, 136
    x, dy, w = _ints(g, 140, K), _ints(g, 140, N), _ints(g, N, K)
    if pass_ == "wgrad":
        wide = torch.zeros(N, 3, K, dtype=torch.float32, device="cuda")
        out = wide.permute(1, 0, 2)
        dpg.dpg_grouped_wgrad(dy, x, _offsets(counts), out=out)
        assert torch.equal(out.double().cpu(), _ref(pass_, counts, 140, dy, x, 3))
    else:
        we = w.expand(3, N, K)
        a = x if pass_ == "forward" else dy
        got = getattr(dpg, "dpg_grouped_" + pass_)(a, we, _offsets(counts), out_dtype=torch.float32)
        assert torch.equal(got.double().cpu(), _ref(pass_, counts, 140, a, we, 3))


@pytest.mark.parametrize("pass_", PASSES)
def test_real_values_within_the_rounding_bound(pass_):
    """Normal inputs: an FP32 sum of n products is off by at most n 2^-24 times
    the sum of their magnitudes (each addition half a step of at most that
    sum), and BF16 rounding adds 2^-8 of the value."""
    g = torch.Generator().manual_seed(3)
    counts, N, K = [100, 0, 333, 1, 70], 520, 712
    R, E = sum(counts), len(counts)
    x, dy, w = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((R, K), (R, N), (E, N, K)))
    a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[pass_]
    ref, mag = _ref(pass_, counts, R, a, b, E), _ref(pass_, counts, R, a.abs(), b.abs(), E)
    n = {"forward": K, "dgrad": N, "wgrad": max(counts)}[pass_]
    bound = n * 2.0 ** -24 * mag
    fn = getattr(dpg, "dpg_grouped_" + pass_)
    for dtype in (torch.float32, torch.bfloat16):
        got = fn(a, b, _offsets(counts), out_dtype=dtype).double().cpu()
        limit = bound if dtype == torch.float32 else bound + 2.0 ** -8 * (ref.abs() + bound)
        assert bool(((got - ref).abs() <= limit).all())


@pytest.mark.parametrize("pass_", PASSES)
def test_infinities_stay_in_their_group(pass_):
    """NaN and infinity in one group's rows or weight leave the others' outputs as they are."""
    g = np.random.default_rng(8)
    counts, N, K = [70, 90, 60], 136, 200
    x, dy, w = _ints(g, 220, K), _ints(g, 220, N), _ints(g, 3, N, K)
    a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[pass_]
    ref = _ref(pass_, counts, 220, a, b, 3)
    a[70:160] = NAN
    if pass_ == "wgrad":
        b[70:160] = float("inf")
    else:
        b[1] = float("inf")
    got = getattr(dpg, "dpg_grouped_" + pass_)(a, b, _offsets(counts), out_dtype=torch.float32).double().cpu()
    parts = (0, 2) if pass_ == "wgrad" else (slice(0, 70), slice(160, 220))
    for p in parts:
        assert torch.equal(got[p], ref[p])


def test_wrong_offsets_stay_in_bounds():
    """Offsets outside the rows, or descending, are clamped: some values, no
    access outside; what lies around the matrices stays as it is."""
    g = np.random.default_rng(9)
    x, dy, w = _ints(g, 100, 64), _ints(g, 100, 128), _ints(g, 4, 128, 64)
    for off in ([0, 500, 700, 90, 100], [-7, -3, 50, 20, 100], [0, 2 ** 31 - 1, 0, -2 ** 31, 9]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        wide = torch.full((102, 128), 7.0, dtype=torch.float32, device="cuda")
        dpg.dpg_grouped_forward(x, w, off, out=wide[1:101])
        dpg.dpg_grouped_dgrad(dy, w, off)
        dpg.dpg_grouped_wgrad(dy, x, off)
        torch.cuda.synchronize()
        assert bool((wide[[0, 101]] == 7.0).all())


@pytest.mark.parametrize("pass_", PASSES)
def test_reruns_streams_and_graph_replays_are_bitwise_equal(pass_):
    g = torch.Generator().manual_seed(4)
    counts = [130, 0, 400, 31]
    R, N, K = sum(counts), 264, 520
    x, dy, w = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((R, K), (R, N), (4, N, K)))
    a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[pass_]
    off = _offsets(counts)
    fn = getattr(dpg, "dpg_grouped_" + pass_)
    first = fn(a, b, off)
    assert all(torch.equal(first, fn(a, b, off)) for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fn(a, b, off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(a, b, off, out=out)
    for shift in (0, 5, -9):  # the group sizes are read at every replay
        off[1:4] += shift
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fn(a, b, off))


def _workspace(pass_, E, R, N, K):
    fn = dpg.lib().dpg_grouped_workspace_size
    fn.argtypes, fn.restype = [ctypes.c_int] + [ctypes.c_int64] * 4, ctypes.c_size_t
    return fn(PASSES.index(pass_), E, R, N, K)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pass_,counts,N,K,tail,split", [
    ("forward", [700, 0, 300], 520, 4096, 0, True), ("forward", [700, 90], 1024, 2056, 33, True),
    ("dgrad", [3000, 0, 900], 4096, 520, 0, True), ("dgrad", [2500], 2056, 264, 70, True),
    ("wgrad", [3000], 264, 136, 0, True), ("wgrad", [2000, 0, 5, 1700], 520, 264, 40, True),
    ("forward", [1, 0, 3, 0, 2], 1024, 4096, 5, False), ("forward", [16, 17, 33, 64, 65], 520, 2056, 9, False),
    ("dgrad", [1, 0, 3, 0, 2], 1024, 4096, 5, False), ("dgrad", [16, 17, 33], 520, 2056, 9, False)])
def test_split_reductions_and_few_rows(pass_, counts, N, K, tail, split, out_dtype):
    """Long reductions of few output tiles are split; the few-row kernels take
    what their row tiles do not fill.  Sums below 2^24: exact."""
    assert (_workspace(pass_, len(counts), sum(counts) + tail, N, K) > 0) == split
    _check(pass_, counts, N, K, out_dtype, tail=tail, pad=8)


def test_workspace():
    g = np.random.default_rng(10)
    dy, x, off = _ints(g, 3000, 264), _ints(g, 3000, 136), _offsets([3000])
    need = _workspace("wgrad", 1, 3000, 264, 136)
    first = dpg.dpg_grouped_wgrad(dy, x, off)
    own = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(dpg.dpg_grouped_wgrad(dy, x, off, workspace=own), first)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_grouped_wgrad(dy, x, off, workspace=own[:need - 16])
    with pytest.raises(ValueError):
        dpg.dpg_grouped_wgrad(dy, x, off, workspace=own.cpu())


def test_refusals():
    x = torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 256, 128, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    off = _offsets([10, 20])
    with pytest.raises(TypeError):
        dpg.dpg_grouped_forward(x, w, off.long())
    with pytest.raises(ValueError):
        dpg.dpg_grouped_forward(x, w, _offsets([10, 20, 30]))
    with pytest.raises(ValueError):
        dpg.dpg_grouped_forward(x, w, off.cpu())
    with pytest.raises(ValueError):
        dpg.dpg_grouped_forward(dy, w, off)
    with pytest.raises(ValueError):
        dpg.dpg_grouped_dgrad(x, w, off)
    with pytest.raises(ValueError):
        dpg.dpg_grouped_wgrad(dy[:60], x, off)
    with pytest.raises(TypeError):
        dpg.dpg_grouped_forward(x.float(), w, off)
    with pytest.raises(ValueError):
        dpg.dpg_grouped_forward(x, w, off, out=torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dpg.DpgError):
        dpg.dpg_grouped_forward(x[:, :100], w[:, :, :100], off)  # 100 is no multiple of 8
