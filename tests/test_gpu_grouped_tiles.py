"""The grouped products' large tiles on the GPU, at sizes that the plan sends to
them (tile_cases.py).  Whole numbers whose sums are exact in FP32 are compared
with 64-bit products bit for bit, as in test_gpu_grouped.py; memory that a call
must not read holds NaN, memory that it must not write a sentinel."""
import numpy as np
import pytest
import torch

import tile_cases

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


NAN, INF = float("nan"), float("inf")
SIZES = {p: [c for c in tile_cases.TILES if c[0] == p] for p in ("forward", "dgrad", "wgrad")}


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _operands(case, make):
    """The two operands, without the rows of no group set apart."""
    pass_, counts, tail, N, K = case[:5]
    E, R = len(counts), sum(counts) + tail
    x, dy, w = (lambda: make(R, K)), (lambda: make(R, N)), (lambda: make(E, N, K))
    return {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[pass_]


def _ints(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").to(torch.bfloat16)


def _ref(case, a, b):
    """64-bit products, group by group."""
    pass_, counts, tail, N, K = case[:5]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    shape = {"forward": (len(a), N), "dgrad": (len(a), K), "wgrad": (len(counts), N, K)}[pass_]
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for e, (i, j) in enumerate(zip(off, off[1:])):
        if i == j:
            continue
        rows = a[i:j].double()
        if pass_ == "wgrad":
            out[e] = rows.t().contiguous() @ b[i:j].double()
        else:
            out[i:j] = rows @ (b[e].double().t().contiguous() if pass_ == "forward" else b[e].double())
    return out


def _padded(t, pad):
    if not pad:
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), NAN, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _call(case, a, b, off, **kw):
    return getattr(dpg, "dpg_grouped_" + case[0])(a, b, off, **kw)


def _check(case, a, b, ref, out_dtype, pad, pad_out):
    """One call into the middle of a wider, longer buffer of sevens."""
    cols = ref.shape[-1]
    lead = (ref.shape[0] + 2,) + tuple(ref.shape[1:-1])
    wide = torch.full((*lead, cols + pad_out), 7.0, dtype=out_dtype, device="cuda")
    out = wide[1:-1, ..., :cols]
    _call(case, _padded(a, pad), _padded(b, pad), _offsets(case[1]), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, ref.to(out_dtype)), (out_dtype, pad, pad_out)
    assert bool((wide[0] == 7.0).all()) and bool((wide[-1] == 7.0).all()) and bool((wide[..., cols:] == 7.0).all())


@pytest.mark.parametrize("case", tile_cases.TILES, ids=tile_cases.ident)
def test_whole_numbers(case):
    """Both output types; rows of whole 64-byte pieces (written past the caches)
    and others, tight and padded by 8 (16 or 32 bytes) and by 64 elements."""
    a, b = (make() for make in _operands(case, _ints(len(case[1]) + case[3])))
    if case[2]:  # rows of no group: not read
        a[-case[2]:] = NAN
        if case[0] == "wgrad":
            b[-case[2]:] = NAN
    ref = _ref(case, a, b)
    for out_dtype in (torch.bfloat16, torch.float32):
        for pad, pad_out in ((0, 0), (8, 8), (64, 64)):
            _check(case, a, b, ref, out_dtype, pad, pad_out)


@pytest.mark.parametrize("case", [c for p in SIZES for c in SIZES[p][:3]], ids=tile_cases.ident)
def test_infinities_stay_in_their_group(case):
    """NaN rows and an infinite weight in the largest group: the other groups'
    outputs are as without them."""
    pass_, counts, tail = case[:3]
    a, b = (make() for make in _operands(case, _ints(1)))
    ref = _ref(case, a, b)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    e = int(np.argmax(counts))
    a[off[e]:off[e + 1]] = NAN
    if pass_ == "wgrad":
        b[off[e]:off[e + 1]] = INF
    else:
        b[e] = INF
    for out_dtype in (torch.bfloat16, torch.float32):
        got = _call(case, a, b, _offsets(counts), out_dtype=out_dtype)
        want = ref.to(out_dtype)
        if pass_ == "wgrad":
            keep = [i for i in range(len(counts)) if i != e]
            assert torch.equal(got[keep], want[keep])
            assert bool(torch.isnan(got[e]).all())
        else:
            used = int(off[-1])
            assert torch.equal(got[:off[e]], want[:off[e]])
            assert torch.equal(got[off[e + 1]:used], want[off[e + 1]:used])
            assert bool((got[used:] == 0).all()) and bool(torch.isnan(got[off[e]:off[e + 1]]).all())


@pytest.mark.parametrize("case", [c for p in SIZES for c in SIZES[p][:4]], ids=tile_cases.ident)
def test_wrong_offsets_stay_in_bounds(case):
    """Offsets outside the rows, or descending, are clamped: some values, and what
    lies around the output stays as it is."""
    pass_, counts, tail, N, K = case[:5]
    E, R = len(counts), sum(counts) + tail
    a, b = (make() for make in _operands(case, _ints(2)))
    good = _offsets(counts)
    far = good * 3 + R // 2
    down = good.flip(0).contiguous()
    wild = good.clone()
    wild[1::3] = 2 ** 31 - 1
    wild[2::3] = -2 ** 31
    shape = (E + 2, N, K) if pass_ == "wgrad" else (R + 2, N if pass_ == "forward" else K)
    for off in (far, down, wild, good - R // 3):
        for out_dtype in (torch.bfloat16, torch.float32):
            wide = torch.full(shape, 7.0, dtype=out_dtype, device="cuda")
            _call(case, a, b, off, out=wide[1:-1])
            torch.cuda.synchronize()
            assert bool((wide[0] == 7.0).all()) and bool((wide[-1] == 7.0).all())


@pytest.mark.parametrize("case", [c for p in SIZES for c in SIZES[p][:3]], ids=tile_cases.ident)
def test_real_values_within_the_rounding_bound(case):
    """Normal inputs: an FP32 sum of n products is off by at most n 2^-24 times the
    sum of their magnitudes (each addition half a step of at most that sum), and
    BF16 rounding adds 2^-8 of the value."""
    g = torch.Generator(device="cuda").manual_seed(3)
    pass_, counts, tail, N, K = case[:5]
    a, b = (make() for make in _operands(case, lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)))
    ref, mag = _ref(case, a, b), _ref(case, a.abs(), b.abs())
    bound = {"forward": K, "dgrad": N, "wgrad": max(counts)}[pass_] * 2.0 ** -24 * mag
    for out_dtype in (torch.float32, torch.bfloat16):
        got = _call(case, a, b, _offsets(counts), out_dtype=out_dtype).double()
        limit = bound if out_dtype == torch.float32 else bound + 2.0 ** -8 * (ref.abs() + bound)
        assert bool(((got - ref).abs() <= limit).all())


@pytest.mark.parametrize("case", [SIZES["forward"][2], SIZES["dgrad"][2], SIZES["wgrad"][1], SIZES["wgrad"][3]],
                         ids=tile_cases.ident)
def test_reruns_and_graph_replays_are_bitwise_equal(case):
    """The group sizes are read at every replay; eager work lies between the replays."""
    g = torch.Generator(device="cuda").manual_seed(4)
    a, b = (make() for make in _operands(case, lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)))
    off = _offsets(case[1])
    first = _call(case, a, b, off)
    assert all(torch.equal(first, _call(case, a, b, off)) for _ in range(3))
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(case, a, b, off, out=out)
    for shift in (0, 37, -64):
        off[1:-1] = (off[1:-1] + shift).clamp(min=0)
        off[1:-1] = torch.minimum(off[1:-1], off[-1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _call(case, a, b, off))
