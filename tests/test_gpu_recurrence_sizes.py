"""The gated recurrence at the sizes of large calls (block_cases.py): spans of
several tiles, accesses past the caches, equal and packed, outputs over inputs.

Tolerances: the bounds of block_reference plus the rounding to the output's type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_cases as cases  # noqa: E402
from test_gpu_recurrence import BF16, F32, _compare, _inputs, _run  # noqa: E402

TYPES = {"bf16": BF16, "f32": F32}


def _columns(D):
    """Channels at the ends of a workgroup's 128 and of the matrix."""
    return sorted({c for c in (0, 1, 2, 63, 64, 65, 126, 127, 128, 129, D // 2, D // 2 + 1, D - 9, D - 8, D - 2, D - 1)
                   if 0 <= c < D})


def _check(d, offsets, R, D, coupled, shape):
    r, b = _run(d, offsets, coupled, shape)
    at = torch.tensor(_columns(D), device="cuda")
    cut = lambda t: t.reshape(-1, D)[:, at]  # noqa: E731
    assert r.h.numel() == R * D
    _compare({k: cut(v) for k, v in d.items()}, offsets, coupled, r._replace(h=cut(r.h), state=cut(r.state)),
             b._replace(dgate=cut(b.dgate), dx=cut(b.dx), dstate=cut(b.dstate)))
    # over the input, and the state over its own, with the same bits
    view = (lambda t: t.view(*shape)) if shape else lambda t: t
    off = None if shape else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, state = view(d["x"].clone()), d["state"].clone()
    own = dpg.dpg_recurrence(view(d["gate"]), x, offsets=off, state=state, coupled=coupled, carries=True, out=x,
                             state_out=state)
    same = lambda a, b: torch.equal(a.nan_to_num(nan=123.0), b.nan_to_num(nan=123.0))  # noqa: E731
    assert same(x, r.h) and same(state, r.state) and same(own.carries, r.carries)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("case", cases.SPANS, ids=str)
def test_spans_of_several_tiles(case, coupled, dtype):
    B, T, D = case
    d = _inputs(B * T, B, D, TYPES[dtype], seed=B * T + D)
    _check(d, [T * i for i in range(B + 1)], B * T, D, coupled, case)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("case", cases.PACKED_SPANS, ids=lambda c: "%s of %d x %d" % (c[0], c[1], c[2]))
def test_packed_spans_of_several_tiles(case, coupled, dtype):
    offsets, R, D = case
    d = _inputs(R, len(offsets) - 1, D, TYPES[dtype], seed=R + len(offsets))
    _check(d, offsets, R, D, coupled, None)


@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("case", cases.STREAMED, ids=str)
def test_past_the_caches(case, coupled):
    kind, B, T, D = case
    d = _inputs(B * T, B, D, TYPES[kind], seed=B * T)
    _check(d, [T * i for i in range(B + 1)], B * T, D, coupled, (B, T, D))


@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("case", cases.PACKED_STREAMED, ids=lambda c: c[0])
def test_packed_past_the_caches(case, coupled):
    kind, offsets, R, D = case
    d = _inputs(R, len(offsets) - 1, D, TYPES[kind], seed=R)
    _check(d, offsets, R, D, coupled, None)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
def test_strange_gates_in_spans_of_several_tiles(coupled, dtype):
    """Gates of NaN, and of -infinity that end one, next to the borders of runs,
    tiles and spans (384), with and without a gradient from behind."""
    B, T, D = cases.SPANS[1]
    d = _inputs(B * T, B, D, TYPES[dtype], seed=4)
    at = _columns(D)
    for i, c in enumerate(at):
        t = (0, 7, 8, 127, 128, 255, 256, 383, 384, 385, 511, 512, 599)[i % 13]
        d["gate"][t, c] = float("nan")
        if i % 3 and t + 2 < T:
            d["gate"][min(T - 1, t + (1, 150)[i % 2]), c] = -float("inf")
        if i % 5 == 0:
            d["dh"][t:, c] = 0
            d["dstate"][0, c] = 0
    _check(d, [0, T], T, D, coupled, (B, T, D))
