"""The sizes of block_cases.py against the library's plans and the thresholds in the
sources: a rule that moves does not leave the kernels of large calls untested unseen."""
import ctypes
import os
import re

import pytest

import block_cases as cases
import deterministic_bf16_projection_amd as dpg

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_bf16_projection_amd",
                    "csrc")
I, Z = ctypes.c_int64, ctypes.c_size_t


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _once(text, pattern):
    found = re.findall(pattern, text)
    assert len(found) == 1, (pattern, found)
    return found[0]


def _recurrence_plan(S, R, D, packed):
    """tiles of an axis, spans of it, from the sizes of what a call has to bring."""
    sizes = {}
    for name in ("workspace", "carries"):
        f = getattr(dpg.lib(), "dpg_recurrence_%s_size" % name)
        f.restype = Z
        sizes[name] = f(I(S), I(R), I(D), 0, int(packed))
    rows = R if packed else R // S * max(1, 128 // (R // S))
    axes = -(-R // rows)
    tiles = sizes["carries"] // (4 * D * 2 * axes)
    assert tiles == -(-rows // 128)
    left = sizes["workspace"] - (-(-4 * R // 16) * 16 if packed else 0)
    if left == 0:
        return tiles, 1
    spans, rest = divmod(left - 4 * S * D, 4 * D * 2 * axes)
    assert rest == 0 and spans > 1
    return tiles, spans


def test_spans_have_several_tiles():
    plans = [_recurrence_plan(B, B * T, D, False) for B, T, D in cases.SPANS]
    plans += [_recurrence_plan(len(off) - 1, R, D, True) for off, R, D in cases.PACKED_SPANS]
    assert all(1 < spans < tiles for tiles, spans in plans)
    # a last span of fewer tiles, one of as many, and one of a single tile
    left = {tiles - (spans - 1) * -(-tiles // spans) - -(-tiles // spans) for tiles, spans in plans}
    assert 0 in left and min(left) < 0
    assert any(tiles % -(-tiles // spans) == 1 for tiles, spans in plans)
    # borders of packed sequences at, next to and away from those of the spans
    for off, R, D in cases.PACKED_SPANS[:1]:
        tiles, spans = _recurrence_plan(len(off) - 1, R, D, True)
        border = [128 * -(-tiles // spans) * i for i in range(1, spans)]
        assert set(border) & set(off) and any(abs(o - b) == 1 for o in off for b in border)


@pytest.mark.parametrize("source", ["dpg_recurrence.hip", "dpg_norm.hip"])
def test_streamed_calls_are_streamed_and_those_below_not(source):
    pattern = r"return R \* D >= \(int64_t\)\(([0-9 <]+)\) / elt" if "rec" in source else \
        r"past = T \* H >= \(int64_t\)\(([0-9 <]+)\) / elt_size"
    least = eval(_once(_source(source), pattern), {"__builtins__": {}})
    size = {"bf16": 2, "f32": 4}
    if "rec" in source:
        shares = [(k, B * T * D * size[k] / least) for k, B, T, D in cases.STREAMED]
        shares += [(k, R * D * size[k] / least) for k, _, R, D in cases.PACKED_STREAMED]
        assert any(_recurrence_plan(B, B * T, D, False)[1] == 1 for k, B, T, D in cases.STREAMED if B * T * D * size[k] >= least)
        assert any(_recurrence_plan(B, B * T, D, False)[1] > 1 for k, B, T, D in cases.STREAMED if B * T * D * size[k] >= least)
    else:
        shares = [(k, T * H * size[k] / least) for k, T, H, _ in cases.DROPOUT]
        assert all(T * H // 8 % 512 for _, T, H, _ in cases.DROPOUT)
    for kind in size:
        s = [v for k, v in shares if k == kind]
        assert any(0.99 < v < 1 for v in s) and any(1 <= v < 1.01 for v in s)


def test_norms_go_through_three_rounds():
    text = _source("dpg_norm.hip")
    assert int(_once(text, r"kNormManyRows = ([0-9]+);")) <= min(T for T, _ in cases.NORM)
    assert _once(text, r"norm_shares_weights\(l.chunks\) \? ([0-9]+) : ([0-9]+); }") == ("512", "2048")
    assert _once(text, r"kGradBlocks = ([0-9]+);") == "256"
    assert "return H <= 64 ? 8 : H <= 128 ? 16 : H <= 256 ? 32 : 64;" in text
    for T, H in cases.NORM:
        step = cases.norm_round(H, True, False)
        assert T > 2 * step and T % step, (T, H)
    for T, H in cases.ADD_NORM:
        step = cases.norm_round(H, True, True)
        assert T > 2 * step and T % step, (T, H)
    size = dpg.lib().dpg_layer_norm_workspace_size
    size.restype = Z
    for T, H in cases.NORM_GRADIENT:
        step = cases.norm_gradient_round(H)
        assert T > 3 * step and T % step, (T, H)
        assert size(I(T), I(H)) == 256 * 2 * 4 * H
    # every cut: groups of eight to a lane by lanes of a row, and rows over several waves
    assert {cases.norm_lanes(H) for _, H in cases.NORM} == {8, 16, 32, 64}
