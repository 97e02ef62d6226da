"""The grouped products' plan description, without a GPU."""
import ctypes

import pytest

import tile_cases

dpg = pytest.importorskip("deterministic_bf16_projection_amd")

I = ctypes.c_int64
L = dpg.lib()
PASSES = (dpg.PASS_FORWARD, dpg.PASS_DGRAD, dpg.PASS_WGRAD)


def plan(pass_, E, R, N, K):
    return dpg.parse_plan(dpg.grouped_plan_describe(pass_, E, R, N, K))


@pytest.mark.parametrize("pass_", PASSES)
def test_description_and_workspace_agree(pass_):
    size = L.dpg_grouped_workspace_size
    size.restype = ctypes.c_size_t
    seen = set()
    for E in (1, 3, 64, 300):
        for R in (1, 40, 3000, 40000):
            for N, K in ((64, 64), (520, 4096), (4096, 520), (1024, 1024)):
                p = plan(pass_, E, R, N, K)
                assert int(p["workspace"]) == size(pass_, I(E), I(R), I(N), I(K))
                outputs = {0: R * N, 1: R * K, 2: E * N * K}[pass_]
                assert int(p["workspace"]) == (0 if p["splits"] == "1" else int(p["splits"]) * outputs * 4)
                assert int(p["grid"]) == min(int(p["units"]), 256 * (1 if p["tile"] == "256x256" else 2))
                assert (p["kernel"] == "few_rows") == (p["tile"] in ("16x16", "32x32", "16x128"))
                seen.add(p["tile"])
    assert seen >= {"256x256", "128x128"} and (pass_ == dpg.PASS_WGRAD) == (seen == {"256x256", "128x128"})


def test_description_refusals():
    buf = ctypes.create_string_buffer(16)
    f = L.dpg_grouped_plan_describe
    assert f(0, I(-1), I(8), I(8), I(8), buf, 16) == 1 and f(2, I(1), I(8), I(8), I(-8), buf, 16) == 1
    assert f(3, I(1), I(8), I(8), I(8), buf, 16) == 1
    assert f(0, I(1), I(8), I(8), I(8), None, 0) == 1
    assert f(0, I(1 << 24), I(8), I(8), I(8), buf, 16) == 2 and f(1, I(1), I(1 << 31), I(8), I(8), buf, 16) == 2
    assert f(2, I((1 << 24) - 1), I(8), I((1 << 31) - 520), I((1 << 31) - 520), buf, 16) == 2
    assert f(0, I(1), I(8), I(8), I(8), buf, 16) == 0 and len(buf.value) == 15  # truncated, with its end
    with pytest.raises(dpg.DpgError):
        dpg.grouped_plan_describe(dpg.PASS_FORWARD, 1, -1, 8, 8)
    for args in ((0, 0, 0, 0), (1, 0, 64, 64), (0, 50, 64, 64)):
        assert plan(dpg.PASS_WGRAD, *args)["splits"] == "1"


@pytest.mark.parametrize("case", tile_cases.TILES, ids=tile_cases.ident)
def test_the_tile_cases_take_their_kernels(case):
    """The sizes that test_gpu_grouped_tiles.py runs reach the kernels they stand for."""
    pass_, counts, tail, N, K, tile, ordered = case
    p = plan(("forward", "dgrad", "wgrad").index(pass_), len(counts), sum(counts) + tail, N, K)
    assert (p["kernel"], p["tile"], p["splits"]) == ("pipelined", tile, "1")
    if ordered is not None:
        assert p["ordered"] == str(ordered)
        if len(counts) > 256:  # not ordered, and several rounds of the grid
            assert int(p["units"]) > int(p["grid"])


def test_the_tile_cases_cover_every_kernel():
    seen = {(c[0], c[5], c[6]) for c in tile_cases.TILES}
    assert seen == {(p, t, None) for p in ("forward", "dgrad") for t in ("256x256", "128x128")} | {
        ("wgrad", t, o) for t in ("256x256", "128x128") for o in (0, 1)}


@pytest.mark.parametrize("N", [1 << 24, (1 << 29) + 1032])
def test_one_wide_row_takes_a_tile(N):
    p = plan(dpg.PASS_FORWARD, 1, 1, N, 8)
    assert (p["kernel"], p["splits"]) == ("pipelined", "1")
