"""The gated recurrence against 64-bit references: lengths from one row to
several tiles and spans, packed and equal sequences, states, strides, gates and
inputs that are infinite or NaN, and reruns.

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


def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _check(name, got, want, bound, dtype):
    got = ref.host(got).reshape(want.shape)
    limit = bound * 1.01 + ref.half_step(dtype) * (np.abs(want) + bound) + 1e-37
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want)), name
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]), name
    bad = np.abs(got - want)[fine] > limit[fine]
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - want)[fine] / limit[fine]).max()))


def _inputs(R, S, D, dtype, seed, state=True, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    gate = _randn(g, R, D, dtype=F32, scale=spread)
    gate += torch.linspace(-1, 5, D, device="cuda")
    d = {"gate": gate.to(dtype), "x": _randn(g, R, D, dtype=dtype), "dh": _randn(g, R, D, dtype=dtype)}
    if state:
        d.update(state=_randn(g, S, D), dstate=_randn(g, S, D))
    return d


def _run(d, offsets, coupled, shape=None, **more):
    """Forward and gradient; shape: [B, T, D] of equal sequences."""
    off = None
    view = lambda t: t.view(*shape) if shape else t  # noqa: E731
    if shape is None:
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    r = dpg.dpg_recurrence(view(d["gate"]), view(d["x"]), offsets=off, state=d.get("state"), coupled=coupled,
                           carries=True, **more)
    b = dpg.dpg_recurrence_dgrad(view(d["dh"]), view(d["gate"]), view(d["x"]), r.carries, offsets=off,
                                 state=d.get("state"), dstate=d.get("dstate"), coupled=coupled)
    return r, b


def _compare(d, offsets, coupled, r, b):
    h = lambda k: ref.host(d[k]) if k in d else None  # noqa: E731
    want = ref.recurrence(h("gate"), h("x"), offsets, h("state"), coupled, h("dh"), h("dstate"))
    dtype = d["x"].dtype
    for name, got in (("h", r.h), ("dgate", b.dgate), ("dx", b.dx)):
        assert got.dtype == dtype
        _check(name, got, want[name], want["e_" + name], dtype)
    _check("state", r.state, want["state"], want["e_state"], F32)
    if "state" in d:
        _check("dstate", b.dstate, want["dstate"], want["e_dstate"], F32)
    else:
        assert b.dstate is None


SHAPES = [(1, 1, 8), (3, 1, 72), (130, 1, 64), (1, 5, 64), (70, 7, 40), (2, 64, 64), (2, 65, 136), (3, 127, 8),
          (2, 128, 64), (2, 129, 72), (5, 200, 64), (1, 1000, 72), (1, 2500, 8), (2, 1153, 200), (40, 33, 24)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_equal_sequences(shape, coupled, dtype):
    B, T, D = shape
    d = _inputs(B * T, B, D, dtype, seed=B + T + D, state=(B + T) % 2 == 0 or T == 1)
    offsets = [T * i for i in range(B + 1)]
    _compare(d, offsets, coupled, *_run(d, offsets, coupled, shape))


PACKED = {"one": [0, 1], "short": [0, 1, 2, 5, 5, 9, 20], "empty first": [0, 0, 0, 7, 130], "all empty": [0, 0, 0],
          "edges": [0, 63, 64, 65, 128, 129, 256, 300], "long": [0, 700, 701, 701, 1900], "tile": [0, 128, 256],
          "last empty": [0, 40, 90, 90, 90]}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("tail", [0, 3, 200])
@pytest.mark.parametrize("name", list(PACKED))
def test_packed_sequences(name, tail, coupled, dtype):
    offsets, D = PACKED[name], 72
    R = offsets[-1] + tail
    d = _inputs(R, len(offsets) - 1, D, dtype, seed=len(name) + tail)
    for k in ("gate", "x", "dh"):
        d[k][offsets[-1]:] = float("nan")  # rows of nobody
    r, b = _run(d, offsets, coupled)
    for t in (r.h, b.dgate, b.dx):
        assert bool((t[offsets[-1]:] == 0).all())
    for k in ("gate", "x", "dh"):
        d[k][offsets[-1]:] = 0
    want_tail = [t[offsets[-1]:] for t in (r.h, b.dgate, b.dx)]
    assert all(bool((t == 0).all()) for t in want_tail)
    _compare(d, offsets, coupled, r, b)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_packed_equals_equal_sequences_in_bits_of_one_axis(dtype):
    """One sequence of all rows is the same cut either way."""
    d = _inputs(900, 1, 72, dtype, seed=5)
    r, b = _run(d, None, True, (1, 900, 72))
    r2, b2 = _run(d, [0, 900], True)
    assert torch.equal(r.h.view(900, 72), r2.h) and torch.equal(r.state, r2.state)
    assert torch.equal(b.dgate.view(900, 72), b2.dgate) and torch.equal(b.dstate, b2.dstate)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
def test_weights_of_zero_leave_their_terms_out(coupled, dtype):
    inf, nan = float("inf"), float("nan")
    B, T, D = 2, 700, 24
    d = _inputs(B * T, B, D, dtype, seed=3)
    gate, x, h0 = d["gate"].view(B, T, D), d["x"].view(B, T, D), d["state"]
    h0[0, 0:4] = torch.tensor([inf, nan, -inf, 1.0])
    gate[0, 0, 0:3] = -inf          # forgets them
    gate[0, 300, 5] = -inf
    x[0, 290, 5] = nan              # until row 300
    x[0, 299, 6] = inf              # for good
    x[1, 650, 7] = nan
    gate[1, 10:20, 8] = inf         # holds the state
    if coupled:
        x[1, 10:20, 8] = nan        # and passes over the input
    gate[1, 5, 9] = nan             # for good
    gate[1, 128, 10], gate[1, 127, 10] = -inf, -inf
    offsets = [0, T, 2 * T]
    r, b = _run(d, offsets, coupled, (B, T, D))
    want = ref.recurrence(ref.host(d["gate"]), ref.host(d["x"]), offsets, ref.host(h0), coupled)
    clean = lambda a: np.where(np.isfinite(a), a, 0)  # noqa: E731
    _check("h", r.h, want["h"], clean(want["e_h"]), dtype)
    _check("state", r.state, want["state"], clean(want["e_state"]), F32)
    # gradients of what nothing strange reaches
    h = ref.host
    want = ref.recurrence(h(d["gate"]), h(d["x"]), offsets, h(h0), coupled, h(d["dh"]), h(d["dstate"]))
    for name, got in (("dgate", b.dgate), ("dx", b.dx)):
        fine = np.isfinite(want[name]) & np.isfinite(want["e_" + name])
        assert fine.mean() > 0.9
        got = h(got).reshape(want[name].shape)
        limit = want["e_" + name] * 1.01 + ref.half_step(dtype) * (np.abs(want[name]) + want["e_" + name]) + 1e-37
        assert bool((np.abs(got - want[name])[fine] <= limit[fine]).all()), name


@pytest.mark.parametrize("T", [1, 700, 40], ids=["steps", "spans", "short"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "free"])
@pytest.mark.parametrize("state", [True, False], ids=["state", "zeros"])
def test_a_gate_of_nan_is_one_of_its_row_on(state, coupled, dtype, T):
    """At places of a run and of a tile, and next to inputs, states and gradients
    of 0, which hide no NaN: outputs from the row on, gradients up to it."""
    B, D = 3, 64
    d = _inputs(B * T, B, D, dtype, seed=12, state=state)
    gate, x, dh = (d[k].view(B, T, D) for k in ("gate", "x", "dh"))
    for i, t in enumerate([0, 1, 7, 8, 39, 63, 64, 65, 127, 128, 300, 512, T - 1]):
        if t >= T:
            continue
        for k in range(4):
            c = 4 * i + k
            gate[1, t, c] = float("nan")
            if k & 1:
                x[1, :t + 1, c] = 0
                if state:
                    d["state"][1, c] = 0
            if k & 2:
                dh[1, t:, c] = 0
                if state:
                    d["dstate"][1, c] = 0
    offsets = [0, T, 2 * T, 3 * T]
    _compare(d, offsets, coupled, *_run(d, offsets, coupled, (B, T, D)))
    _compare(d, offsets, coupled, *_run(d, offsets, coupled))


def test_an_infinite_state_outlives_products_that_underflow():
    """900 steps of f = e^-2 / (1 + e^-2): the product is 10^-830, the state stays
    infinite."""
    gate = torch.full((1, 900, 8), -2.0, device="cuda")
    x = torch.ones(1, 900, 8, device="cuda")
    h0 = torch.full((1, 8), float("inf"), device="cuda")
    r = dpg.dpg_recurrence(gate, x, state=h0)
    assert bool(torch.isinf(r.h).all()) and bool(torch.isinf(r.state).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("length", [700, 1])
def test_state_in_place(dtype, length):
    d = _inputs(3 * length, 3, 40, dtype, seed=8)
    shape = (3, length, 40)
    want = dpg.dpg_recurrence(d["gate"].view(shape), d["x"].view(shape), state=d["state"])
    own = d["state"].clone()
    version = own._version
    x = d["x"].view(shape).clone()
    got = dpg.dpg_recurrence(d["gate"].view(shape), x, state=own, state_out=own, out=x)
    assert got.state is own or got.state.data_ptr() == own.data_ptr()
    assert torch.equal(own, want.state) and torch.equal(x, want.h) and own._version > version


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_steps_one_by_one_are_the_sequence(dtype):
    """A prefill and then single tokens: within the bound of either."""
    B, T, D = 3, 150, 40
    d = _inputs(B * T, B, D, dtype, seed=9)
    gate, x = d["gate"].view(B, T, D), d["x"].view(B, T, D)
    state = d["state"].clone()
    first = dpg.dpg_recurrence(gate[:, :100].contiguous(), x[:, :100].contiguous(), state=state)
    state = first.state
    rows = [first.h]
    for t in range(100, T):
        r = dpg.dpg_recurrence(gate[:, t:t + 1], x[:, t:t + 1], state=state, state_out=state)
        rows.append(r.h)
    offsets = [T * i for i in range(B + 1)]
    want = ref.recurrence(ref.host(d["gate"]), ref.host(d["x"]), offsets, ref.host(d["state"]), True)
    _check("h", torch.cat(rows, 1).reshape(B * T, D), want["h"], want["e_h"], dtype)
    _check("state", state, want["state"], want["e_state"], F32)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides_and_untouched_columns(dtype):
    B, T, D, W = 2, 300, 72, 96
    d = _inputs(B * T, B, D, dtype, seed=10)
    wide = {k: torch.full((B, T, W), 7.0, dtype=dtype, device="cuda") for k in ("gate", "x", "dh", "out")}
    for k in ("gate", "x", "dh"):
        wide[k][:, :, 8:8 + D] = d[k].view(B, T, D)
    cut = lambda k: wide[k][:, :, 8:8 + D]  # noqa: E731
    want, back = _run(d, None, True, (B, T, D))
    r = dpg.dpg_recurrence(cut("gate"), cut("x"), state=d["state"], carries=True, out=cut("out"))
    assert torch.equal(cut("out"), want.h)
    assert bool((wide["out"][:, :, :8] == 7).all()) and bool((wide["out"][:, :, 8 + D:] == 7).all())
    b = dpg.dpg_recurrence_dgrad(cut("dh"), cut("gate"), cut("x"), r.carries, state=d["state"], dstate=d["dstate"])
    assert torch.equal(b.dgate, back.dgate) and torch.equal(b.dx, back.dx) and torch.equal(b.dstate, back.dstate)


def test_no_rows_and_no_channels():
    for shape in ((0, 5, 8), (4, 0, 8), (4, 5, 0)):
        x = torch.zeros(shape, dtype=BF16, device="cuda")
        state = torch.randn(shape[0], shape[2], device="cuda")
        r = dpg.dpg_recurrence(x, x, state=state, carries=True)
        assert r.h.shape == x.shape and r.state.shape == state.shape
        if shape[1] == 0:
            assert torch.equal(r.state, state)
            b = dpg.dpg_recurrence_dgrad(x, x, x, r.carries, state=state, dstate=state)
            assert torch.equal(b.dstate, state)


def test_packed_rows_of_no_sequence():
    x = torch.full((300, 16), float("nan"), dtype=BF16, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = dpg.dpg_recurrence(x, x, offsets=off, carries=True)
    assert bool((r.h == 0).all()) and r.state.shape == (0, 16)
    b = dpg.dpg_recurrence_dgrad(x, x, x, r.carries, offsets=off)
    assert bool((b.dgate == 0).all()) and bool((b.dx == 0).all())


def test_offsets_out_of_range_stay_inside():
    """Values are unspecified; what lies around the outputs stays."""
    for offsets in ([0, 5, 5000, 7, 90], [0, -3, 40, 1 << 30, 60], [50, 10, 80, 20, 400]):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        d = _inputs(300, 4, 24, F32, seed=1)
        whole = torch.full((320, 24), 7.0, device="cuda")
        last = torch.full((8, 24), 7.0, device="cuda")
        dpg.dpg_recurrence(d["gate"], d["x"], offsets=off, state=d["state"], out=whole[10:310], state_out=last[2:6])
        assert bool((whole[:10] == 7).all()) and bool((whole[310:] == 7).all())
        assert bool((last[:2] == 7).all()) and bool((last[6:] == 7).all())


def test_two_streams_at_once():
    d = [_inputs(2 * 3000, 2, 72, BF16, seed=20 + i) for i in range(2)]
    want = [_run(x, None, True, (2, 3000, 72)) for x in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_run(d[i], None, True, (2, 3000, 72)))
    torch.cuda.synchronize()
    for i in range(2):
        for r, b in got[i]:
            assert torch.equal(r.h, want[i][0].h) and torch.equal(r.state, want[i][0].state)
            assert all(torch.equal(x, y) for x, y in zip(b, want[i][1]))


def test_captured_with_the_state_in_place():
    """A graph of a prefill in spans and of generation steps, replayed: each replay
    starts from the state the one before left."""
    d = _inputs(2000, 1, 40, BF16, seed=30)
    gate, x = d["gate"].view(1, 2000, 40), d["x"].view(1, 2000, 40)
    state = d["state"].clone()

    def both(s):
        a = dpg.dpg_recurrence(gate, x, state=s, state_out=s)
        return a.h, dpg.dpg_recurrence(gate[:, :1], x[:, :1], state=s, state_out=s).h
    both(state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, step = both(state)
    state.copy_(d["state"])
    own = d["state"].clone()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        a, b = both(own)
        assert torch.equal(h, a) and torch.equal(step, b) and torch.equal(state, own)


@pytest.mark.parametrize("packed", [False, True])
def test_reruns_give_the_same_bits(packed):
    d = _inputs(4000, 4, 72, BF16, seed=11)
    offsets, shape = [0, 1000, 1000, 3999, 4000], None if packed else (4, 1000, 72)
    first = _run(d, offsets, True, shape)
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(0xff)
    for _ in range(5):
        again = _run(d, offsets, True, shape)
        for a, b in zip((first[0].h, first[0].state, *first[1]), (again[0].h, again[0].state, *again[1])):
            assert torch.equal(a, b)


def test_many_channels_and_many_sequences():
    """Cuts with one span, many axes, and channels that fill no block."""
    for B, T, D in ((600, 20, 1000), (9, 260, 4104)):
        d = _inputs(B * T, B, D, BF16, seed=B, spread=1.0)
        r, b = _run(d, None, True, (B, T, D))
        pick = [0, B // 2, B - 1]
        for s in pick:
            rows = slice(s * T, s * T + T)
            h = lambda k: ref.host(d[k][rows])  # noqa: E731
            want = ref.recurrence(h("gate"), h("x"), [0, T], ref.host(d["state"][s:s + 1]), True, h("dh"),
                                  ref.host(d["dstate"][s:s + 1]))
            _check("h", r.h[s], want["h"], want["e_h"], BF16)
            _check("dgate", b.dgate[s], want["dgate"], want["e_dgate"], BF16)
            _check("dx", b.dx[s], want["dx"], want["e_dx"], BF16)
            _check("dstate", b.dstate[s:s + 1], want["dstate"], want["e_dstate"], F32)


def test_gradient_of_x_is_the_difference():
    """h is linear in x and the state: the difference over a step along any
    direction is the gradient's product with it, but for the outputs' FP32 errors."""
    B, T, D = 2, 600, 16
    d = _inputs(B * T, B, D, F32, seed=12)
    shape = (B, T, D)
    r, b = _run(d, None, True, shape)
    g = torch.Generator().manual_seed(1)
    direction = _randn(g, *shape)
    offsets = [0, T, 2 * T]
    value = {}
    bound = 0.0
    for sign in (1, -1):
        x = d["x"].view(shape) + sign * direction
        s = dpg.dpg_recurrence(d["gate"].view(shape), x, state=d["state"])
        value[sign] = float((s.h.double() * d["dh"].view(shape).double()).sum() + (s.state.double() * d["dstate"].double()).sum())
        want = ref.recurrence(ref.host(d["gate"]), ref.host(x).reshape(-1, D), offsets, ref.host(d["state"]), True)
        bound += float(((want["e_h"] + ref.U * np.abs(want["h"])) * np.abs(ref.host(d["dh"]))).sum())
        bound += float((want["e_state"] * np.abs(ref.host(d["dstate"]))).sum())
        # x + direction is rounded
        bound += float((ref.U * (x.double().abs() * b.dx.double().abs())).sum()) * 2
    want = ref.recurrence(ref.host(d["gate"]), ref.host(d["x"]), offsets, ref.host(d["state"]), True,
                          ref.host(d["dh"]), ref.host(d["dstate"]))
    bound += float(((want["e_dx"] + ref.U * np.abs(want["dx"])) * np.abs(ref.host(direction).reshape(-1, D))).sum()) * 2
    slope = float((b.dx.double() * direction.double()).sum())
    assert abs((value[1] - value[-1]) / 2 - slope) <= bound / 2
    assert abs(slope) > 20 * bound  # the test can tell


def test_refusals():
    x = torch.zeros(2, 5, 16, dtype=BF16, device="cuda")
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match=r"\[B, T, D\]"):
        dpg.dpg_recurrence(x.view(10, 16), x.view(10, 16))
    with pytest.raises(ValueError, match="with offsets"):
        dpg.dpg_recurrence(x, x, offsets=off)
    with pytest.raises(TypeError):
        dpg.dpg_recurrence(x.float(), x)
    with pytest.raises(ValueError):
        dpg.dpg_recurrence(x[:, :4], x)
    with pytest.raises(ValueError, match="follow each other"):
        dpg.dpg_recurrence(x[:, :4], x[:, :4])
    with pytest.raises(TypeError):
        dpg.dpg_recurrence(x, x, state=torch.zeros(2, 16, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        dpg.dpg_recurrence(x, x, state=torch.zeros(3, 16, device="cuda"))
    with pytest.raises(TypeError):
        dpg.dpg_recurrence(x, x, out=torch.zeros(2, 5, 16, device="cuda"))
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_recurrence(x[:, :, :12], x[:, :, :12])
    assert e.value.status == 3
    r = dpg.dpg_recurrence(x, x, carries=True)
    with pytest.raises(ValueError, match="carries"):
        dpg.dpg_recurrence_dgrad(x, x, x, r.carries[:-4])
    with pytest.raises(TypeError):
        dpg.dpg_recurrence_dgrad(x, x, x, None)
    y = torch.zeros(1, 2000, 16, dtype=BF16, device="cuda")
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_recurrence(y, y, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
