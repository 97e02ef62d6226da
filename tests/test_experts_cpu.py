"""What the expert-layer entry points refuse, without a GPU: the C ABI through
ctypes (every call here is refused, or empty, before any launch) and the
compiled binding on host tensors."""
import ctypes

import pytest
import torch

import deterministic_bf16_projection_amd as dpg

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(5)
P = ctypes.c_void_p(0x10000)     # never read: the call ends before a launch
ODD = ctypes.c_void_p(0x10002)
I, Z = ctypes.c_int64, ctypes.c_size_t


def _grouped(name, a=P, lda=64, b=P, ldb=64, stride=4096, c=P, ldc=64, dtype=0, offsets=P, E=4, R=10, N=64, K=64):
    if name == "wgrad":
        args = (a, I(lda), b, I(ldb), c, I(ldc), I(stride), dtype, offsets, I(E), I(R), I(N), I(K), P, Z(1 << 40), None)
    else:
        args = (a, I(lda), b, I(ldb), I(stride), c, I(ldc), dtype, offsets, I(E), I(R), I(N), I(K), P, Z(1 << 40),
                None)
    return getattr(dpg.lib(), "dpg_grouped_" + name)(*args)


@pytest.mark.parametrize("name", ["forward", "dgrad", "wgrad"])
def test_grouped_refusals(name):
    assert _grouped(name, dtype=2) == INVALID
    for bad in ({"E": -1}, {"R": -1}, {"N": -8}, {"K": -8}, {"stride": -64}, {"a": None}, {"b": None}, {"c": None},
                {"offsets": None}, {"lda": 56}, {"ldb": 56}, {"ldc": 56}):
        assert _grouped(name, **bad) == INVALID, bad
    for bad in ({"a": ODD}, {"b": ODD}, {"c": ODD}, {"lda": 65}, {"stride": 4100}, {"N": 60}, {"K": 60},
                {"offsets": ctypes.c_void_p(0x10001)}):
        assert _grouped(name, **bad) == ALIGNMENT, bad
    for bad in ({"lda": 1 << 22}, {"R": 1 << 31}, {"E": 1 << 24}):
        assert _grouped(name, **bad) == UNSUPPORTED, bad
    empty = {"forward": {"R": 0}, "dgrad": {"K": 0}, "wgrad": {"E": 0}}[name]
    assert _grouped(name, a=None, b=None, c=None, offsets=None, **empty) in (OK, INVALID)
    if name == "wgrad":
        assert _grouped(name, stride=2048) == INVALID  # outputs that overlap


def _route(logits=P, ldl=16, T=100, E=16, k=4, experts=P, weights=P, offsets=P, rows=P, positions=P, ws=P, size=None):
    need = dpg.lib().dpg_route_workspace_size
    need.restype = Z
    size = need(I(T), I(E), I(k)) if size is None else size
    return dpg.lib().dpg_route(logits, I(ldl), I(T), I(E), I(k), 1, experts, weights, offsets, rows, positions, ws,
                               Z(size), None)


def test_route_refusals():
    for bad in ({"k": 0}, {"k": 17}, {"E": 0}, {"T": -1}, {"ldl": 15}, {"logits": None}, {"experts": None},
                {"weights": None}, {"offsets": None}, {"rows": None}, {"positions": None}):
        assert _route(**bad) == INVALID, bad
    for bad in ({"E": 513, "ldl": 513}, {"E": 64, "k": 33, "ldl": 64}, {"T": 1 << 30}):
        assert _route(**bad) == UNSUPPORTED, bad
    for bad in ("logits", "experts", "weights", "offsets", "rows", "positions"):
        assert _route(**{bad: ODD}) == ALIGNMENT, bad
    assert _route(ws=None) == WORKSPACE and _route(size=16) == WORKSPACE


def test_rows_refusals():
    lib = dpg.lib()

    def dispatch(x=P, ldx=64, pos=P, off=P, xs=P, ldxs=64, dtype=0, T=5, R=10, H=64, E=4, k=2):
        return lib.dpg_dispatch(x, I(ldx), pos, off, xs, I(ldxs), dtype, I(T), I(R), I(H), I(E), I(k), None)
    assert dispatch(T=0) == OK and dispatch(H=0) == OK
    for bad in ({"x": None}, {"pos": None}, {"off": None}, {"xs": None}, {"dtype": 2}, {"k": 0}, {"E": -1}, {"ldx": 56}):
        assert dispatch(**bad) == INVALID, bad
    for bad in ({"x": ODD}, {"pos": ODD}, {"off": ODD}, {"H": 60}, {"ldxs": 65}):
        assert dispatch(**bad) == ALIGNMENT, bad
    assert dispatch(T=1 << 30, R=1 << 30, k=4) == UNSUPPORTED and dispatch(R=1 << 31) == UNSUPPORTED
    assert lib.dpg_combine(P, I(64), 2, P, P, P, P, I(64), 0, I(5), I(10), I(64), I(4), I(2), None) == INVALID
    assert lib.dpg_combine(P, I(64), 0, P, P, ODD, P, I(64), 0, I(5), I(10), I(64), I(4), I(2), None) == ALIGNMENT
    assert lib.dpg_combine_dgrad(P, I(64), P, I(64), P, P, None, P, I(64), P, 0, I(5), I(10), I(64), I(4), I(2),
                                 None) == INVALID


class _Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "ms", "vs", "w")] + [("n", I)]


class _Options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "b1", "b2", "eps", "wd")] + [
        ("step", I), ("gs", ctypes.c_void_p), ("gd", ctypes.c_int), ("sd", ctypes.c_int), ("seed", ctypes.c_uint32)]


def test_adamw_refusals():
    a = 0x10000

    def call(count=1, tensor=None, **change):
        t = _Tensor(a, a, a, a, a, a, a, 100)
        for k, v in (tensor or {}).items():
            setattr(t, k, v)
        o = _Options(1e-3, 0.9, 0.99, 1e-8, 0.1, 1, None, 1, 2, 0)
        for k, v in change.items():
            setattr(o, k, v)
        return dpg.lib().dpg_adamw(ctypes.byref(t), I(count), ctypes.byref(o), None)
    assert call(count=0) == OK and call(tensor={"n": 0, "p": None}) == OK
    assert call(count=-1) == INVALID
    nan = float("nan")
    for bad in ({"lr": nan}, {"lr": -1.0}, {"b1": 1.0}, {"b1": nan}, {"b2": -0.5}, {"eps": float("inf")}, {"wd": nan},
                {"step": 0}, {"gd": 2}, {"sd": 0}):
        assert call(**bad) == INVALID, bad
    for field in ("p", "g", "m", "v", "ms", "vs"):
        assert call(tensor={field: None}) == INVALID, field
    assert call(tensor={"n": -1}) == INVALID
    for field, at in (("p", a + 2), ("g", a + 2), ("ms", a + 2), ("vs", a + 1), ("w", a + 1)):
        assert call(tensor={field: at}) == ALIGNMENT, field
    assert call(gs=a + 2) == ALIGNMENT
    assert call(sd=1, tensor={"m": a + 2}) == ALIGNMENT
    assert call(tensor={"n": 1 << 36}) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_other_objects():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 8, 8, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    lg = torch.zeros(4, 8)
    pos = torch.zeros(4, 1, dtype=torch.int32)
    calls = [lambda a: dpg.dpg_grouped_forward(a, w, off), lambda a: dpg.dpg_grouped_dgrad(a, w, off),
             lambda a: dpg.dpg_grouped_wgrad(a, x, off), lambda a: dpg.dpg_dispatch(a, pos, off),
             lambda a: dpg.dpg_combine(a, pos, off), lambda a: dpg.dpg_combine_dgrad(a, x, pos, off, lg)]
    for call in calls:
        with pytest.raises(ValueError, match="device tensor"):
            call(x)
        for other in (x.double(), None, 3):
            with pytest.raises(TypeError):
                call(other)
    for call in (lambda a: dpg.dpg_route(a, 2), lambda a: dpg.dpg_route_dgrad(a, pos, lg, lg)):
        with pytest.raises(ValueError, match="device tensor"):
            call(lg)
        with pytest.raises(TypeError):
            call(lg.double())
    with pytest.raises(ValueError, match="device tensors"):
        dpg.dpg_adamw([lg], [lg], [lg], [lg], lr=1e-3)
    with pytest.raises(TypeError):
        dpg.dpg_adamw([lg], 5, [lg], [lg], lr=1e-3)
