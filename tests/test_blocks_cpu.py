"""What the entry points between a block's projections refuse, without a GPU: the
C ABI through ctypes (every call here is refused, or empty, before any launch)
and the compiled binding on host tensors.  And the references that the GPU tests
use, against differences."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as ref
import deterministic_bf16_projection_amd as dpg

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(5)
P = ctypes.c_void_p(0x10000)     # never read: the call ends before a launch
ODD = ctypes.c_void_p(0x10002)
I, Z, D = ctypes.c_int64, ctypes.c_size_t, ctypes.c_double
BIG = 1 << 40


class _Drop(ctypes.Structure):
    _fields_ = [("p", D), ("seed", ctypes.c_uint64), ("step", ctypes.c_void_p)]


def _drop(p=0.1, step=None):
    return ctypes.byref(_Drop(p, 1, step))


def test_dropout_refusals():
    def call(x=P, ldx=64, xt=0, r=P, ldr=64, y=P, ldy=64, yt=0, T=5, H=64, drop=None, none=False):
        return dpg.lib().dpg_dropout(x, I(ldx), xt, r, I(ldr), y, I(ldy), yt, I(T), I(H),
                                     None if none else (drop or _drop()), None)
    assert call(T=0) == OK and call(H=0) == OK
    for bad in ({"x": None}, {"y": None}, {"xt": 2}, {"yt": 2}, {"T": -1}, {"H": -8}, {"ldx": 56}, {"ldr": 56},
                {"ldy": 56}, {"none": True}, {"drop": _drop(1.5)}, {"drop": _drop(-0.1)},
                {"drop": _drop(float("nan"))}):
        assert call(**bad) == INVALID, bad
    for bad in ({"x": ODD}, {"r": ODD}, {"y": ODD}, {"ldx": 65}, {"H": 60}, {"drop": _drop(step=0x10004)}):
        assert call(**bad) == ALIGNMENT, bad
    assert call(T=1 << 31) == UNSUPPORTED and call(H=1 << 31, ldx=1 << 31, ldr=1 << 31, ldy=1 << 31) == UNSUPPORTED


def test_layer_norm_refusals():
    def call(x=P, ldx=64, xt=0, w=P, b=P, y=P, ldy=64, yt=0, mean=P, rstd=P, T=5, H=64, eps=1e-5):
        return dpg.lib().dpg_layer_norm(x, I(ldx), xt, w, b, y, I(ldy), yt, mean, rstd, I(T), I(H), D(eps), None)
    assert call(T=0) == OK and call(H=0) == OK
    for bad in ({"x": None}, {"y": None}, {"mean": None}, {"rstd": None}, {"xt": 2}, {"yt": -1}, {"T": -1},
                {"ldx": 56}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert call(**bad) == INVALID, bad
    for bad in ({"x": ODD}, {"y": ODD}, {"w": ODD}, {"b": ODD}, {"H": 60}, {"ldy": 65},
                {"mean": ctypes.c_void_p(0x10001)}, {"rstd": ctypes.c_void_p(0x10001)}):
        assert call(**bad) == ALIGNMENT, bad
    assert call(H=16392, ldx=16392, ldy=16392) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED

    def add(r=P, s=P, st=1, lds=64, drop=None, x=P):
        return dpg.lib().dpg_add_layer_norm(x, I(64), 0, r, I(64), s, I(lds), st, P, P, P, I(64), 0, P, P, I(5), I(64),
                                            D(1e-5), drop, None)
    for bad in ({"r": None}, {"s": None}, {"x": None}, {"st": 2}, {"lds": 32}, {"drop": _drop(2.0)}):
        assert add(**bad) == INVALID, bad
    for bad in ({"r": ODD}, {"s": ODD}, {"drop": _drop(step=0x10001)}):
        assert add(**bad) == ALIGNMENT, bad


def test_layer_norm_gradient_refusals():
    size = dpg.lib().dpg_layer_norm_workspace_size
    size.restype = Z
    assert size(I(0), I(64)) == 0 and size(I(-1), I(64)) == Z(-1).value and size(I(5), I(16392)) == Z(-1).value
    need = size(I(5), I(64))
    assert need > 0 and need % 16 == 0

    def call(dy=P, x=P, mean=P, rstd=P, w=P, dx=P, dw=P, db=P, T=5, H=64, ws=P, bytes_=None, dyt=0, xt=0, ld=64):
        return dpg.lib().dpg_layer_norm_dgrad(dy, I(ld), dyt, x, I(ld), xt, mean, rstd, w, dx, I(ld), dw, db, I(T),
                                              I(H), ws, Z(need if bytes_ is None else bytes_), None)
    assert call(H=0) == OK and call(T=0, dw=None, db=None) == OK
    for bad in ({"dy": None}, {"x": None}, {"mean": None}, {"rstd": None}, {"dx": None}, {"dyt": 2}, {"xt": 2},
                {"ld": 56}, {"T": -1}):
        assert call(**bad) == INVALID, bad
    for bad in ({"dy": ODD}, {"x": ODD}, {"dx": ODD}, {"w": ODD}, {"H": 60}, {"dw": ODD}):
        assert call(**bad) == ALIGNMENT, bad
    for bad in ({"ws": None}, {"bytes_": need - 1}, {"ws": ctypes.c_void_p(0x10004)}):
        assert call(**bad) == WORKSPACE, bad

    def add(dsum=P, lddsum=64, dres=P, dxt=0, drop=None, ws=P, sum_=P):
        return dpg.lib().dpg_add_layer_norm_dgrad(P, I(64), 0, sum_, I(64), 1, P, P, P, dsum, I(lddsum), P, I(64), dxt,
                                                  dres, I(64), P, P, I(5), I(64), drop, ws, Z(need), None)
    for bad in ({"dres": None}, {"sum_": None}, {"dxt": 2}, {"lddsum": 8}, {"drop": _drop(-1.0)}):
        assert add(**bad) == INVALID, bad
    assert add(dsum=ODD) == ALIGNMENT and add(ws=None) == WORKSPACE


@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_refusals(packed):
    lib = dpg.lib()
    for name in ("workspace", "carries"):
        f = getattr(lib, "dpg_recurrence_%s_size" % name)
        f.restype = Z
        assert f(I(2), I(-1), I(8), 0, int(packed)) == Z(-1).value
        assert f(I(2), I(0), I(8), 0, int(packed)) == 0
        assert f(I(2), I(10), I(8), 2, int(packed)) == Z(-1).value
    assert lib.dpg_recurrence_carries_size(I(2), I(2000), I(64), 0, int(packed)) >= 2000 // 128 * 64 * 4

    def call(gate=P, x=P, h=P, kind=0, state=P, last=P, carries=P, S=2, R=2000, D_=64, ld=64, ws=P, size=BIG,
             off=None):
        off = (off or P) if packed else None
        return lib.dpg_recurrence(gate, I(ld), x, I(ld), h, I(ld), kind, state, last, carries, off, I(S), I(R), I(D_),
                                  1, ws, Z(size), None)

    def grad(dh=P, gate=P, x=P, carries=P, state=P, dstate=P, dgate=P, dx=P, first=ctypes.c_void_p(0x20000), kind=0,
             S=2, R=2000, D_=64, ld=64, ws=P, size=BIG):
        return lib.dpg_recurrence_dgrad(dh, I(ld), gate, I(ld), x, I(ld), carries, state, dstate, dgate, I(ld), dx,
                                        I(ld), first, kind, P if packed else None, I(S), I(R), I(D_), 1, ws, Z(size),
                                        None)
    assert call(D_=0) == OK and grad(D_=0) == OK
    assert call(S=0, R=0, last=None) == OK and grad(S=0, R=0, first=None) == OK
    for bad in ({"gate": None}, {"x": None}, {"kind": 2}, {"S": -1}, {"R": -1}, {"ld": 56}):
        assert call(**bad) == INVALID and grad(**bad) == INVALID, bad
    assert call(h=None) == INVALID
    for bad in ({"dh": None}, {"dgate": None}, {"dx": None}, {"carries": None}, {"first": P}):
        assert grad(**bad) == INVALID, bad
    for bad in ({"gate": ODD}, {"x": ODD}, {"state": ODD}, {"carries": ODD}, {"D_": 60}, {"ld": 66}):
        assert call(**bad) == ALIGNMENT and grad(**bad) == ALIGNMENT, bad
    assert call(last=ODD) == ALIGNMENT and grad(first=ODD) == ALIGNMENT and grad(dstate=ODD) == ALIGNMENT
    for bad in ({"R": (1 << 30) + 2}, {"S": (1 << 24) + 2, "R": (1 << 24) + 2}, {"D_": (1 << 24) + 8, "ld": 1 << 25}):
        assert call(**bad) == UNSUPPORTED and grad(**bad) == UNSUPPORTED, bad
    for bad in ({"ws": None}, {"size": 16}, {"ws": ODD}):
        assert call(**bad) == WORKSPACE and grad(**bad) == WORKSPACE, bad
    if packed:
        assert call(off=ctypes.c_void_p(0x10001)) == ALIGNMENT
    else:
        assert call(S=3) == INVALID and call(S=0) == INVALID  # not a whole number of rows each


def test_binding_refuses_host_tensors_and_other_objects():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    s = x.view(1, 4, 8)
    one = torch.zeros(4)
    calls = [dpg.dpg_layer_norm, lambda a: dpg.dpg_dropout(a, 0.1, 1), lambda a: dpg.dpg_add_layer_norm(a, x),
             lambda a: dpg.dpg_layer_norm_dgrad(a, x, one, one), lambda a: dpg.dpg_add_layer_norm_dgrad(a, x, one, one),
             lambda a: dpg.dpg_recurrence(s, a), lambda a: dpg.dpg_recurrence_dgrad(s, s, a, one)]
    for call in calls:
        with pytest.raises(ValueError, match="device tensor"):
            call(x)
        for other in (x.double(), None, 3, [x]):
            with pytest.raises(TypeError):
                call(other)


def _difference(value, at, t):
    """Central difference of value() by every element of `at`, changed in place."""
    d = np.zeros_like(at)
    for i in np.ndindex(at.shape):
        old = at[i]
        at[i] = old + t
        up = value()
        at[i] = old - t
        d[i] = (up - value()) / (2 * t)
        at[i] = old
    return d


@pytest.mark.parametrize("coupled", [True, False])
def test_recurrence_reference_against_differences(coupled):
    g = np.random.default_rng(1)
    offsets, D_ = [0, 3, 3, 8], 2
    gate, x, dh = (g.standard_normal((9, D_)) for _ in range(3))
    h0, dlast = g.standard_normal((3, D_)), g.standard_normal((3, D_))
    dh[8] = 0

    def value():
        r = ref.recurrence(gate, x, offsets, h0, coupled)
        return float((r["h"] * dh).sum() + (r["state"] * dlast).sum())
    r = ref.recurrence(gate, x, offsets, h0, coupled, dh, dlast)
    for name, at in (("dgate", gate), ("dx", x), ("dstate", h0)):
        # values of order 10 at 2^-53, over 2^-16: 1e-10; truncation 2^-32
        assert np.abs(_difference(value, at, 2.0 ** -17) - r[name]).max() < 1e-8


def test_layer_norm_reference_against_differences():
    g = np.random.default_rng(2)
    x, dy, w, b = g.standard_normal((3, 8)), g.standard_normal((3, 8)), g.standard_normal(8), g.standard_normal(8)

    def value():
        return float((ref.layer_norm(x, w, b, 1e-5)[0] * dy).sum())
    _, mean, rstd, *_ = ref.layer_norm(x, w, b, 1e-5)
    dx, dw, db, *_ = ref.layer_norm_dgrad(dy, x, mean, rstd, w)
    for at, grad in ((x, dx), (w, dw), (b, db)):
        assert np.abs(_difference(value, at, 2.0 ** -17) - grad).max() < 1e-8


def test_autograd_refuses_a_residual_of_another_shape():
    """As matrices both have 8 rows."""
    from deterministic_bf16_projection_amd import autograd
    x, residual = torch.zeros(2, 4, 8), torch.zeros(8, 8)
    with pytest.raises(ValueError, match=r"residual has shape \(8, 8\), x \(2, 4, 8\)"):
        autograd.add_layer_norm(x, residual)
    with pytest.raises(ValueError, match=r"residual has shape \(8, 8\), x \(2, 4, 8\)"):
        autograd.dropout(x, 0.1, 1, residual=residual)
