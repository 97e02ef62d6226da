"""Layer norm, dropout and the recurrence in matrices of more than 2^31 elements and
2^32 bytes: rows at both ends and in between against 64-bit references.

Tolerances: the bounds of block_reference plus the rounding to the output's type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import block_reference as ref  # noqa: E402
from test_gpu_block_sizes import _kept, _rand  # noqa: E402
from test_gpu_layer_norm import BF16, EPS, F32, _check  # noqa: E402
from test_gpu_recurrence import _compare  # noqa: E402

T, H = 263001, 8192  # 2.15e9 elements, 4.3e9 bytes in BF16
EDGE = [0, 1, 131071, 131072, 262143, 262144, 262145, T - 2, T - 1]


@pytest.fixture(autouse=True)
def _additions_of_this_cut(monkeypatch):
    """64 additions in a lane, 6 over the lanes, up to 16 over the waves, a few more."""
    monkeypatch.setattr(ref, "ROW_SUM", 64 + 6 + 16 + 10)


def test_norm_and_its_gradient():
    assert T * H > 1 << 31
    x, dy = _rand(1, T, H, dtype=BF16, scale=2.0), _rand(2, T, H, dtype=BF16)
    w, b = _rand(3, H, scale=0.3, mean=1.0), _rand(4, H)
    n = dpg.dpg_layer_norm(x, w, b, eps=EPS)
    hx, hw = ref.host(x[EDGE]), ref.host(w)
    wy, wm, wr, ey, em, er = ref.layer_norm(hx, hw, ref.host(b), EPS)
    _check("y", n.y[EDGE], wy, ey, BF16)
    _check("mean", n.mean[EDGE], wm, em)
    _check("rstd", n.rstd[EDGE], wr, er)
    d = dpg.dpg_layer_norm_dgrad(dy, x, n.mean, n.rstd, w, weight_grads=False)
    dx, _, _, ex, _, _ = ref.layer_norm_dgrad(ref.host(dy[EDGE]), hx, ref.host(n.mean[EDGE]), ref.host(n.rstd[EDGE]), hw)
    _check("dx", d.dx[EDGE], dx, ex, BF16)


@pytest.mark.parametrize("pad", [0, 8])
def test_dropout(pad):
    x = _rand(1, T, H + pad, dtype=BF16)[:, :H]
    p, seed = 0.25, 99
    y = dpg.dpg_dropout(x, p, seed, out=x)  # over the input
    assert y.data_ptr() == x.data_ptr()
    again = _rand(1, T, H + pad, dtype=BF16)[:, :H]
    part = np.where(_kept(EDGE, H, p, seed, 0), ref.host(again[EDGE]) * ref.keep_scale(p), 0.0)
    _check("y", y[EDGE], part, 2 * ref.U * np.abs(part), BF16)


@pytest.mark.parametrize("packed", [False, True], ids=["equal", "packed"])
def test_recurrence_and_its_gradient(packed):
    B, N, D = 8, 32800, 8200
    R = B * N
    assert R * D > 1 << 31
    d = {"gate": _rand(1, R, D, dtype=BF16, mean=2.0), "x": _rand(2, R, D, dtype=BF16), "dh": _rand(3, R, D, dtype=BF16),
         "state": _rand(4, B, D), "dstate": _rand(5, B, D)}
    view = (lambda t: t) if packed else (lambda t: t.view(B, N, D))
    offsets = [N * i for i in range(B + 1)]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda") if packed else None
    r = dpg.dpg_recurrence(view(d["gate"]), view(d["x"]), offsets=off, state=d["state"], carries=True)
    b = dpg.dpg_recurrence_dgrad(view(d["dh"]), view(d["gate"]), view(d["x"]), r.carries, offsets=off, state=d["state"],
                                 dstate=d["dstate"])
    col = torch.tensor([0, 1, 127, 128, 4100, D - 2, D - 1], device="cuda")
    for s in (0, B - 1):
        rows = slice(s * N, s * N + N)
        cut = lambda t: t.view(R, D)[rows][:, col]  # noqa: E731
        one = lambda t: t[s:s + 1][:, col]  # noqa: E731
        part = {k: one(v) if "state" in k else cut(v) for k, v in d.items()}
        _compare(part, [0, N], True, r._replace(h=cut(r.h), state=one(r.state)),
                 b._replace(dgate=cut(b.dgate), dx=cut(b.dx), dstate=one(b.dstate)))
    assert r.state.dtype == F32
