"""Row movement on the GPU beyond what the Python entry points pass: through the C
ABI, more sorted rows than slots and positions that leave rows out."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

dpg = pytest.importorskip("deterministic_bf16_projection_amd")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

I = ctypes.c_int64
CODE = {torch.bfloat16: 0, torch.float32: 1}


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,H,more,masked,dropped", [
    (1, 1, 1, 8, 1, 0.0, 0), (3, 2, 4, 264, 0, 0.0, 3), (70, 6, 9, 136, 37, 0.4, 5), (5, 2, 4, 24, 1000, 1.0, 0),
    (300, 4, 16, 1024, 0, 0.6, 100), (2, 1, 3, 4096, 20000, 0.0, 0)])
def test_every_row_past_the_routed_ones_is_zero(T, k, E, H, more, masked, dropped, dtype):
    """R = T top_k + `more` rows; `dropped` of the slots without an expert are given
    the position -1.  What lies around the matrices stays as it is."""
    g = torch.Generator().manual_seed(T + H)
    lg = torch.randn(T, E, generator=g)
    lg[torch.rand(T, E, generator=g) < masked] = -float("inf")
    r = dpg.dpg_route(lg.cuda(), k)
    used, R = int(r.offsets[-1]), T * k + more
    pos = r.positions.clone().reshape(-1)
    unused = (pos >= used).nonzero().reshape(-1)[:dropped]
    pos[unused] = -1
    x, dy = (torch.randn(T, H, generator=g).to(dtype).cuda() for _ in range(2))
    ys = torch.randn(R, H, generator=g).to(dtype).cuda()
    ys[used:] = float("nan")  # never read
    wide = [torch.full((R + 2, H), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    xs, dys = (t[1:R + 1] for t in wide)
    dw = torch.full((T, k), 7.0, device="cuda")
    lib, code = dpg.lib(), CODE[dtype]
    assert lib.dpg_dispatch(_p(x), I(H), _p(pos), _p(r.offsets), _p(xs), I(H), code, I(T), I(R), I(H), I(E), I(k),
                            _stream()) == 0
    assert lib.dpg_combine_dgrad(_p(dy), I(H), _p(ys), I(H), _p(pos), _p(r.offsets), _p(r.weights), _p(dys), I(H),
                                 _p(dw), code, I(T), I(R), I(H), I(E), I(k), _stream()) == 0
    torch.cuda.synchronize()
    token = (r.rows[:used] // k).long()
    assert torch.equal(xs[:used], x[token])
    weight = r.weights.reshape(-1)[r.rows[:used].long()][:, None]
    assert torch.equal(dys[:used], (weight * dy[token].float()).to(dtype))  # one product, rounded once
    for t in (xs, dys):
        assert bool((t[used:] == 0).all())
    for t in wide:
        assert bool((t[[0, R + 1]] == 7.0).all())
    live = (r.positions < used)
    assert bool((dw[~live] == 0).all()) and bool(torch.isfinite(dw).all())


def test_no_tokens_write_nothing():
    r = dpg.dpg_route(torch.zeros(0, 4, device="cuda"), 2)
    xs = torch.full((5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    nothing = ctypes.c_void_p(None)
    assert dpg.lib().dpg_dispatch(nothing, I(64), nothing, _p(r.offsets), _p(xs), I(64), 0, I(0), I(5), I(64), I(4),
                                  I(2), _stream()) == 0
    torch.cuda.synchronize()
    assert bool((xs == 7.0).all())
