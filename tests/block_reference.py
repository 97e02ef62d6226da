"""64-bit references of layer norm, dropout and the gated recurrence, with bounds
on what FP32 arithmetic may add.  u = 2^-24 is FP32's unit roundoff; a rounding
to BF16 is off by at most 2^-8 of the value (half a step)."""
import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def host(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------- dropout --
def philox(group, seed, step):
    """Philox4x32 with ten rounds of the counter (group, step) under the key seed:
    uint64 arrays of 32-bit words, [4, len(group)]."""
    m = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    group = np.asarray(group, dtype=np.uint64)
    step = np.uint64(step & 0xFFFFFFFFFFFFFFFF)
    c = [group & m, group >> s32, np.full_like(group, step & m), np.full_like(group, step >> s32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k0), b & m, (a >> s32) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c)


def kept(T, H, p, seed, step=0):
    """Truth values [T, H]: which elements stay."""
    w = philox(np.arange(T * H // 8), seed, step)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 1).reshape(8, -1).T.reshape(T, H)
    return bits >= np.uint64(int(np.floor(p * 65536 + 0.5)))


def keep_scale(p):
    bar = int(np.floor(p * 65536 + 0.5))
    return 65536.0 / (65536 - bar) if bar < 65536 else 0.0


def dropped(x, p, seed, step=0):
    """Elements left out are 0 whatever they hold."""
    return np.where(kept(*x.shape, p, seed, step), x * keep_scale(p), 0.0)


# ------------------------------------------------------------- layer norm --
# additions that one column's value goes through in a sum over a row: 32 in a
# lane, 6 over the lanes, 8 over the waves, and a few for the composition
ROW_SUM = 32 + 6 + 8 + 4


def layer_norm(v, w, b, eps):
    """y, mean, rstd of v and bounds on the FP32 error of each (y's before its
    rounding to the output's type)."""
    mean = v.mean(1, keepdims=True)
    d = v - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = (var + eps) ** -0.5
    n = d * rstd
    y = n * w + b
    e_mean = ROW_SUM * U * np.abs(v).mean(1, keepdims=True)
    # each difference is off by the mean's error and a rounding; the squares' sum by ROW_SUM roundings and their own
    e_d = e_mean + U * np.abs(d)
    e_var = (2 * np.abs(d) * e_d + e_d ** 2).mean(1, keepdims=True) + (ROW_SUM + 3) * U * var
    e_rstd = rstd * (0.5 * e_var / (var + eps) * 1.01 + 4 * U)
    e_y = np.abs(w) * (e_d * rstd + np.abs(d) * e_rstd) * 1.01 + 3 * U * (np.abs(n * w) + np.abs(b))
    return y, mean[:, 0], rstd[:, 0], e_y, e_mean[:, 0], e_rstd[:, 0]


def layer_norm_dgrad(dy, v, mean, rstd, w):
    """dv, dweight, dbias from given statistics, and bounds on the FP32 error."""
    H = v.shape[1]
    n = (v - mean[:, None]) * rstd[:, None]
    g = dy * w
    s1, s2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    dv = rstd[:, None] * (g - s1 - n * s2)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    del H
    e_dv = rstd[:, None] * U * (4 * np.abs(g) + (ROW_SUM + 5) * (a1 + np.abs(n) * a2) + 4 * np.abs(n) * a2)
    # a column's sum passes through at most all rows, 4 waves and 32 + 16 parts; n itself is off by 2 u
    depth = (dy.shape[0] + 4 + 48 + 3) * U
    return dv, (dy * n).sum(0), dy.sum(0), e_dv, depth * np.abs(dy * n).sum(0), depth * np.abs(dy).sum(0)


# -------------------------------------------------------------- recurrence --
def gates(g):
    """f and 1 - f, and a bound on their relative error: the exponential's argument
    is rounded (|g| u of the result), and a dozen roundings cover the exponential,
    the reciprocal, and one step's product, sum and composition."""
    with np.errstate(over="ignore"):
        small = np.exp(-np.abs(g))
    f = np.where(g >= 0, 1.0, small) / (1 + small)
    rest = np.where(g >= 0, small, 1.0) / (1 + small)
    return f, rest, (12 + 2 * np.where(np.isfinite(g), np.abs(g), 0)) * U


def recurrence(g, x, offsets, h0, coupled, dh=None, dlast=None):
    """A dict of h, state and, with dh, dgate, dx and dstate, each with the bound
    on its FP32 error under "e_" + name.  g, x, dh [R, D]; offsets a list.

    The recursion of the bound: with M the recursion of magnitudes (M_t = f M_(t-1)
    + |w x|), a step adds d M_t, d as of gates(), to f times the bound before it,
    and composing runs adds up the same terms in another order."""
    R, D = x.shape
    f, rest, d = gates(g)
    w = rest if coupled else np.ones_like(rest)
    S = len(offsets) - 1
    h0 = np.zeros((S, D)) if h0 is None else h0
    out = {k: np.zeros((R, D)) for k in ("h", "e_h")}
    out.update(state=h0.copy(), e_state=np.zeros((S, D)))
    before, m_before, e_before = np.zeros((R, D)), np.zeros((R, D)), np.zeros((R, D))
    times = lambda a, b: np.where(a == 0, 0.0, a * b)  # noqa: E731  a weight of 0 leaves its term out
    with np.errstate(invalid="ignore"):
        for s in range(S):
            h, m, e = h0[s].copy(), np.abs(h0[s]), np.zeros(D)
            for t in range(offsets[s], offsets[s + 1]):
                before[t], m_before[t], e_before[t] = h, m, e
                h = times(f[t], h) + times(w[t], x[t])
                m = times(f[t], m) + times(w[t], np.abs(x[t]))
                e = times(f[t], e) + d[t] * m
                out["h"][t], out["e_h"][t] = h, e
            out["state"][s], out["e_state"][s] = h, e
        if dh is None:
            return out
        dlast = np.zeros((S, D)) if dlast is None else dlast
        for k in ("dgate", "dx", "e_dgate", "e_dx"):
            out[k] = np.zeros((R, D))
        out.update(dstate=dlast.copy(), e_dstate=np.zeros((S, D)))
        for s in range(S):
            q, m, e = dlast[s].copy(), np.abs(dlast[s]), np.zeros(D)
            for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
                r, m, e = dh[t] + q, np.abs(dh[t]) + m, e + U * (np.abs(dh[t]) + m)
                slope = f[t] * rest[t]
                inner = before[t] - x[t] if coupled else before[t]
                m_inner = m_before[t] + np.abs(x[t]) if coupled else m_before[t]
                out["dx"][t] = times(w[t], r)
                out["e_dx"][t] = times(w[t], e + d[t] * m)
                out["dgate"][t] = times(slope, r * inner)
                out["e_dgate"][t] = times(slope, e * m_inner + m * e_before[t] + 2 * d[t] * m * m_inner)
                q, m, e = times(f[t], r), times(f[t], m), times(f[t], e + d[t] * m)
            out["dstate"][s], out["e_dstate"][s] = q, e
    return out
