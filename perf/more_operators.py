"""Measured cases of the operators between the projections of a residual block.

Three operators, each reached through ``deterministic_bf16_projection_amd``:

* layer norm, alone or of a residual sum whose new part passes through dropout,
  and its gradient with those of the weight and the bias;
* dropout from a counter-based generator, whose mask is never stored;
* a gated linear recurrence over sequences, its state, and its gradient.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's kernels; ``exact`` restates each operator's
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one generated token: the launch's latency
        {"name": "layer norm, one token", "op": "norm", "pass": "forward", "tokens": 1, "hidden": 4096, "x": "bf16",
         "y": "bf16"},
        # a training micro-batch
        {"name": "layer norm, training", "op": "norm", "pass": "forward", "tokens": 16384, "hidden": 4096,
         "x": "bf16", "y": "bf16"},
        {"name": "layer norm gradient, training", "op": "norm", "pass": "gradient", "tokens": 16384, "hidden": 4096,
         "x": "bf16", "y": "bf16"},
        # an odd number of short FP32 rows: a small model's last batch
        {"name": "layer norm gradient, odd, f32", "op": "norm", "pass": "gradient", "tokens": 1999, "hidden": 1032,
         "x": "f32", "y": "f32"},
        # an FP32 residual stream takes a sublayer's BF16 output through dropout, and its norm feeds the next one
        {"name": "residual sum and norm, training", "op": "add_norm", "pass": "forward", "tokens": 8192,
         "hidden": 4096, "x": "f32", "y": "bf16", "branch": "bf16", "p": 0.1},
        # the gradient of that at another width, with the gradient that comes down the stream
        {"name": "residual sum and norm, gradient", "op": "add_norm", "pass": "gradient", "tokens": 5003,
         "hidden": 5120, "x": "f32", "y": "bf16", "branch": "bf16", "p": 0.1},
        # a small batch's activations
        {"name": "dropout, small", "op": "dropout", "tokens": 32, "hidden": 1024, "x": "bf16", "residual": False,
         "p": 0.1},
        # the inner activations of a training micro-batch
        {"name": "dropout, training", "op": "dropout", "tokens": 16384, "hidden": 12288, "x": "bf16",
         "residual": False, "p": 0.1},
        # one generated token of each of 32 sequences, state in and out
        {"name": "recurrence, one token", "op": "recurrence", "pass": "forward", "sequences": 32, "length": 1,
         "packed": False, "tail": 0, "channels": 4096, "type": "bf16", "coupled": True, "state": True},
        # a training micro-batch, forward and backward
        {"name": "recurrence, training", "op": "recurrence", "pass": "train", "sequences": 8, "length": 4096,
         "packed": False, "tail": 0, "channels": 4096, "type": "bf16", "coupled": True, "state": False},
        # one long document before generation starts: few channels, many steps
        {"name": "recurrence, long sequence", "op": "recurrence", "pass": "forward", "sequences": 1,
         "length": 65536, "packed": False, "tail": 0, "channels": 2048, "type": "bf16", "coupled": True,
         "state": True},
        # sequences of any length packed one after the other, FP32, forward and backward, rows behind the last one
        {"name": "recurrence, packed, f32", "op": "recurrence", "pass": "train", "sequences": 37, "length": 541,
         "packed": True, "tail": 13, "channels": 1032, "type": "f32", "coupled": False, "state": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "add_norm", "dropout", "recurrence", "recurrence"))
    if kind != "recurrence":
        hidden = 8 * _log(rng, 2, 2048)
        tokens = max(1, min(_log(rng, 1, 65536), (1 << 26) // hidden))
        types = ("bf16", "f32")
        if kind == "dropout":
            return {"op": kind, "tokens": tokens, "hidden": hidden, "x": rng.choice(types),
                    "residual": rng.random() < 0.5, "p": round(rng.uniform(0.02, 0.6), 3)}
        case = {"op": kind, "pass": rng.choice(("forward", "gradient")), "tokens": tokens, "hidden": hidden}
        if kind == "norm":
            return {**case, "x": rng.choice(types), "y": rng.choice(types)}
        return {**case, "x": "f32", "y": rng.choice(types), "branch": rng.choice(types),
                "p": rng.choice((0.0, round(rng.uniform(0.02, 0.6), 3)))}
    channels = 8 * _log(rng, 2, 1024)
    rows = min(_log(rng, 1, 65536), (1 << 27) // channels)
    sequences = _log(rng, 1, min(rows, 4096))
    length = max(1, rows // sequences)
    packed = rng.random() < 0.4
    return {"op": "recurrence", "pass": rng.choice(("forward", "train")), "sequences": sequences, "length": length,
            "packed": packed, "tail": rng.choice((0, 5)) if packed else 0, "channels": channels,
            "type": rng.choice(("bf16", "f32")), "coupled": rng.random() < 0.5, "state": rng.random() < 0.5}


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0, mean=0.0):
    """Normal values, made in the type they are kept in (to spare memory)."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.normal_(mean, scale, generator=g)
    return t


# ------------------------------------------------------------------ inputs --
def _offsets(case, seed):
    """First row of each packed sequence and the end: skewed lengths, some of them zero."""
    rng = np.random.default_rng(seed)
    p = rng.standard_exponential(case["sequences"]) * (rng.random(case["sequences"]) > 0.05)
    p[rng.integers(case["sequences"])] += 0.5
    counts = rng.multinomial(case["sequences"] * case["length"], p / p.sum())
    return np.concatenate([[0], np.cumsum(counts)])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "recurrence":
        b, t, c, kind = case["sequences"], case["length"], case["channels"], _dtype(case["type"])
        rows = b * t + case["tail"]
        # gates whose memory reaches from one step to about a thousand, by channel
        s["gate"] = _randn(g, rows, c, dtype=kind, scale=1.0)
        s["gate"] += torch.empty(c, device=DEV).uniform_(-1.0, 7.0, generator=g).to(kind)
        s["x"] = _randn(g, rows, c, dtype=kind)
        if case["state"]:
            s["h0"] = _randn(g, b, c)
        if case["pass"] == "train":
            s["dh"] = _randn(g, rows, c, dtype=kind)
            if case["state"]:
                s["dlast"] = _randn(g, b, c)
        s["longest"] = t
        if case["packed"]:
            off = _offsets(case, seed)
            s["offsets"] = torch.from_numpy(off).to(DEV, torch.int32)
            s["longest"] = int(np.diff(off).max())
        else:
            for name in ("gate", "x", "dh"):
                if name in s:
                    s[name] = s[name].view(b, t, c)
        return s
    t, h = case["tokens"], case["hidden"]
    if case["op"] != "norm":
        s["seed"] = (seed * 0x9E3779B97F4A7C15 + 1) & ((1 << 63) - 1)
        s["step"] = torch.full((1,), seed % 1000, dtype=torch.int64, device=DEV)
    if case["op"] == "dropout":
        s["x"] = _randn(g, t, h, dtype=_dtype(case["x"]))
        if case["residual"]:
            s["r"] = _randn(g, t, h)
        return s
    s["weight"] = _randn(g, h, scale=0.2, mean=1.0)
    s["bias"] = _randn(g, h, scale=0.1)
    # rows of different sizes around a mean that is not zero
    stream = _randn(g, t, h, dtype=_dtype(case["x"]), mean=0.25)
    stream *= torch.empty(t, 1, device=DEV).uniform_(0.5, 3.0, generator=g).to(stream.dtype)
    if case["pass"] == "forward":
        if case["op"] == "norm":
            s["x"] = stream
        else:
            s["r"] = stream
            s["x"] = _randn(g, t, h, dtype=_dtype(case["branch"]))
        return s
    s["sum"] = stream  # what the forward pass normalised, and the statistics that it kept
    mean, rstd = torch.empty(t, device=DEV), torch.empty(t, device=DEV)
    for i in range(0, t, 8192):
        part = stream[i:i + 8192].double()
        mean[i:i + 8192] = part.mean(1)
        rstd[i:i + 8192] = (part.var(1, unbiased=False) + EPS).rsqrt()
    s["mean"], s["rstd"] = mean, rstd
    s["dy"] = _randn(g, t, h, dtype=_dtype(case["y"]))
    if case["op"] == "add_norm":
        s["dsum"] = _randn(g, t, h, dtype=stream.dtype)
    return s


# --------------------------------------------------------------------- run --
def run(state):
    if own:
        return {"norm": _own_norm, "add_norm": _own_add_norm, "dropout": _own_dropout,
                "recurrence": _own_recurrence}[state["op"]](state)
    return {"norm": _plain_norm, "add_norm": _plain_add_norm, "dropout": _plain_dropout,
            "recurrence": _plain_recurrence}[state["op"]](state)


def _own_norm(s):
    import deterministic_bf16_projection_amd as dpg
    if s["pass"] == "forward":
        n = dpg.dpg_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=_dtype(s["y"]))
        return {"y": n.y, "mean": n.mean, "rstd": n.rstd}
    d = dpg.dpg_layer_norm_dgrad(s["dy"], s["sum"], s["mean"], s["rstd"], s["weight"])
    return {"dx": d.dx, "dweight": d.dweight, "dbias": d.dbias}


def _own_add_norm(s):
    import deterministic_bf16_projection_amd as dpg
    if s["pass"] == "forward":
        n = dpg.dpg_add_layer_norm(s["x"], s["r"], s["weight"], s["bias"], eps=EPS, p=s["p"], seed=s["seed"],
                                   step=s["step"], out_dtype=_dtype(s["y"]))
        return {"y": n.y, "sum": n.sum, "mean": n.mean, "rstd": n.rstd}
    d = dpg.dpg_add_layer_norm_dgrad(s["dy"], s["sum"], s["mean"], s["rstd"], s["weight"], dsum=s["dsum"], p=s["p"],
                                     seed=s["seed"], step=s["step"], x_dtype=_dtype(s["branch"]))
    return {"dx": d.dx, "dresidual": d.dresidual, "dweight": d.dweight, "dbias": d.dbias}


def _own_dropout(s):
    import deterministic_bf16_projection_amd as dpg
    return dpg.dpg_dropout(s["x"], s["p"], s["seed"], step=s["step"], residual=s.get("r"))


def _own_recurrence(s):
    import deterministic_bf16_projection_amd as dpg
    train = s["pass"] == "train"
    r = dpg.dpg_recurrence(s["gate"], s["x"], offsets=s.get("offsets"), state=s.get("h0"), coupled=s["coupled"],
                           carries=train)
    out = {"h": r.h, "state": r.state}
    if train:
        d = dpg.dpg_recurrence_dgrad(s["dh"], s["gate"], s["x"], r.carries, offsets=s.get("offsets"),
                                     state=s.get("h0"), dstate=s.get("dlast"), coupled=s["coupled"])
        out.update(dgate=d.dgate, dx=d.dx)
        if s["state"]:
            out["dstate"] = d.dstate
    return out


def _product(a, m):
    """High and low words of a (32 bits, in 64) times the constant m."""
    wide = a * m                      # modulo 2^64: the sign bit is the product's highest
    return (wide >> 32) & 0xFFFFFFFF, wide & 0xFFFFFFFF


def _random16(n, seed, step):
    """16 random bits for each of n elements: element 8 g + j takes half j % 2 (low first) of word j // 2 of
    Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, 2011) of the counter (g, step), both in 64 bits, low
    words first, under the key `seed`."""
    g = torch.arange(-(-n // 8), device=DEV)
    c = [g & 0xFFFFFFFF, g >> 32, (step & 0xFFFFFFFF).expand_as(g), ((step >> 32) & 0xFFFFFFFF).expand_as(g)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):  # the generator's rounds
        h0, l0 = _product(c[0], 0xD2511F53)
        h1, l1 = _product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]


def _dropped(x, s):
    """x with each element left out with probability p (a multiple of 2^-16), the others scaled, in 32 bits."""
    bar = round(s["p"] * 65536)
    if bar == 0:
        return x.float()
    kept = (_random16(x.numel(), s["seed"], s["step"]) >= bar).view(x.shape)
    return torch.where(kept, x.float() * (65536.0 / (65536 - bar)), torch.zeros((), device=DEV))


def _plain_dropout(s):
    v = _dropped(s["x"], s)
    return v + s["r"] if s["residual"] else v.to(s["x"].dtype)


def _plain_statistics(x):
    mean = x.mean(1, keepdim=True)
    centred = x - mean
    return mean, torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    if s["pass"] == "gradient":
        dx, dw, db = _plain_norm_gradient(s)
        return {"dx": dx.to(s["sum"].dtype), "dweight": dw, "dbias": db}
    x = s["x"].float()
    mean, rstd = _plain_statistics(x)
    return {"y": ((x - mean) * rstd * s["weight"] + s["bias"]).to(_dtype(s["y"])), "mean": mean[:, 0],
            "rstd": rstd[:, 0]}


def _plain_norm_gradient(s):
    dy, xhat = s["dy"].float(), (s["sum"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    u = dy * s["weight"]
    dx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _plain_add_norm(s):
    if s["pass"] == "gradient":
        dx, dw, db = _plain_norm_gradient(s)
        dx = dx + s["dsum"].float()
        return {"dx": _dropped(dx, s).to(_dtype(s["branch"])), "dresidual": dx.to(s["sum"].dtype), "dweight": dw,
                "dbias": db}
    total = s["r"].float() + _dropped(s["x"], s)
    mean, rstd = _plain_statistics(total)
    return {"y": ((total - mean) * rstd * s["weight"] + s["bias"]).to(_dtype(s["y"])), "sum": total.to(s["r"].dtype),
            "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _rows(t):
    return t.view(-1, t.shape[-1]) if t.dim() == 3 else t


def _scan(f, b, longest):
    """h[t] = f[t] h[t - 1] + b[t] over the rows (f zero where a sequence starts), by doubling the reach."""
    a, h, k = f.clone(), b.clone(), 1
    while k < longest:
        h[k:] = h[k:] + a[k:] * h[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return h


def _shift(t):
    """Row r - 1 at row r, zeros at the first."""
    return torch.cat([torch.zeros_like(t[:1]), t[:-1]])


def _plain_recurrence(s):
    gate, x, kind = _rows(s["gate"]).float(), _rows(s["x"]).float(), s["x"].dtype
    rows, c, n = gate.shape[0], gate.shape[1], s["sequences"]
    off = s["offsets"].long() if s["packed"] else torch.arange(n + 1, device=DEV) * s["length"]
    row = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(off[1:], row, right=True)                 # n behind the last sequence
    live, at = (seq < n)[:, None], seq.clamp(max=n - 1)
    first = live & (row == off[at])[:, None]
    last = live & (row == off[at + 1] - 1)[:, None]
    small = torch.exp(-gate.abs())                                     # the smaller of both weights, over their sum
    f = torch.where(gate >= 0, torch.ones_like(small), small) / (1 + small)
    i = torch.where(gate >= 0, small, torch.ones_like(small)) / (1 + small)
    h0 = s["h0"] if s["state"] else torch.zeros(n, c, device=DEV)
    weight = i if s["coupled"] else torch.ones_like(i)
    zero = torch.zeros((), device=DEV)
    b = torch.where(live, weight * x, zero) + torch.where(first, f * h0[at], zero)
    on = torch.where(live & ~first, f, zero)                           # what reaches a row from the one before
    h = _scan(on, b, s["longest"])
    filled = (off[1:] > off[:-1])[:, None]
    out = {"h": h.to(kind).view(s["x"].shape), "state": torch.where(filled, h[(off[1:] - 1).clamp(min=0)], h0)}
    if s["pass"] == "train":
        dh = torch.where(live, _rows(s["dh"]).float(), zero)
        if s["state"]:
            dh = dh + torch.where(last, s["dlast"][at], zero)
        back = _shift(on.flip(0))                                      # row r + 1's weight at row r, from the end
        r = _scan(back, dh.flip(0), s["longest"]).flip(0)
        before = torch.where(first, h0[at], _shift(h))
        out["dgate"] = (f * i * r * (before - x if s["coupled"] else before)).to(kind)
        out["dx"] = (weight * r).to(kind)
        for name in ("dgate", "dx"):
            out[name] = torch.where(live, out[name], torch.zeros((), dtype=kind, device=DEV)).view(s["x"].shape)
        if s["state"]:
            start = off[:-1].clamp(max=rows - 1)
            out["dstate"] = torch.where(filled, f[start] * r[start], s["dlast"])
    return out


# -------------------------------------------------------------------- work --
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "recurrence":
        b, c, e = case["sequences"], case["channels"], size[case["type"]]
        n, every = b * case["length"] * c, (b * case["length"] + case["tail"]) * c
        states = b * c * 4
        data, flops = 2 * n * e + every * e + states * (2 if case["state"] else 1), 8 * n
        if case["pass"] == "train":
            # the inputs again, the gradient of h, and the gradients of both inputs
            data += 3 * n * e + 2 * every * e + (3 * states if case["state"] else 0)
            flops += 16 * n
        return {"bytes": data + (4 * (b + 1) if case["packed"] else 0), "flops": flops}
    n, t, h = case["tokens"] * case["hidden"], case["tokens"], case["hidden"]
    if case["op"] == "dropout":
        e = size[case["x"]]
        return {"bytes": n * (e + (8 if case["residual"] else e)), "flops": 2 * n}
    data = n * (size[case["x"]] + size[case["y"]]) + 8 * t + 8 * h     # input and output, statistics, weights
    flops = 8 * n
    if case["pass"] == "gradient":
        data += n * size[case["x"]] + 4 * h                            # dx; dweight and dbias, without the bias
        flops = 14 * n
    if case["op"] == "add_norm":
        data += n * (size[case["branch"]] + size[case["x"]])           # the branch or its gradient; the sum or dsum
        flops += 2 * n
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "add_norm": _exact_norm, "dropout": _exact_dropout,
            "recurrence": _exact_recurrence}[case["op"]](s)


def _exact_words(n, seed, step):
    """The generator's words for n elements, products from 16-bit limbs: int64 [4, n / 8 rounded up]."""
    groups = torch.arange((n + 7) // 8, device=DEV)
    low = 2 ** 32 - 1
    step = int(step)
    state = torch.stack([groups % 2 ** 32, groups // 2 ** 32, torch.full_like(groups, step & low),
                         torch.full_like(groups, step >> 32 & low)])
    for i in range(10):
        keys = [(seed + i * 0x9E3779B9) & low, ((seed >> 32) + i * 0xBB67AE85) & low]
        high, rest = [], []
        for word, m in ((state[0], 0xD2511F53), (state[2], 0xCD9E8D57)):
            by_low, by_high = word * (m % 65536), word * (m // 65536)  # below 2^48
            upper = by_high + by_low // 65536                          # the product without its lowest 16 bits
            high.append(upper // 65536)
            rest.append(upper % 65536 * 65536 + by_low % 65536)
        state = torch.stack([high[1] ^ state[1] ^ keys[0], rest[1], high[0] ^ state[3] ^ keys[1], rest[0]])
    return state


def _exact_kept(shape, s):
    """1 / (1 - p) where an element stays, 0 where it is left out."""
    n, bar = math.prod(shape), int(math.floor(s["p"] * 65536 + 0.5))
    words = _exact_words(n, s["seed"], s["step"])
    halves = torch.stack([words % 65536, words // 65536], 1)            # [word, half, group]
    bits = halves.reshape(8, -1).T.reshape(-1)[:n].view(shape)
    return (bits >= bar).double() / (1.0 - bar / 65536.0)


def _exact_dropout(s):
    y = s["x"].double()
    y *= _exact_kept(y.shape, s)
    return y + s["r"].double() if s["residual"] else y


def _exact_norm(s):
    add = s["op"] == "add_norm"
    w = s["weight"].double()
    h = w.numel()
    if s["pass"] == "forward":
        total = s["x"].double()
        if add:
            total = s["r"].double() + total * _exact_kept(total.shape, s)
        mean = total.sum(1) / h
        var = (total - mean[:, None]).square().sum(1) / h
        rstd = 1.0 / torch.sqrt(var + EPS)
        out = {"y": (total - mean[:, None]) * rstd[:, None] * w + s["bias"].double(), "mean": mean, "rstd": rstd}
        return {**out, "sum": total} if add else out
    rstd = s["rstd"].double()[:, None]
    unit, dy = (s["sum"].double() - s["mean"].double()[:, None]) * rstd, s["dy"].double()
    out = {"dweight": torch.sum(dy * unit, 0), "dbias": torch.sum(dy, 0)}
    grad = dy * w
    grad = (grad - grad.sum(1, keepdim=True) / h - unit * ((grad * unit).sum(1, keepdim=True) / h)) * rstd
    if not add:
        return {**out, "dx": grad}
    grad = grad + s["dsum"].double()
    return {**out, "dresidual": grad, "dx": grad * _exact_kept(grad.shape, s)}


def _exact_recurrence(s):
    """Step by step: all sequences at once where they are equally long, else one after the other."""
    c, n = s["channels"], s["sequences"]
    shape = s["x"].shape
    f = torch.sigmoid(s["gate"].double())
    i = torch.sigmoid(-s["gate"].double())
    x = s["x"].double()
    u = i * x if s["coupled"] else x
    h0 = s["h0"].double() if s["state"] else torch.zeros(n, c, dtype=torch.float64, device=DEV)
    train = s["pass"] == "train"
    dh = s["dh"].double() if train else None
    dlast = s["dlast"].double() if train and s["state"] else torch.zeros_like(h0)
    h, before, r = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    state, dstate = h0.clone(), dlast.clone()

    def steps(places, v, w):
        """Forward from v over the places, then backward from w."""
        for at in places:
            before[at] = v
            v = f[at] * v + u[at]
            h[at] = v
        if train:
            for at in reversed(places):
                w = dh[at] + w
                r[at] = w
                w = f[at] * w
        return v, w

    if s["packed"]:
        off = s["offsets"].cpu().tolist()
        for q in range(n):
            state[q], dstate[q] = steps(range(off[q], off[q + 1]), h0[q], dlast[q])
    else:
        state, dstate = steps([(slice(None), t) for t in range(shape[1])], h0, dlast)
    out = {"h": h, "state": state}
    if train:
        out["dx"] = i * r if s["coupled"] else r
        out["dgate"] = f * i * r * (before - x if s["coupled"] else before)
        if s["state"]:
            out["dstate"] = dstate
    return out
