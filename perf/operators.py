"""Measured cases of the expert-layer training operators.

Three operators, each reached through ``deterministic_bf16_projection_amd``:

* grouped projections: the rows of a token batch, sorted by expert, times each
  expert's own weight matrix, in the three directions of training;
* routing: the choice of experts from router logits, the rows moved into
  expert order and back, and the gradients of all of that;
* AdamW over many tensors at once, with 32-bit or 8-bit moments.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's kernels; ``exact`` restates each operator's
definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 256          # elements that share one scale of an 8-bit moment
BETA1, BETA2, EPS, DECAY, LR, STEP = 0.9, 0.95, 1e-8, 0.1, 3e-4, 10


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one generated token, 8 of 256 experts: eight weight matrices are read for eight rows
        {"name": "grouped forward, one token", "op": "grouped", "pass": "forward", "rows": 8, "experts": 256,
         "n": 512, "k": 4096, "out": "bf16", "tail": 0},
        # a serving batch of 32 tokens, 8 experts each: a few rows for nearly every expert
        {"name": "grouped forward, 32 tokens", "op": "grouped", "pass": "forward", "rows": 256, "experts": 64,
         "n": 1024, "k": 4096, "out": "bf16", "tail": 0},
        # a training micro-batch of 8192 tokens, 8 experts each
        {"name": "grouped forward, training", "op": "grouped", "pass": "forward", "rows": 65536, "experts": 64,
         "n": 1024, "k": 4096, "out": "bf16", "tail": 0},
        # the input gradient of a smaller batch with an odd number of rows, some of them routed nowhere
        {"name": "grouped input gradient, odd", "op": "grouped", "pass": "dgrad", "rows": 24573, "experts": 40,
         "n": 1032, "k": 4096, "out": "bf16", "tail": 29},
        # the weight gradient of the training micro-batch, in FP32 for the optimizer
        {"name": "grouped weight gradient, f32", "op": "grouped", "pass": "wgrad", "rows": 65536, "experts": 64,
         "n": 1024, "k": 4096, "out": "f32", "tail": 0},
        # few tokens for each of 16 small experts, BF16 gradients
        {"name": "grouped weight gradient, small", "op": "grouped", "pass": "wgrad", "rows": 2001, "experts": 16,
         "n": 512, "k": 1024, "out": "bf16", "tail": 0},
        # routing of one generated token: the launches' latency
        {"name": "routing, one token", "op": "route", "tokens": 1, "experts": 256, "top_k": 8, "hidden": 4096,
         "renormalize": True, "grad": False, "masked": 0.0},
        # routing of a serving batch where an eighth of the experts is switched off
        {"name": "routing, 201 tokens, masked", "op": "route", "tokens": 201, "experts": 64, "top_k": 6,
         "hidden": 2048, "renormalize": False, "grad": False, "masked": 0.125},
        # routing of a training batch, forward and backward
        {"name": "routing, training", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "hidden": 4096,
         "renormalize": True, "grad": True, "masked": 0.0},
        # the norms, biases and routers of a small model: many little tensors
        {"name": "AdamW, small tensors", "op": "adamw", "tensors": 48, "largest": 65536, "total": 400000,
         "state": "f32", "grad": "f32", "copy": True},
        # the experts of one layer with 32-bit moments and BF16 gradients
        {"name": "AdamW, 32-bit moments", "op": "adamw", "tensors": 12, "largest": 64 * 1024 * 1024,
         "total": 201326592, "state": "f32", "grad": "bf16", "copy": True},
        # the experts of one layer with 8-bit moments and FP32 gradients
        {"name": "AdamW, 8-bit moments", "op": "adamw", "tensors": 12, "largest": 64 * 1024 * 1024,
         "total": 201326592, "state": "e4m3", "grad": "f32", "copy": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("grouped", "grouped", "route", "adamw"))
    if kind == "grouped":
        n, k = 8 * _log(rng, 8, 256), 8 * _log(rng, 16, 512)
        experts = _log(rng, 1, 256)
        experts = max(1, min(experts, (1 << 28) // (n * k)))
        rows = _log(rng, 1, 65536)
        rows = max(1, min(rows, (1 << 38) // (n * k)))
        return {"op": "grouped", "pass": rng.choice(("forward", "dgrad", "wgrad")), "rows": rows, "experts": experts,
                "n": n, "k": k, "out": rng.choice(("bf16", "f32")), "tail": rng.choice((0, 0, min(rows - 1, 17)))}
    if kind == "route":
        experts = _log(rng, 2, 512)
        top_k = rng.randint(1, min(experts, 10))
        hidden = 8 * _log(rng, 16, 640)
        tokens = _log(rng, 1, 32768)
        tokens = max(1, min(tokens, (1 << 29) // (top_k * hidden)))
        return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
                "renormalize": rng.random() < 0.5, "grad": rng.random() < 0.5,
                "masked": rng.choice((0.0, round(rng.uniform(0.05, 0.6), 3)))}
    tensors = _log(rng, 1, 100)
    largest = _log(rng, 256, 1 << 26)
    return {"op": "adamw", "tensors": tensors, "largest": largest,
            "total": max(tensors, min(201326592, int(largest * rng.uniform(0.5, 1.0) * tensors))),
            "state": rng.choice(("f32", "e4m3")), "grad": rng.choice(("f32", "bf16")), "copy": rng.random() < 0.5}


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    """Normal values, made in the type they are kept in (a slice at a time, to spare memory)."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.normal_(0.0, scale, generator=g)
    return t


# ------------------------------------------------------------------ inputs --
def _counts(case, seed):
    """Rows of each expert: a skewed split of the routed rows, some experts without any."""
    rng = np.random.default_rng(seed)
    p = np.exp(0.6 * rng.standard_normal(case["experts"]))
    return rng.multinomial(case["rows"] - case["tail"], p / p.sum())


def _sizes(case):
    """Element counts of the tensors: odd ones among them, the same for every seed."""
    rng = random.Random(case["tensors"] * 7919 + case["total"])
    left, n = case["total"], case["tensors"]
    sizes = []
    for i in range(n):
        share = left / (n - i)
        s = int(max(1, min(case["largest"], share * rng.uniform(0.2, 1.8))))
        sizes.append(s if i + 1 < n else max(1, min(case["largest"], left)))
        left = max(1, left - sizes[-1])
    return sizes


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "grouped":
        counts = _counts(case, seed)
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
        s["active"] = torch.tensor(np.nonzero(counts)[0], dtype=torch.int64, device=DEV)  # the experts with rows
        s["longest"] = int(counts.max())
        if case["pass"] != "dgrad":
            s["x"] = _randn(g, r, k, dtype=torch.bfloat16)
        if case["pass"] != "forward":
            s["dy"] = _randn(g, r, n, dtype=torch.bfloat16)
        if case["pass"] != "wgrad":
            s["w"] = _randn(g, e, n, k, dtype=torch.bfloat16, scale=0.02)
        return s
    if case["op"] == "route":
        t, e, k, h = case["tokens"], case["experts"], case["top_k"], case["hidden"]
        logits = _randn(g, t, e) + 0.5 * _randn(g, 1, e)
        if case["masked"]:
            logits = torch.where(torch.rand(t, e, generator=g, device=DEV) < case["masked"],
                                 torch.full_like(logits, -math.inf), logits)
            logits[t // 2] = -math.inf  # a token that no expert may take
        s["logits"] = logits
        s["x"] = _randn(g, t, h, dtype=torch.bfloat16)
        s["ys"] = _randn(g, t * k, h, dtype=torch.bfloat16)  # the experts' outputs
        if case["grad"]:
            s["dy"] = _randn(g, t, h, dtype=torch.bfloat16)
            s["dxs"] = _randn(g, t * k, h, dtype=torch.bfloat16)  # gradient of the moved rows
        return s
    # Every tensor is a view of one flat buffer, as a bucketing trainer keeps them; each starts at a block.
    sizes = _sizes(case)
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
    total, s["sizes"] = int(starts[-1]), sizes
    # what lies between the tensors belongs to none of them and stays zero
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for n, a in zip(sizes, starts):
        inside[int(a):int(a) + n] = True
    flat = {"p": _randn(g, total, scale=0.02), "g": _randn(g, total, dtype=_dtype(case["grad"]), scale=1e-3)}
    if case["state"] == "f32":
        flat["m"] = _randn(g, total, scale=3e-4)
        flat["v"] = _randn(g, total, scale=1e-3).square_()
    else:
        # moments as an earlier step leaves them: codes whose block's largest is near the type's top
        flat["m"] = _randn(g, total, scale=120.0).clamp_(-448, 448)
        flat["v"] = _randn(g, total, scale=120.0).abs_().clamp_(0.002, 448)
    for t in flat.values():
        t.mul_(inside)
    if case["state"] == "e4m3":
        flat["m"], flat["v"] = (flat[n].to(torch.float8_e4m3fn) for n in ("m", "v"))
        for name in ("ms", "vs"):
            e = torch.randint(-20, -17, (total // BLOCK,), generator=g, device=DEV)
            flat[name] = torch.exp2(e.float())
    if case["copy"]:
        flat["w"] = flat["p"].to(torch.bfloat16)
    s["flat"] = flat
    for name, t in flat.items():
        unit = BLOCK if name in ("ms", "vs") else 1
        s[name] = [t[int(a) // unit: int(a) // unit + -(-n // unit)] for a, n in zip(starts, sizes)]
    s["grad_scale"] = torch.rand(1, generator=g, device=DEV) * 0.5 + 0.5  # clipping factor, from the gradients' norm
    s["seed"] = seed & 0xFFFFFFFF
    return s


# --------------------------------------------------------------------- run --
def run(state):
    if own:
        return {"grouped": _own_grouped, "route": _own_route, "adamw": _own_adamw}[state["op"]](state)
    return {"grouped": _plain_grouped, "route": _plain_route, "adamw": _plain_adamw}[state["op"]](state)


def _own_grouped(s):
    import deterministic_bf16_projection_amd as dpg
    out = _dtype(s["out"])
    if s["pass"] == "forward":
        return dpg.dpg_grouped_forward(s["x"], s["w"], s["offsets"], out_dtype=out)
    if s["pass"] == "dgrad":
        return dpg.dpg_grouped_dgrad(s["dy"], s["w"], s["offsets"], out_dtype=out)
    return dpg.dpg_grouped_wgrad(s["dy"], s["x"], s["offsets"], out_dtype=out)


def _own_route(s):
    import deterministic_bf16_projection_amd as dpg
    r = dpg.dpg_route(s["logits"], s["top_k"], renormalize=s["renormalize"])
    out = {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "rows": r.rows,
           "positions": r.positions,
           "xs": dpg.dpg_dispatch(s["x"], r.positions, r.offsets),
           "y": dpg.dpg_combine(s["ys"], r.positions, r.offsets, r.weights)}
    if s["grad"]:
        out["dys"], out["dweights"] = dpg.dpg_combine_dgrad(s["dy"], s["ys"], r.positions, r.offsets, r.weights)
        out["dlogits"] = dpg.dpg_route_dgrad(s["logits"], r.experts, r.weights, out["dweights"],
                                             renormalize=s["renormalize"])
        out["dx"] = dpg.dpg_combine(s["dxs"], r.positions, r.offsets)
    return out


def _own_adamw(s):
    import deterministic_bf16_projection_amd as dpg
    dpg.dpg_adamw(s["p"], s["g"], s["m"], s["v"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                  step=STEP, copies=s.get("w"), avg_scales=s.get("ms"), sq_scales=s.get("vs"),
                  grad_scale=s["grad_scale"], seed=s["seed"])
    return {k: v for k, v in s["flat"].items() if k != "g"}


def _plain_grouped(s):
    # rows go to a [experts with rows, longest group] frame, one batched product, and back
    off, out = s["offsets"].long(), _dtype(s["out"])
    a, longest, n = s["active"], s["longest"], s["rows"] - s["tail"]
    row = torch.arange(n, device=DEV)
    expert = torch.searchsorted(off[1:], row, right=True)
    group, slot = torch.searchsorted(a, expert), row - off[expert]

    def frame(t):
        f = torch.zeros(len(a), longest, t.shape[1], device=DEV)
        f[group, slot] = t[:n].float()
        return f

    def back(f):
        r = torch.zeros(s["rows"], f.shape[2], dtype=out, device=DEV)
        r[:n] = f[group, slot].to(out)
        return r

    if s["pass"] == "forward":
        return back(torch.bmm(frame(s["x"]), s["w"][a].float().transpose(1, 2)))
    if s["pass"] == "dgrad":
        return back(torch.bmm(frame(s["dy"]), s["w"][a].float()))
    dw = torch.zeros(s["experts"], s["n"], s["k"], dtype=out, device=DEV)
    dw[a] = torch.bmm(frame(s["dy"]).transpose(1, 2), frame(s["x"])).to(out)
    return dw


def _plain_route(s):
    logits, k, e = s["logits"], s["top_k"], s["experts"]
    t, h = s["x"].shape
    value, index = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lowest index first
    value, index = value[:, :k], index[:, :k]
    chosen = value > -math.inf
    top = torch.where(chosen[:, :1], value[:, :1], torch.zeros_like(value[:, :1]))
    part = torch.where(chosen, torch.exp(value - top), torch.zeros_like(value))
    whole = part if s["renormalize"] else torch.exp(logits - top)
    total = whole.sum(1, keepdim=True)
    weights = part / torch.where(total > 0, total, torch.ones_like(total))
    key = torch.where(chosen, index, torch.full_like(index, e)).reshape(-1)
    key, rows = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=DEV))
    positions = torch.empty_like(rows)
    positions[rows] = torch.arange(t * k, device=DEV)
    positions = positions.view(t, k)
    routed = (torch.arange(t * k, device=DEV) < offsets[e])[:, None]
    out = {"experts": torch.where(chosen, index, torch.full_like(index, -1)).int(), "weights": weights,
           "offsets": offsets.int(), "rows": rows.int(), "positions": positions.int(),
           "xs": torch.where(routed, s["x"][rows // k], torch.zeros((), dtype=s["x"].dtype, device=DEV))}
    back = torch.where(chosen[..., None], s["ys"][positions], torch.zeros((), dtype=s["ys"].dtype, device=DEV))
    out["y"] = (back.float() * weights[..., None]).sum(1).to(torch.bfloat16)
    if s["grad"]:
        dy = s["dy"].float()
        out["dweights"] = (back.float() * dy[:, None, :]).sum(2)
        dys = torch.zeros(t * k, h, dtype=torch.bfloat16, device=DEV)
        dys[positions.reshape(-1)] = (dy[:, None, :] * weights[..., None]).to(torch.bfloat16).view(t * k, h)
        out["dys"] = dys
        inner = (weights * out["dweights"]).sum(1, keepdim=True)
        if s["renormalize"]:
            dlogits = torch.zeros_like(logits)
        else:
            dlogits = -torch.exp(logits - top) / torch.where(total > 0, total, torch.ones_like(total)) * inner
        d = weights * (out["dweights"] - inner) if s["renormalize"] else weights * out["dweights"]
        out["dlogits"] = dlogits.scatter_add(1, index, torch.where(chosen, d, torch.zeros_like(d)))
        dx = torch.where(chosen[..., None], s["dxs"][positions], torch.zeros((), dtype=torch.bfloat16, device=DEV))
        out["dx"] = dx.float().sum(1).to(torch.bfloat16)
    return out


def _random_words(seed, tensor, n):
    """One 32-bit word for each of a tensor's n (< 2^32) elements, from the call's seed and the tensor's place
    among the call's tensors: x = i * A + key, then two rounds of (x ^= x >> s; x *= odd) and a last x ^= x >> 16,
    all modulo 2^32; the key is the same mix of seed + (tensor + 1) * A."""
    mask = 0xFFFFFFFF
    a, b, c = 0x9E3779B9, 0x6A09E667, 0xBB67AE85  # fractions of the golden ratio, sqrt(2) and sqrt(3), odd

    def mix(x):
        x = x ^ (x >> 16)
        x = (x * b) & mask
        x = x ^ (x >> 15)
        x = (x * c) & mask
        return x ^ (x >> 16)

    key = mix((seed + (tensor + 1) * a) & mask)
    return mix((torch.arange(n, device=DEV) * a + key) & mask)


def _scale_of(block_max):
    """The power of two that brings a block's largest magnitude to (224, 448]; 1 for a block of zeros."""
    f, e = torch.frexp(block_max / 448.0)
    e = torch.where(f == 0.5, e - 1, e).clamp(-120, 127)
    return torch.where(block_max > 0, torch.exp2(e.float()), torch.ones_like(block_max))


def _to_e4m3(x, bits16, scale, floor):
    """|x| / scale rounded up or down to a neighbouring E4M3 value, up with the probability of its distance from
    the lower one (16 random bits); with `floor`, positive values are not rounded to zero. As float8 values."""
    mag = (x.abs() / scale.repeat_interleave(BLOCK)[: x.numel()]).clamp_(max=448.0)
    r = (bits16 << 4) + 8
    big = (mag.view(torch.int32).long() + r) >> 20          # sign-free bits: 8 exponent and 3 mantissa bits
    big = big - (120 << 3)                                   # exponent bias 127 -> 7
    small = ((mag * 2.0 ** 29).long() + r) >> 20             # below 2^-6 the steps are 2^-9
    code = torch.where(mag < 2.0 ** -6, small, big).clamp_(max=126)
    if floor:
        code = torch.where(mag > 0, code.clamp(min=1), code)
    code = torch.where(x < 0, code | 128, code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn)


def _block_max(x):
    n = x.numel()
    pad = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK))
    return pad.view(-1, BLOCK).amax(1)


def _plain_step(i, s):
    p, g = s["p"][i], s["g"][i].float() * s["grad_scale"]
    m, v = s["m"][i], s["v"][i]
    bc1, bc2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    if s["state"] == "e4m3":
        m32 = m.float() * s["ms"][i].repeat_interleave(BLOCK)[: p.numel()]
        v32 = (v.float() * s["vs"][i].repeat_interleave(BLOCK)[: p.numel()]).square()  # the root is what is kept
    else:
        m32, v32 = m, v
    m32 = BETA1 * m32 + (1.0 - BETA1) * g
    v32 = BETA2 * v32 + (1.0 - BETA2) * g * g
    root = torch.sqrt(v32)
    p.mul_(1.0 - LR * DECAY).sub_((LR / bc1) * m32 / (root / math.sqrt(bc2) + EPS))
    if s["copy"]:
        s["w"][i].copy_(p)
    if s["state"] == "f32":
        m.copy_(m32)
        v.copy_(v32)
        return
    word = _random_words(s["seed"], i, p.numel())
    ms, vs = _scale_of(_block_max(m32)), _scale_of(_block_max(root))
    m.copy_(_to_e4m3(m32, word & 0xFFFF, ms, False))
    v.copy_(_to_e4m3(root, word >> 16, vs, True))
    s["ms"][i].copy_(ms)
    s["vs"][i].copy_(vs)


def _plain_adamw(s):
    for i in range(len(s["p"])):  # one tensor after the other
        _plain_step(i, s)
    return {k: v for k, v in s["flat"].items() if k != "g"}


# -------------------------------------------------------------------- work --
def work(case):
    if case["op"] == "grouped":
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        routed, out = r - case["tail"], 2 if case["out"] == "bf16" else 4
        if case["pass"] == "wgrad":
            data = routed * (n + k) * 2 + e * n * k * out
        else:
            # experts that hold a row, about: each one's weights are read once
            used = min(e, e * (1.0 - math.exp(-routed / e)) + 1)
            data = routed * (k if case["pass"] == "forward" else n) * 2 + used * n * k * 2
            data += r * (n if case["pass"] == "forward" else k) * out
        return {"bytes": data + 4 * (e + 1), "flops": 2.0 * routed * n * k}
    if case["op"] == "route":
        t, e, k, h = case["tokens"], case["experts"], case["top_k"], case["hidden"]
        data = t * e * 4 + t * k * 16 + (e + 1) * 4       # logits; experts, weights, rows and positions
        data += t * h * 2 + t * k * h * 2                 # rows moved
        data += t * k * h * 2 + t * h * 2                 # rows joined
        flops = t * e * 4 + 2 * t * k * h
        if case["grad"]:
            data += t * h * 2 + 2 * t * k * h * 2 + t * k * 4  # dy, ys read again, dys and dweights written
            data += 2 * t * e * 4 + t * k * h * 2 + t * h * 2  # dlogits from the logits, dx
            flops += 4 * t * k * h + t * e * 4
        return {"bytes": data, "flops": flops}
    n = sum(_sizes(case))
    each = 8 + (2 if case["grad"] == "bf16" else 4) + (2 if case["copy"] else 0)
    each += 16 if case["state"] == "f32" else 4 + 4 * 4 / BLOCK
    return {"bytes": n * each, "flops": n * 16}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    return {"grouped": _exact_grouped, "route": _exact_route, "adamw": _exact_adamw}[case["op"]](s)


def _exact_grouped(s):
    off = s["offsets"].cpu().tolist()
    rows, n, k = s["rows"], s["n"], s["k"]
    shape = {"forward": (rows, n), "dgrad": (rows, k), "wgrad": (s["experts"], n, k)}[s["pass"]]
    out = torch.zeros(shape, dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        if s["pass"] == "forward":
            out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
        elif s["pass"] == "dgrad":
            out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        else:
            out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
    return out


def _exact_route(s):
    lg, k = s["logits"].double().cpu().numpy(), s["top_k"]
    t, e = lg.shape
    h = s["x"].shape[1]
    order = np.lexsort((np.broadcast_to(np.arange(e), lg.shape), -lg), axis=1)[:, :k]
    val = np.take_along_axis(lg, order, 1)
    ok = np.isfinite(val)
    top = np.where(np.isfinite(lg).any(1), lg.max(1), 0.0)[:, None]
    z = np.exp(lg - top)
    picked = np.zeros_like(z)
    np.put_along_axis(picked, order, ok.astype(float), 1)
    base = z * picked if s["renormalize"] else z
    den = base.sum(1, keepdims=True)
    prob = base / np.where(den > 0, den, 1.0)
    w = np.take_along_axis(prob, order, 1) * ok
    slot_expert = np.where(ok, order, e).reshape(-1)
    counts = np.bincount(slot_expert, minlength=e + 1)
    offsets = np.concatenate([[0], np.cumsum(counts[:e])])
    rows = np.lexsort((np.arange(t * k), slot_expert))
    place = np.argsort(rows)
    dev = lambda v, d=torch.float64: torch.from_numpy(np.ascontiguousarray(v)).to(DEV, d)  # noqa: E731
    live = dev(np.arange(t * k) < offsets[e])[:, None]
    at, w2, okd = dev(place, torch.int64).view(t, k), dev(w), dev(ok)
    out = {"experts": dev(np.where(ok, order, -1), torch.int32), "weights": w2, "offsets": dev(offsets, torch.int32),
           "rows": dev(rows, torch.int32), "positions": dev(place, torch.int32).view(t, k),
           "xs": s["x"].double()[dev(rows // k, torch.int64)] * live}
    y, dx = torch.zeros(t, h, dtype=torch.float64, device=DEV), torch.zeros(t, h, dtype=torch.float64, device=DEV)
    for j in range(k):
        y += s["ys"][at[:, j]].double() * (w2[:, j] * okd[:, j])[:, None]
    out["y"] = y
    if s["grad"]:
        dy = s["dy"].double()
        dys = torch.zeros(t * k, h, dtype=torch.float64, device=DEV)
        dw = torch.zeros(t, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            dys[at[:, j]] = dy * (w2[:, j] * okd[:, j])[:, None]
            dw[:, j] = (dy * s["ys"][at[:, j]].double()).sum(1) * okd[:, j]
            dx += s["dxs"][at[:, j]].double() * okd[:, j, None]
        # softmax: d logit_i = p_i (g_i - sum_j p_j g_j), with g zero where no weight was taken
        gfull = np.zeros_like(lg)
        np.put_along_axis(gfull, order, dw.cpu().numpy() * ok, 1)
        out["dlogits"] = dev(prob * (gfull - (prob * gfull).sum(1, keepdims=True)))
        out["dys"], out["dweights"], out["dx"] = dys, dw, dx
    return out


def _exact_moment(x, word16, floor):
    """The nearest E4M3 neighbours of 64-bit values in blocks, and which of them the random bits take."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    high = blocks.abs().amax(1, keepdim=True)
    scale = torch.where(high > 0, 2.0 ** torch.ceil(torch.log2(high / 448.0)), torch.ones_like(high))
    mag = (blocks.abs() / scale).view(-1)[:n]
    step = 2.0 ** (torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    low = torch.floor(mag / step)
    up = (mag / step - low) + (word16.double() + 0.5) / 65536.0 >= 1.0
    val = ((low + up) * step).clamp(max=448.0)
    if floor:
        val = torch.where(mag > 0, val.clamp(min=2.0 ** -9), val)
    return torch.where(x < 0, -val, val), scale.view(-1)


def _exact_adamw(s):
    out = {k: [] for k in s["flat"] if k != "g"}
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.numel() % BLOCK))  # noqa: E731
    for i, p in enumerate(s["p"]):
        n = p.numel()
        g = s["g"][i].double() * s["grad_scale"].double()
        if s["state"] == "f32":
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            grow = lambda q, c: q.float().double() * c.double().repeat_interleave(BLOCK)[:n]  # noqa: E731
            m, v = grow(s["m"][i], s["ms"][i]), grow(s["v"][i], s["vs"][i]) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        new = p.double() - LR * DECAY * p.double() - LR * mhat / (vhat.sqrt() + EPS)
        out["p"].append(pad(new))
        if "w" in out:
            out["w"].append(pad(new))
        if s["state"] == "f32":
            out["m"].append(pad(m))
            out["v"].append(pad(v))
            continue
        word = _random_words(s["seed"], i, n)
        for name, x, bits in (("m", m, word & 0xFFFF), ("v", v.sqrt(), word >> 16)):
            val, scale = _exact_moment(x, bits, name == "v")
            out[name].append(pad(val))
            out[name + "s"].append(scale)
    return {k: torch.cat(v) for k, v in out.items()}
