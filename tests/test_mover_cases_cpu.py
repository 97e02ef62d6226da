"""The sizes of mover_cases.py against the thresholds in the sources: a threshold
that moves past them does not leave their kernels untested unseen."""
import os
import re

import mover_cases

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_bf16_projection_amd",
                    "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _number(text, pattern):
    found = re.findall(pattern, text)
    assert len(found) == 1, pattern
    return eval(found[0], {"__builtins__": {}})


def test_routes_are_beyond_a_wave_a_token_and_use_every_register_count():
    wide = _number(_source("dpg_route.hip"), r"kWideTokens = ([0-9]+);")
    assert all(T > wide for T, _, _ in mover_cases.ROUTES)
    assert {next(i for i, n in enumerate((64, 128, 256, 512)) if E <= n) for _, E, _ in mover_cases.ROUTES} == {0, 1, 2, 3}
    assert any(k > 16 for _, _, k in mover_cases.ROUTES)


def test_streamed_rows_are_streamed():
    text = _source("dpg_route.hip")
    least = _number(text, r"return R \* H >= \(int64_t\)\(([0-9 <]+)\) / elt")
    piece = _number(text, r"\(uint64_t\)\(H \* elt\)\) & ([0-9]+)\) == 0;") + 1
    for T, k, H, pad in mover_cases.STREAMED:
        for elt in (2, 4):
            assert T * k * H * elt >= least and H * elt % piece == 0 and (H + pad) * elt % piece == 0


def test_the_adamw_call_is_not_one_of_few_elements():
    few = re.findall(r"kFewElements\[2\] = \{([0-9 <]+), ([0-9 <]+)\}", _source("dpg_adamw.hip"))
    assert len(few) == 1 and all(sum(mover_cases.ADAMW) > eval(v, {"__builtins__": {}}) for v in few[0])
    steps = _number(_source("adamw_kernel.h"), r"kAdamwSteps = ([0-9]+);")
    chunk = 4 * steps * 256
    assert {n % chunk for n in mover_cases.ADAMW} >= {0, 1, chunk - 1}
