"""Sizes of grouped products that reach each kernel of the training-sized plans.
test_grouped_plan_cpu.py holds them to the kernels named here, so that a change
of the plan that sends one elsewhere does not pass unseen; test_gpu_grouped_tiles.py
runs them.

A case: pass, counts of the groups, rows of no group, N, K, and the plan it has
to take: tile, and for the weight gradient whether its groups are ordered by size."""
import numpy as np


def skewed(groups, rows, seed):
    """Counts of the groups that sum to `rows`: skewed, a few empty."""
    g = np.random.default_rng(seed)
    p = np.exp(1.0 * g.standard_normal(groups))
    p[::7] = 0 if groups > 7 else p[::7]
    return g.multinomial(rows, p / p.sum()).tolist()


EIGHT = [700, 3, 0, 1200, 257, 255, 400, 185]                 # 3000 rows
TILES = [
    ("forward", EIGHT, 0, 1032, 1032, "128x128", None),
    ("forward", EIGHT, 77, 1024, 1032, "128x128", None),      # rows of 64-byte pieces in both types
    ("forward", skewed(16, 39000, 1), 1000, 1024, 1032, "256x256", None),
    ("forward", skewed(16, 40000, 2), 0, 1048, 520, "256x256", None),
    ("forward", skewed(300, 40000, 3), 300, 512, 264, "128x128", None),   # five groups to a lane
    ("forward", skewed(700, 120000, 4), 0, 512, 264, "128x128", None),    # eleven: three passes of four
    ("dgrad", EIGHT, 0, 1032, 1032, "128x128", None),
    ("dgrad", EIGHT, 77, 1032, 1024, "128x128", None),
    ("dgrad", skewed(16, 39000, 5), 1000, 1032, 1024, "256x256", None),
    ("dgrad", skewed(16, 40000, 6), 0, 520, 1048, "256x256", None),
    ("dgrad", skewed(300, 40000, 7), 300, 264, 512, "256x256", None),
    ("wgrad", EIGHT, 77, 1032, 1032, "256x256", 0),
    ("wgrad", skewed(64, 3000, 8), 0, 512, 1032, "256x256", 1),
    ("wgrad", skewed(256, 20000, 9), 333, 512, 520, "256x256", 1),       # the most groups that are ordered
    ("wgrad", skewed(300, 40000, 10), 0, 512, 512, "256x256", 0),
    ("wgrad", skewed(100, 2500, 11), 20, 264, 520, "128x128", 1),
    ("wgrad", skewed(300, 3000, 12), 0, 264, 264, "128x128", 0),
]


def ident(case):
    p, counts, tail, N, K = case[:5]
    return "%s-%dgroups-%drows-%dx%d" % (p, len(counts), sum(counts) + tail, N, K)
