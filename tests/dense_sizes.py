"""Sizes at which w4a16_dense takes each of its kernels, widths and splits (test
infrastructure): found by asking it, so that no width goes untested on another
device or behind another estimate."""

import functools
import itertools

import torch

from w4a16_int4_moe_gb300 import ops

CLUSTERS, PAIRS = 1, 2   # DenseInfo.kernel
SHAPES = ([(PAIRS, rows, 1) for rows in range(64, 257, 32)]
          + [(CLUSTERS, rows, split) for rows in range(64, 257, 64) for split in (1, 2, 4, 8)])
KINDS = [(gated, dtype) for gated in (False, True) for dtype in (torch.bfloat16, torch.float32)]

TOKENS = (33, 64, 100, 129, 200, 257, 300, 400, 520, 577, 700, 1025, 1300, 2050, 2500, 3000, 4099,
          5000, 8192)
ROWS = (8, 130, 300, 514, 1000, 1542, 2002, 2600, 3222, 3326, 3906, 4096, 4802, 5002, 6200, 7168,
        9728, 12290, 18432, 36864)
COLUMNS = (64, 72, 264, 512, 1032, 2088, 4104, 7168, 18432)


@functools.lru_cache(maxsize=None)
def sizes(at_once=None):
    """{(kernel, tile_rows, split), gated, dtype: (tokens, n, k)}: of those where more than two
    accumulators follow one another, and pairs go over more than two tiles, the
    one with the least work; else the one with the least work."""
    found = {}
    pairs = at_once[0] if at_once else torch.cuda.get_device_properties(0).multi_processor_count // 2
    for tokens, n, k, (gated, dtype) in itertools.product(TOKENS, ROWS, COLUMNS, KINDS):
        i = ops.w4a16_dense_info(tokens, n, k, gated, dtype, at_once)
        tiles = -(-tokens // 256) * -(-n // i.tile_rows)
        far = k > 2 * i.split * i.run and (i.kernel == CLUSTERS or tiles > 2 * pairs)
        key, cost = ((i.kernel, i.tile_rows, i.split), gated, dtype), (not far, tokens * n * k)
        if key not in found or cost < found[key][0]:
            found[key] = cost, (tokens, n, k)
    return {key: size for key, (_, size) in found.items()}
