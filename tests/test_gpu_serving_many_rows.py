"""Properties of the serving operators on the kernels for many rows: more than 48 rows
of a group for attention, more than 112 for weights.

Tolerances as in test_gpu_serving.py.
"""
import numpy as np
import pytest

import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import Pool, attend, dev, gpu, rows_on_device  # noqa: F401 (gpu: fixture)
from test_gpu_serving_limits import check_weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_len,counts,heads,kv_heads,causal,again", [
    ([8192], [128], 8, 8, True, 300),                      # 512 items of one step, one in the last tile
    ([8192], [113], 8, 8, False, 100),
    ([128 + i % 3 for i in range(400)], [128] * 400, 1, 1, True, 50),
    ([700] * 60, [25, 2] * 30, 5, 1, True, 50),            # one step of 25 rows of five heads
])
def test_items_of_one_step(kv_len, counts, heads, kv_heads, causal, again):
    """An item's steps are shared by two CTAs: with a single one the second CTA has none."""
    torch = torch_mod()
    pool = Pool(kv_len, kv_heads, 64, seed=len(kv_len))
    pool.on_device()
    R, scale = sum(counts), 0.125
    q = pool.rng.standard_normal((R, heads, 64)).astype(np.float16)
    lse = pool.rng.uniform(4, 6, (R, heads)).astype(np.float32)
    check_weigh(pool, counts, heads, q, lse, scale, 0.0, causal)
    qd, lsed, batch = rows_on_device(q.reshape(R, -1), 0), dev(lse), pool.batch(counts)
    first = None
    for i in range(again):
        pool.t[4].zero_()
        tql.exl3_kv8_weigh(pool.cache, batch, qd, heads, scale, lsed, causal=causal)
        if first is None:
            first = pool.t[4].clone()
        assert torch.equal(pool.t[4], first), i
