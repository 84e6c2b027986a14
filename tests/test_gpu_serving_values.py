"""The serving operators on values of unusual size: small and missing value blocks,
caps far above the scores, weights spread over many tokens, scales of either sign.

Tolerances as in test_gpu_serving.py, or stated at the test.
"""
import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import Pool, attend, check_attention, dev, gpu, rows_on_device  # noqa: F401 (gpu: fixture)

pytestmark = pytest.mark.gpu


def check_pool(pool, counts, heads, scale=None, cap=0.0, causal=True):
    pool.on_device()
    scale = pool.dim ** -0.5 if scale is None else scale
    q = (2 * pool.rng.standard_normal((sum(counts), heads, pool.dim))).astype(np.float16)
    got, lse = attend(pool, counts, q, heads, scale, cap, causal)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, pool.kv_len, counts, q,
                         scale, cap, causal)
    check_attention(got, lse, want, pool.dim, cap, max(pool.kv_len))
    return got


def small_values(pool, blocks, exponent):
    """The sequences' value blocks `blocks` get the scale 2^exponent, or all-zero codes and the scale of zeros (None)."""
    for s, length in enumerate(pool.kv_len):
        for b in range(-(-length // 64)):
            if blocks != "all" and b != -(-length // 64) - 1:
                continue
            page = pool.table[s][b]
            pool.scales[1][page] = 2.0 ** (-32 if exponent is None else exponent)
            if exponent is None:
                used = min(64, length - 64 * b)
                pool.codes[1][page, :, :used] = 0


@pytest.mark.parametrize("kv_len,counts", [([65], [1]), ([65], [65]), ([1], [60]), ([129], [50]), ([777], [64]), ([777, 300], [130, 128]),
                                           ([64, 20000], [50, 49])])
@pytest.mark.parametrize("blocks", ["all", "last"])
@pytest.mark.parametrize("exponent", [None, -32, -17, -16])
def test_small_values_in_blocks(kv_len, counts, blocks, exponent):
    """Odd numbers of blocks: the last one's neighbour in a 128-token unit does not exist."""
    pool = Pool(kv_len, 1, 64, seed=sum(kv_len) + counts[0])
    small_values(pool, blocks, exponent)
    got = check_pool(pool, counts, 1)
    if exponent is None and blocks == "all":
        assert np.all(got == 0)
