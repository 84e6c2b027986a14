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


@pytest.mark.parametrize("rows,heads", [(200, 4), (600, 2), (20, 2)])
def test_weights_of_the_lse_that_attention_returned(rows, heads):
    """A row's weights add up to 1: exp(s - lse) with the lse of the same scores. Rows of one heavy token each, |s| about
    100: an error of s that the two kernels share cancels, and a relative one of only one of them, however small, would
    show in the mean over the rows, where the roundings of single scores (2^-24 of |s| a few times) average out. What stays
    is that of the constants log2 e and ln 2 (2^-26)."""
    torch = torch_mod()
    length, dim = 1500, 64
    pool = Pool([length] * 8, 1, dim, seed=rows, spread=0)
    pool.on_device()
    R = 8 * rows
    q = (12 * pool.rng.standard_normal((R, heads, dim))).astype(np.float16)
    _, lse = attend(pool, [rows] * 8, q, heads, 0.5, 0.0, False)
    pool.t[4].zero_()
    tql.exl3_kv8_weigh(pool.cache, pool.batch([rows] * 8), rows_on_device(q.reshape(R, -1), 0), heads, 0.5, dev(lse), causal=False)
    total = float(pool.t[4].double().sum()) / (R * heads)
    size = float(np.abs(lse).mean())
    assert size > 80
    assert abs(total - 1) <= 2.0 ** -25 * size + 4 * 2.0 ** -24 * size / (R * heads) ** 0.5 + 2.0 ** -22, (total - 1, size)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 50, 128])
def test_scores_of_heavy_tokens_have_no_common_error(dim, rows):
    """Sequences of one token whose key has the query's signs, so that partial sums grow evenly: the lse is the score, and
    weights for an exact lse are exp(its error). Roundings average out over 50000 scores; what all scores share stays within
    3/4 of a step of fp32, the constants log2 e and ln 2 (0.1) with it."""
    torch = torch_mod()
    n = max(50000 // rows, 400)
    g = torch.Generator(device="cuda").manual_seed(dim + rows)
    k = torch.randn((n, 1, 64, dim), generator=g, device="cuda").to(torch.float8_e4m3fn)
    key = k[:, 0, 0].double().repeat_interleave(rows, 0)
    q = (torch.randn((n * rows, dim), generator=g, device="cuda").abs() * key.sign()).half()
    ones = torch.ones((n, 1), device="cuda")
    cache = tql.Exl3Kv8Cache(k, k, ones, ones, torch.zeros((n, 1, 64), device="cuda"))
    batch = tql.Exl3Kv8Batch(torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                             torch.ones(n, dtype=torch.int32, device="cuda"),
                             torch.arange(n + 1, dtype=torch.int32, device="cuda") * rows, n * rows, rows)
    out, lse = torch.empty_like(q), torch.empty((n * rows, 1), device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
    tql.exl3_kv8_attention(cache, batch, q, 1, 1.0, out, ws, causal=False, lse=lse)
    s = (q.double() * key).sum(1)
    step = 2.0 ** -23 * float(s.sum())
    assert abs(float((lse[:, 0].double() - s).sum())) <= 0.75 * step
    exact = s.float()
    tql.exl3_kv8_weigh(cache, batch, q, 1, 1.0, exact, causal=False)
    got = cache._keep[4][:, 0, 0].double().view(n, 1) / rows
    want = torch.exp(s - exact.double()).view(n, rows).mean(1, keepdim=True)
    assert abs(float(((got - want) * rows).sum())) <= 0.75 * step
