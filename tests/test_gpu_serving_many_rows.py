"""Properties of the serving operators on the kernels for many rows: more than 48 rows
of a group for attention, more than 112 for weights.

Tolerances as in test_gpu_serving.py.
"""
import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import U, Pool, attend, check_attention, dev, gpu, rows_on_device  # noqa: F401 (gpu: fixture)
from test_gpu_serving_limits import check_both, check_weigh

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


@pytest.mark.parametrize("kv_len,counts,heads,causal", [([400, 290, 333], [120, 130, 1], 4, True), ([700, 290, 500], [60, 57, 60], 4, False)])
def test_sequences_that_share_pages(kv_len, counts, heads, causal):
    """A common beginning is read by all of them, and gets the weight of all: many rows add to it at once."""
    pool = Pool(kv_len, 2, 64, seed=13)
    for s in (1, 2):
        pool.table[s][:2] = pool.table[0][:2]
    check_both(pool, counts, heads, causal=causal)


@pytest.mark.parametrize("rows", [49, 113, 150])
def test_pages_past_32_bit_offsets(rows):
    """Pages more than 4 GiB into the pool."""
    torch = torch_mod()
    n, heads, dim, length = 70000, 8, 128, 200
    codes = [torch.zeros((n, heads, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((n, heads), device="cuda") for _ in range(2)]
    cache = tql.Exl3Kv8Cache(*codes, *scales, torch.zeros((n, heads, 64), device="cuda"))
    at = np.array([n - 1, n - 7, 3, n - 20])
    small = Pool([length], heads, dim, seed=rows)
    order = small.table[0][:4]
    for i in range(2):
        codes[i][at] = dev(small.codes[i][order])
        scales[i][at] = dev(small.scales[i][order])
    batch = tql.Exl3Kv8Batch(dev(at[None].astype(np.int32)), dev(np.array([length], dtype=np.int32)), dev(np.array([0, rows], dtype=np.int32)),
                             rows, rows)
    q = small.rng.standard_normal((rows, heads, dim)).astype(np.float16)
    got, lse = attend(type("P", (), {"cache": cache, "dim": dim}), [rows], q, heads, 0.1, 0.0, True, batch=batch)
    want = ref.attention(small.codes[0], small.scales[0], small.codes[1], small.scales[1], small.table, [length], [rows], q, 0.1, 0.0, True)
    check_attention(got, lse, want, dim, 0.0, length)
    lse = want[1].astype(np.float32)
    tql.exl3_kv8_weigh(cache, batch, rows_on_device(q.reshape(rows, -1), 0), heads, 0.1, dev(lse))
    w = cache._keep[4][at].cpu().numpy().transpose(1, 0, 2).reshape(heads, -1)
    add, bound = ref.weigh(small.codes[0], small.scales[0], small.table, [length], [rows], q, lse, 0.1, 0.0, True, 256)
    assert np.all(np.abs(w - add[0]) <= ((dim + 8) * U + 2.0 ** -20) * bound[0] + (rows + 2) * U * add[0])


@pytest.mark.parametrize("table,kv_len,start", [([[-1] * 3, [1 << 30] * 3], [100, 100], [0, 130, 260]),
                                                (None, [1000, -5], [0, 130, 260]), (None, [100, 100], [0, 261, 260]),
                                                (None, [100, 100], [-3, 0, 260])])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_bad_indexes_on_the_device(table, kv_len, start, cap):
    """Reported and not followed, by the kernels of 130 rows of a group; pages that no sequence has are untouched."""
    torch = torch_mod()
    pool = Pool([100, 100], 1, 128, seed=1)
    cache = pool.on_device()
    before = [t.clone() for t in pool.t]
    q = rows_on_device(np.ones((260, 128), dtype=np.float16), 0)
    batch = tql.Exl3Kv8Batch(dev(np.array(pool.table if table is None else table, dtype=np.int32)), dev(np.array(kv_len, dtype=np.int32)),
                             dev(np.array(start, dtype=np.int32)), 260, 130)
    out = torch.zeros((260, 128), dtype=torch.float16, device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
    for call in (lambda: tql.exl3_kv8_attention(cache, batch, q, 1, 1.0, out, ws, softcap=cap),
                 lambda: tql.exl3_kv8_weigh(cache, batch, q, 1, 1.0, torch.zeros((260, 1), device="cuda"), softcap=cap),
                 lambda: tql.exl3_kv8_append(cache, batch, q, q)):
        call()
        assert tql.exl3_get_device_status() == 10
        assert tql.exl3_get_device_status() == 0
    same = np.setdiff1d(np.arange(pool.n), pool.table.ravel())
    for t, b in zip(pool.t, before):
        assert torch.equal(t[same], b[same])
