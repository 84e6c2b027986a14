"""The serving operators where a launch's fixed sizes end: more sequences than one
launch's plan holds, page tables whose keys pass one CTA's shared memory, more
heads to a key/value head than a step's columns, and of the logits many rows,
long histories, more entries or tokens than are listed.

Tolerances as in test_gpu_serving.py.
"""
import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import U, Pool, attend, check_attention, dev, gpu, rows_on_device  # noqa: F401 (gpu: fixture)

pytestmark = pytest.mark.gpu


def check_weigh(pool, counts, heads, q, lse, scale, cap, causal):
    """Adds the weights, and compares them page by page (a page may be in several sequences)."""
    R, dim, kv_len = sum(counts), pool.dim, pool.kv_len
    tql.exl3_kv8_weigh(pool.cache, pool.batch(counts), rows_on_device(q.reshape(R, -1), 8), heads, scale, dev(lse),
                       softcap=cap, causal=causal)
    torch_mod().cuda.synchronize()
    got = pool.t[4].cpu().numpy()
    add, bound = ref.weigh(pool.codes[0], pool.scales[0], pool.table, kv_len, counts, q, lse, scale, cap, causal,
                           64 * pool.max_pages)
    want, tol = pool.weight.astype(np.float64), np.zeros(pool.weight.shape)
    terms = max(counts) * (heads // pool.heads)
    for s in range(len(kv_len)):
        for b in range(pool.max_pages):
            page = pool.table[s][b]
            a, e = add[s, :, 64 * b:64 * b + 64], bound[s, :, 64 * b:64 * b + 64]
            want[page] += a
            tol[page] += ((dim + 8) * U + 2.0 ** -20) * e + cap * 2.0 ** -21 * a + (terms + 2) * U * (a + want[page]) * (a != 0)
    assert np.all(np.abs(got - want) <= tol)


def check_both(pool, counts, heads, cap=0.0, causal=True):
    pool.on_device()
    q = (2 * pool.rng.standard_normal((sum(counts), heads, pool.dim))).astype(np.float16)
    scale = pool.dim ** -0.5
    got, lse = attend(pool, counts, q, heads, scale, cap, causal)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, pool.kv_len, counts, q,
                         scale, cap, causal)
    check_attention(got, lse, want, pool.dim, cap, max(pool.kv_len))
    check_weigh(pool, counts, heads, q, want[1].astype(np.float32), scale, cap, causal)


@pytest.mark.parametrize("most", [1, 19, 40, 60])
def test_more_sequences_than_a_launch_holds(most):
    rng = np.random.default_rng(most)
    kv_len = rng.integers(0, 100, 1100)
    counts = np.minimum(rng.integers(0, min(most, 19) + 1, 1100), kv_len)
    counts[0] = min(most, kv_len[0])
    kv_len[1030], counts[1030] = 77, most  # in every launch
    check_both(Pool(kv_len, 1, 64, seed=most), counts.tolist(), 2)


@pytest.mark.parametrize("kv_len,counts,heads,dim,cap,causal", [
    ([130, 700, 9], [5, 13, 9], 8, 64, 0.0, True),        # 20, 52 and 36 rows of a group of four
    ([3000, 64], [12, 1], 10, 128, 20.0, True),           # 60 rows, segments over several CTAs
    ([500, 501], [24, 23], 4, 64, 0.0, False),            # 48: the most that the tiles of 16 take
    ([500, 501], [25, 1], 4, 128, 0.0, True),             # 50
    ([500, 501], [32, 31], 4, 64, 0.0, False),            # 64
    ([500, 501], [1, 1], 130, 128, 0.0, True),            # 65
    ([900], [56], 4, 128, 0.0, True), ([900], [57], 4, 64, 0.0, True),  # 112 and 114, where weights change over
    ([40, 200], [0, 20], 2, 128, 0.0, True),
])
def test_rows_around_the_tiles_of_sixteen(kv_len, counts, heads, dim, cap, causal):
    check_both(Pool(kv_len, 2, dim, seed=sum(kv_len) + heads), counts, heads, cap, causal)


def test_append_to_more_sequences_than_a_launch_holds():
    pool = Pool([65] * 1100, 1, 64, seed=8, spread=1)
    pool.on_device()
    x = pool.rng.standard_normal((1100, 1, 64)).astype(np.float16)
    want = [(c.copy(), s.copy()) for c, s in zip(pool.codes, pool.scales)]
    for c, s in want:
        ref.append(c, s, pool.table, pool.kv_len, [1] * 1100, x)
    xd = rows_on_device(x.reshape(1100, -1), 0)
    tql.exl3_kv8_append(pool.cache, pool.batch([1] * 1100), xd, xd)
    for i in range(2):
        assert np.array_equal(pool.t[2 + i].cpu().numpy(), want[i][1])
        got = pool.t[i].cpu().numpy()
        assert np.array_equal(np.where(got & 0x7F, got, 0), np.where(want[i][0] & 0x7F, want[i][0], 0))


@pytest.mark.parametrize("rows,heads,cap", [(2, 130, 0.0), (3, 256, 30.0), (1, 200, 0.0)])
def test_more_heads_of_a_group_than_a_step_has_columns(rows, heads, cap):
    check_both(Pool([290, 70], 1, 64, seed=heads), [rows, rows], heads, cap)


@pytest.mark.parametrize("counts", [[1, 2, 1], [20, 30, 1]])
def test_sequences_that_share_pages(counts):
    """A common beginning is read by all of them, and gets the weight of all."""
    pool = Pool([400, 290, 333], 2, 64, seed=12)
    for s in (1, 2):
        pool.table[s][:4] = pool.table[0][:4]  # whole blocks in front of every sequence's new rows
    check_both(pool, counts, 4)


@pytest.mark.parametrize("kv_len,max_pages,budget,recent", [
    ([900, 3000], 800, 500, 100),        # keys of 51200 tokens: two CTAs
    ([130, 0], 2500, 64, 0),             # four
    ([30000], 6000, 1000, 10),           # eight
])
def test_evict_with_long_page_tables(kv_len, max_pages, budget, recent):
    torch = torch_mod()
    blocks = -(-budget // 64)
    pool = Pool(kv_len, 1, 64, seed=max_pages, extra=len(kv_len) * blocks)
    pool.weight = np.where(pool.rng.random(pool.weight.shape) < 0.5, np.float32(0.25), pool.weight)  # many ties
    pool.on_device()
    free = np.setdiff1d(np.arange(pool.n), pool.table.ravel())
    dst = free[:len(kv_len) * blocks].reshape(len(kv_len), blocks).astype(np.int32)
    table = np.full((len(kv_len), max_pages), -1, dtype=np.int32)
    table[:, :pool.max_pages] = pool.table
    kept = torch.full((len(kv_len), 1, budget), -7, dtype=torch.int32, device="cuda")
    new_len = torch.full((len(kv_len),), -7, dtype=torch.int32, device="cuda")
    tql.exl3_kv8_evict(pool.cache, tql.Exl3Kv8Batch(dev(table), dev(np.array(kv_len, dtype=np.int32))), dev(dst), budget,
                       recent, kept, new_len)
    assert new_len.tolist() == [min(budget, x) for x in kv_len]
    weight = pool.t[4].cpu().numpy()
    for s, length in enumerate(kv_len):
        keep = ref.evict_choice(pool.weight[pool.table[s], 0].ravel(), length, budget, recent)
        assert kept[s, 0].tolist() == keep + [-1] * (budget - len(keep))
        at = np.array(keep, dtype=np.int64)
        assert np.array_equal(weight[dst[s], 0].ravel()[:at.size], pool.weight[pool.table[s][at // 64], 0, at % 64])


def test_evict_of_more_keys_than_a_cluster_holds():
    """400000 tokens: eight CTAs hold the keys of 360448 in shared memory, the rest are read again."""
    torch = torch_mod()
    length, budget, recent = 400000, 3000, 17
    blocks, n = -(-budget // 64), -(-length // 64)
    rng = np.random.default_rng(3)
    pages = n + blocks
    cache = tql.Exl3Kv8Cache(*[torch.zeros((pages, 1, 64, 64), dtype=torch.uint8, device="cuda") for _ in range(2)],
                             *[torch.ones((pages, 1), device="cuda") for _ in range(2)], dev(np.zeros((pages, 1, 64), np.float32)))
    weight = rng.integers(0, 5000, (pages, 1, 64)).astype(np.float32)
    cache._keep[4].copy_(dev(weight))
    order = rng.permutation(pages).astype(np.int32)
    table, dst = order[None, :n], order[None, n:]
    kept = torch.empty((1, 1, budget), dtype=torch.int32, device="cuda")
    new_len = torch.empty((1,), dtype=torch.int32, device="cuda")
    tql.exl3_kv8_evict(cache, tql.Exl3Kv8Batch(dev(table), dev(np.array([length], dtype=np.int32))), dev(dst), budget, recent,
                       kept, new_len)
    assert kept[0, 0].tolist() == ref.evict_choice(weight[table[0], 0].ravel(), length, budget, recent)
    assert new_len.item() == budget


def logits_case(rng, M, n, hist, bias, masked):
    """Runs both forms of output and compares with the same fp32 operations one by one."""
    torch = torch_mod()
    ld = -(-n // 4) * 4
    logits = (3 * rng.standard_normal((M, ld))).astype(np.float32)
    gen = np.array([len(h) // 3 for h in hist], dtype=np.int32)
    rep, pres, freq = (rng.uniform(a, b, M).astype(np.float32) for a, b in ((0.8, 1.6), (-0.5, 1.0), (-0.1, 0.5)))
    kw = dict(history=dev(np.concatenate(hist).astype(np.int32)), generated_from=dev(gen),
              history_start=dev(np.cumsum([0] + [len(h) for h in hist]).astype(np.int32)),
              repetition=dev(rep), presence=dev(pres), frequency=dev(freq),
              bias_id=dev(np.array([t for b in bias for t, _ in b], dtype=np.int32)),
              bias_value=dev(np.array([v for b in bias for _, v in b], dtype=np.float32)),
              bias_start=dev(np.cumsum([0] + [len(b) for b in bias]).astype(np.int32)))
    allow = None
    if masked:
        allow = np.zeros((M, -(-n // 32) * 32), dtype=bool)
        allow[:, :n] = rng.random((M, n)) < 0.7
        kw |= dict(allowed=dev(np.packbits(allow, axis=1, bitorder="little").view(np.uint32).view(np.int32)))
    x = dev(logits)
    out = torch.full((M, ld), 9.0, device="cuda")
    am = torch.full((M,), -9, dtype=torch.int32, device="cuda")
    tql.exl3_logits_adjust(x, n, out, am, **kw)
    got = out.cpu().numpy()
    for m in range(M):
        want, pick = ref.adjust(logits[m, :n], hist[m], gen[m], rep[m], pres[m], freq[m], bias[m],
                                allow[m, :n] if masked else None, np.float32)
        assert np.array_equal(got[m, :n], want)
        assert int(am[m]) == pick


def some_biases(rng, n, count):
    return [(int(t), float(np.float32(rng.standard_normal()))) for t in rng.integers(-1, n + 1, count)]


@pytest.mark.parametrize("M,n", [(12, 300001), (33, 5000), (16, 140000), (150, 129)])
@pytest.mark.parametrize("masked", [False, True])
def test_logits_of_many_rows(M, n, masked):
    rng = np.random.default_rng([M, n])
    hist = [rng.integers(-2, n + 2, int(rng.integers(0, 3000))) for _ in range(M)]
    bias = [some_biases(rng, n, 40) for _ in range(M)]
    bias[0] += [(5, 1.0), (5, -0.25), (n - 1, 3.0), (5, 0.125)]  # duplicates
    bias[1] = []
    hist[2] = hist[2][:0]
    logits_case(rng, M, n, hist, bias, masked)


@pytest.mark.parametrize("M", [2, 11])
@pytest.mark.parametrize("n", [3000, 200003])
def test_logits_with_long_histories(M, n):
    """Past 14 bits of count, past the list of a CTA's entries, past the list of tokens with a word."""
    rng = np.random.default_rng([M, n, 1])
    hist = [rng.integers(0, n, 700) for _ in range(M)]
    hist[0] = np.concatenate([np.full(20000, 11), rng.integers(0, n, 20000)])   # 20000 times the same token
    hist[1] = np.concatenate([rng.integers(0, 128, 9000), np.arange(min(n, 60000))])[:16383]  # one CTA's tokens
    hist[M - 1] = rng.permutation(np.concatenate([hist[M - 1], np.arange(n), rng.integers(0, n, 5000)]))  # every token
    logits_case(rng, M, n, hist, [some_biases(rng, n, 200) for _ in range(M)], True)
