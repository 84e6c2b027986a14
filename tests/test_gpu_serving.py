"""Serving operators on the GPU against plain 64-bit implementations
(serving_ref.py): the 8-bit paged cache, attention over it, accumulated
attention weight, eviction, and the adjustment of logits.

Tolerances, from the operators' own roundings:
  - append, evict: none (codes, scales, positions and weights are equal);
  - lse: fp32 products and sums, (D + 8) ulp of the sum of magnitudes, a few ulp
    of the result, softcap's tanh to 2^-21 of the cap;
  - attention: fp16 result (2^-11) and fp16 probabilities (2^-11 of the sum of
    p |v|, and 2^-25 absolute for each token below fp16's range), the fp32 score
    error on top;
  - weights: each term exp(s - lse) to the error of s; a sum of n terms to n ulp;
  - logits: equal to the same fp32 operations done one by one.
"""
import ctypes

import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # fp32 unit roundoff


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tql.build()
    torch.cuda.set_device(0)
    tql.exl3_init(0)
    tql.exl3_get_device_status()
    yield
    assert tql.exl3_get_device_status() == 0


def dev(a):
    return torch_mod().from_numpy(np.ascontiguousarray(a)).cuda()


def rows_on_device(x, pad):
    """R x width fp16 rows inside a wider matrix (row stride width + pad)."""
    torch = torch_mod()
    m = torch.zeros((max(1, x.shape[0]), x.shape[1] + pad), dtype=torch.float16, device="cuda")
    m[:x.shape[0], :x.shape[1]] = dev(x)
    return m[:x.shape[0], :x.shape[1]]


class Pool:
    """A cache with randomly placed pages whose unused slots hold NaN codes."""

    def __init__(self, kv_len, heads, dim, seed, spread=3, gain=1.0, extra=3):
        self.rng = np.random.default_rng([seed, 7])
        rng = self.rng
        self.kv_len = list(kv_len)
        self.max_pages = max(1, max(-(-x // 64) for x in kv_len)) + 1
        n = len(kv_len) * self.max_pages + extra
        self.n, self.heads, self.dim = n, heads, dim
        self.table = rng.permutation(n)[:len(kv_len) * self.max_pages].reshape(len(kv_len), -1).astype(np.int32)
        self.codes, self.scales = [], []
        for _ in range(2):
            x = rng.standard_normal((n, heads, 64, dim)) * gain * 2.0 ** rng.integers(-spread, spread + 1, (n, heads, 1, 1))
            e = np.array([[ref.block_exponent(b) for b in page] for page in x])
            c = ref.nearest_code(x * 2.0 ** -e[:, :, None, None].astype(np.float64))
            self.codes.append(c)
            self.scales.append((2.0 ** e).astype(np.float32))
        used = np.zeros((n, 64), dtype=bool)
        for s, length in enumerate(self.kv_len):
            for b in range(self.max_pages):
                used[self.table[s][b], :max(0, min(64, length - 64 * b))] = True
        for c in self.codes:  # what lies past a length is never used
            c[~used[:, None, :].repeat(heads, 1)] = 0x7F
        self.weight = rng.random((n, heads, 64)).astype(np.float32)

    def on_device(self):
        self.t = [dev(c) for c in self.codes] + [dev(s) for s in self.scales] + [dev(self.weight)]
        self.cache = tql.Exl3Kv8Cache(*self.t)
        return self.cache

    def batch(self, counts):
        q = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        return tql.Exl3Kv8Batch(dev(self.table), dev(np.array(self.kv_len, dtype=np.int32)), dev(q), int(q[-1]),
                                max(counts, default=0))


ATTENTION = [
    # kv_len, rows, heads, kv_heads, dim, cap, causal
    ([1], [1], 1, 1, 64, 0.0, True),
    ([64], [1], 8, 1, 128, 0.0, True),
    ([63, 65, 128, 1], [1, 1, 1, 1], 8, 8, 128, 0.0, True),
    ([777], [1], 32, 8, 128, 0.0, True),
    ([300, 0, 17, 1000], [1, 1, 1, 1], 10, 2, 64, 25.0, True),          # an empty sequence
    ([200, 5], [4, 3], 15, 3, 128, 0.0, True),                          # speculated rows, five heads a group
    ([200, 5], [4, 3], 12, 3, 128, 50.0, False),
    ([2, 70], [5, 3], 4, 2, 64, 0.0, True),                             # rows in front of the cache see nothing
    ([130, 40], [16, 1], 1, 1, 128, 0.0, True),
    ([517], [1], 17, 1, 128, 0.0, True),                                # more heads to a key head than a 16-row tile
    ([290], [1], 96, 1, 64, 30.0, True),
    ([150, 333, 90], [17, 65, 90], 2, 1, 64, 0.0, True),                # chunks
    ([333], [129], 5, 1, 128, 0.0, True),
    ([400, 64], [257, 0], 4, 2, 128, 20.0, True),                       # a sequence without rows
    ([260], [200], 3, 3, 64, 0.0, False),
    ([3000], [2], 8, 2, 128, 0.0, True),
    ([600, 599, 33, 2, 1], [130, 1, 30, 2, 1], 8, 2, 128, 0.0, True),   # chunks and single tokens together
    ([450], [450], 2, 2, 128, 15.0, True),
]


def attend(pool, counts, q, heads, scale, cap, causal, batch=None, stream=None):
    torch = torch_mod()
    cache, batch = pool.cache, batch or pool.batch(counts)
    R = sum(counts)
    qd = rows_on_device(q.reshape(R, -1), 24)
    out = torch.full((max(1, R), heads * pool.dim + 8), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((max(1, R), heads), float("nan"), device="cuda")
    n = tql.exl3_kv8_attention_workspace_bytes(cache, batch, heads)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    tql.exl3_kv8_attention(cache, batch, qd, heads, scale, out[:, :heads * pool.dim], ws, softcap=cap, causal=causal,
                           lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, heads * pool.dim:]).all()  # past a row's width nothing is written
    return out[:R, :heads * pool.dim].float().cpu().numpy().reshape(R, heads, pool.dim), lse[:R].cpu().numpy()


def check_attention(got, lse, want, dim, cap, lengths):
    out, wlse, mag, sabs = want
    seen = np.isfinite(wlse)
    assert np.array_equal(np.isneginf(lse), ~seen)
    s_err = (dim + 8) * U * sabs + cap * 2.0 ** -21 + 2.0 ** -21 * (1 + np.abs(np.where(seen, wlse, 0)) + np.minimum(sabs, cap or np.inf))
    assert np.all(np.abs(lse[seen] - wlse[seen]) <= s_err[seen])
    vmax = np.abs(mag).max(initial=0.0) if mag.size else 0.0
    tol = 2.0 ** -11 * np.abs(out) + (2.0 ** -11 + 2 * s_err[:, :, None]) * mag + lengths * 2.0 ** -25 * vmax + 2.0 ** -25
    assert np.all(np.abs(got - out) <= tol), float((np.abs(got - out) - tol).max())
    assert np.all(got[~seen] == 0)


@pytest.mark.parametrize("kv_len,counts,heads,kv_heads,dim,cap,causal", ATTENTION)
def test_attention(kv_len, counts, heads, kv_heads, dim, cap, causal):
    pool = Pool(kv_len, kv_heads, dim, seed=len(kv_len) * 1000 + heads)
    pool.on_device()
    q = (2 * pool.rng.standard_normal((sum(counts), heads, dim))).astype(np.float16)
    scale = dim ** -0.5
    got, lse = attend(pool, counts, q, heads, scale, cap, causal)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts, q,
                         scale, cap, causal)
    check_attention(got, lse, want, dim, cap, max(kv_len))


@pytest.mark.parametrize("counts", [[1], [40]])
def test_attention_wide_value_scales(counts):
    """Blocks whose values differ by 2^16 in size: the small ones still count where they get the weight."""
    pool = Pool([500], 1, 128, seed=5, spread=8)
    pool.codes[0][:] = np.where(pool.codes[0] == 0x7F, 0x7F, pool.codes[0])
    pool.on_device()
    q = (4 * pool.rng.standard_normal((sum(counts), 4, 128))).astype(np.float16)
    got, lse = attend(pool, counts, q, 4, 0.01, 0.0, True)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, [500], counts, q,
                         0.01, 0.0, True)
    check_attention(got, lse, want, 128, 0.0, 500)


@pytest.mark.parametrize("counts", [[1, 1, 1], [33, 1, 70]])
def test_attention_sharp_scores(counts):
    """Scores of several hundred: one token takes all the weight, the others underflow."""
    kv_len = [300, 90, 180]
    pool = Pool(kv_len, 2, 64, seed=9, spread=1)
    pool.on_device()
    q = (30 * pool.rng.standard_normal((sum(counts), 4, 64))).astype(np.float16)
    got, lse = attend(pool, counts, q, 4, 1.0, 0.0, True)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts, q,
                         1.0, 0.0, True)
    check_attention(got, lse, want, 64, 0.0, max(kv_len))


@pytest.mark.parametrize("counts", [[1, 1], [60, 30]])
def test_attention_nan_and_inf_queries_stay_in_their_rows(counts):
    pool = Pool([150, 95], 1, 128, seed=11)
    pool.on_device()
    R = sum(counts)
    q = pool.rng.standard_normal((R, 2, 128)).astype(np.float16)
    clean, _ = attend(pool, counts, q, 2, 0.1, 0.0, True)
    q[R - 1, 1, 5] = np.nan
    q[0, 0, 3] = np.inf
    got, _ = attend(pool, counts, q, 2, 0.1, 0.0, True)
    assert np.isnan(got[R - 1, 1]).all() and np.isnan(got[0, 0]).any()
    rest = np.ones((R, 2), dtype=bool)
    rest[R - 1, 1] = rest[0, 0] = False
    assert np.array_equal(got[rest], clean[rest])


@pytest.mark.parametrize("counts", [[1, 1], [20, 70]])
def test_attention_same_result_every_time_and_on_another_stream(counts):
    torch = torch_mod()
    pool = Pool([700, 333], 2, 128, seed=3)
    pool.on_device()
    q = pool.rng.standard_normal((sum(counts), 10, 128)).astype(np.float16)
    a = attend(pool, counts, q, 10, 0.1, 0.0, True)
    b = attend(pool, counts, q, 10, 0.1, 0.0, True, stream=torch.cuda.Stream())
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_attention_lengths_change_under_one_graph():
    """A captured call serves other lengths, pages and rows within its bounds."""
    torch = torch_mod()
    pool = Pool([500, 64], 2, 64, seed=21)
    cache = pool.on_device()
    batch = pool.batch([2, 1])
    q = pool.rng.standard_normal((3, 4, 64)).astype(np.float16)
    qd = rows_on_device(q.reshape(3, -1), 0)
    out = torch.zeros((3, 256), dtype=torch.float16, device="cuda")
    lse = torch.zeros((3, 4), device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 4), dtype=torch.uint8, device="cuda")

    def call():
        tql.exl3_kv8_attention(cache, batch, qd, 4, 0.2, out, ws, lse=lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for kv_len, counts in (([500, 64], [2, 1]), ([77, 3], [1, 2]), ([1, 0], [2, 1])):
        batch._keep[1].copy_(dev(np.array(kv_len, dtype=np.int32)))
        batch._keep[2].copy_(dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts,
                             q, 0.2, 0.0, True)
        check_attention(out.float().cpu().numpy().reshape(3, 4, 64), lse.cpu().numpy(), want, 64, 0.0, 500)


@pytest.mark.parametrize("rows", [1, 40])
def test_cache_past_32_bit_offsets(rows):
    """Pages more than 4 GiB into the pool."""
    torch = torch_mod()
    n, heads, dim = 70000, 8, 128
    codes = [torch.zeros((n, heads, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((n, heads), device="cuda") for _ in range(2)]
    cache = tql.Exl3Kv8Cache(*codes, *scales, torch.zeros((n, heads, 64), device="cuda"))
    length = 100
    table = np.array([[n - 1, n - 7]], dtype=np.int32)
    batch = tql.Exl3Kv8Batch(dev(table), dev(np.array([length], dtype=np.int32)), dev(np.array([0, length], dtype=np.int32)),
                             length, length)
    rng = np.random.default_rng(4)
    kv = rng.standard_normal((2, length, heads, dim)).astype(np.float16)
    tql.exl3_kv8_append(cache, batch, rows_on_device(kv[0].reshape(length, -1), 0), rows_on_device(kv[1].reshape(length, -1), 16))
    at = np.array([n - 1, n - 7])
    small = [codes[i][at].cpu().numpy() for i in range(2)]
    s = [scales[i][at].cpu().numpy() for i in range(2)]
    q = rng.standard_normal((rows, 8, dim)).astype(np.float16)
    b2 = tql.Exl3Kv8Batch(dev(table), dev(np.array([length], dtype=np.int32)), dev(np.array([0, rows], dtype=np.int32)), rows, rows)
    pool = type("P", (), {"cache": cache, "dim": dim})
    got, lse = attend(pool, [rows], q, 8, 0.1, 0.0, True, batch=b2)
    want = ref.attention(small[0], s[0], small[1], s[1], [[0, 1]], [length], [rows], q, 0.1, 0.0, True)
    check_attention(got, lse, want, dim, 0.0, length)
    tql.exl3_kv8_weigh(cache, b2, rows_on_device(q.reshape(rows, -1), 0), 8, 0.1, dev(lse))
    w = cache._keep[4][at].cpu().numpy().transpose(1, 0, 2).reshape(8, -1)
    add, bound = ref.weigh(small[0], s[0], [[0, 1]], [length], [rows], q, lse, 0.1, 0.0, True, 128)
    assert np.all(np.abs(w - add[0]) <= 1e-4 * add[0] + 1e-12)


# --------------------------------------------------------------------------- append


@pytest.mark.parametrize("kv_len,counts,kv_heads,dim", [
    ([1], [1], 1, 64), ([64], [1], 2, 128), ([65], [1], 2, 128), ([200, 3, 64, 129], [1, 1, 1, 1], 3, 64),
    ([300, 130, 70], [5, 130, 0], 2, 128), ([1000], [777], 1, 128), ([40, 128], [40, 64], 4, 64)])
@pytest.mark.parametrize("gain", [1.0, 300.0, 2.0 ** -13])
def test_append_equals_the_definition(kv_len, counts, kv_heads, dim, gain):
    torch = torch_mod()
    before = [a - b for a, b in zip(kv_len, counts)]
    pool = Pool(kv_len, kv_heads, dim, seed=sum(kv_len) + kv_heads, spread=1)
    pool.on_device()
    x = [(gain * pool.rng.standard_normal((sum(counts), kv_heads, dim)) * 2.0 ** pool.rng.integers(-4, 5, (sum(counts), 1, 1)))
         .clip(-65504, 65504).astype(np.float16) for _ in range(2)]
    x[0][0, 0, :4] = [0.0, -0.0, 6e-8, -6e-8]
    x[0][-1, -1, 0] = 65504.0
    want = [(c.copy(), s.copy()) for c, s in zip(pool.codes, pool.scales)]
    for (c, s), r in zip(want, x):
        ref.append(c, s, pool.table, kv_len, counts, r)
    tql.exl3_kv8_append(pool.cache, pool.batch(counts), rows_on_device(x[0].reshape(sum(counts), -1), 8),
                        rows_on_device(x[1].reshape(sum(counts), -1), 0))
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(pool.t[2 + i].cpu().numpy(), want[i][1])
        got = pool.t[i].cpu().numpy()
        zero = (got & 0x7F == 0) & (want[i][0] & 0x7F == 0)  # a value that became 0 has either sign
        assert np.array_equal(np.where(zero, 0, got), np.where(zero, 0, want[i][0]))
    w = pool.weight.copy()
    for s, length in enumerate(kv_len):
        for t in range(before[s], length):
            w[pool.table[s][t // 64], :, t % 64] = 0
    assert np.array_equal(pool.t[4].cpu().numpy(), w)


def test_append_infinities_and_nan():
    pool = Pool([70], 1, 64, seed=2)
    pool.on_device()
    x = pool.rng.standard_normal((70, 1, 64)).astype(np.float16)
    x[3, 0, 1], x[4, 0, 2], x[66, 0, 5] = np.inf, -np.inf, np.nan
    x[69] = 0
    want = [(c.copy(), s.copy()) for c, s in zip(pool.codes, pool.scales)]
    for c, s in want:
        ref.append(c, s, pool.table, [70], [70], x)
    tql.exl3_kv8_append(pool.cache, pool.batch([70]), rows_on_device(x.reshape(70, -1), 0), rows_on_device(x.reshape(70, -1), 0))
    for i in range(2):
        got = pool.t[i].cpu().numpy()
        assert np.array_equal(pool.t[2 + i].cpu().numpy(), want[i][1])
        nan = (got & 0x7F) == 0x7F
        assert np.array_equal(nan, (want[i][0] & 0x7F) == 0x7F) and np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want[i][0]))


def test_append_token_by_token_equals_the_definition():
    """A block filled one token at a time, its scale growing on the way."""
    pool = Pool([0], 2, 64, seed=6)
    pool.max_pages, pool.table = 2, np.array([[1, 2]], dtype=np.int32)
    pool.on_device()
    want = [(c.copy(), s.copy()) for c, s in zip(pool.codes, pool.scales)]
    for t in range(70):
        with np.errstate(over="ignore"):  # the last ones are infinite
            x = (pool.rng.standard_normal((1, 2, 64)) * 1.2 ** t).astype(np.float16)
        pool.kv_len = [t + 1]
        tql.exl3_kv8_append(pool.cache, pool.batch([1]), rows_on_device(x.reshape(1, -1), 0), rows_on_device(-x.reshape(1, -1), 0))
        ref.append(*want[0], pool.table, [t + 1], [1], x)
        ref.append(*want[1], pool.table, [t + 1], [1], -x)
    for i in range(2):
        assert np.array_equal(pool.t[2 + i].cpu().numpy(), want[i][1])
        got = pool.t[i].cpu().numpy()
        assert np.array_equal(np.where(got & 0x7F, got, 0), np.where(want[i][0] & 0x7F, want[i][0], 0))


# --------------------------------------------------------------------------- weigh


@pytest.mark.parametrize("kv_len,counts,heads,kv_heads,dim,cap,causal", ATTENTION)
def test_weigh(kv_len, counts, heads, kv_heads, dim, cap, causal):
    torch = torch_mod()
    pool = Pool(kv_len, kv_heads, dim, seed=len(kv_len) * 500 + heads)
    pool.on_device()
    R = sum(counts)
    q = (2 * pool.rng.standard_normal((R, heads, dim))).astype(np.float16)
    scale = dim ** -0.5
    _, lse, _, _ = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts,
                                 q, scale, cap, causal)
    lse = lse.astype(np.float32)
    tql.exl3_kv8_weigh(pool.cache, pool.batch(counts), rows_on_device(q.reshape(R, -1), 8), heads, scale, dev(lse),
                       softcap=cap, causal=causal)
    torch.cuda.synchronize()
    got = pool.t[4].cpu().numpy()
    add, bound = ref.weigh(pool.codes[0], pool.scales[0], pool.table, kv_len, counts, q, lse, scale, cap, causal,
                           64 * pool.max_pages)
    untouched = np.ones(pool.n, dtype=bool)
    terms = max(counts) * (heads // kv_heads)
    for s, length in enumerate(kv_len):
        for b in range(pool.max_pages):
            page = pool.table[s][b]
            untouched[page] = False
            a, e = add[s, :, 64 * b:64 * b + 64], bound[s, :, 64 * b:64 * b + 64]
            w = pool.weight[page].astype(np.float64) + a
            tol = ((dim + 8) * U + 2.0 ** -20) * e + cap * 2.0 ** -21 * a + (terms + 2) * U * (a + w)
            assert np.all(np.abs(got[page] - w) <= tol)
            assert np.array_equal(got[page][a == 0], pool.weight[page][a == 0])
    assert np.array_equal(got[untouched], pool.weight[untouched])


def test_weigh_same_result_every_time():
    kv_len, counts = [900, 200], [130, 7]
    results = []
    for _ in range(2):
        pool = Pool(kv_len, 2, 128, seed=77)
        pool.on_device()
        q = pool.rng.standard_normal((137, 8, 128)).astype(np.float16)
        lse = np.full((137, 8), 5.0, dtype=np.float32)
        tql.exl3_kv8_weigh(pool.cache, pool.batch(counts), rows_on_device(q.reshape(137, -1), 0), 8, 0.1, dev(lse))
        results.append(pool.t[4].cpu().numpy())
    assert np.array_equal(*results)


# --------------------------------------------------------------------------- evict


@pytest.mark.parametrize("kv_len,budget,recent,kv_heads,dim", [
    ([1], 1, 0, 1, 64), ([65], 64, 64, 1, 128), ([65], 64, 0, 2, 128), ([300, 0, 17, 100], 100, 30, 2, 64),
    ([1100], 1000, 128, 2, 64), ([2500, 1999], 130, 1, 3, 128), ([5000], 70, 69, 1, 64), ([5000], 4999, 7, 1, 64)])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict(kv_len, budget, recent, kv_heads, dim, kind):
    torch = torch_mod()
    blocks = -(-budget // 64)
    pool = Pool(kv_len, kv_heads, dim, seed=budget + recent, extra=len(kv_len) * blocks)
    rng = pool.rng
    if kind == "ties":
        pool.weight = rng.integers(0, 3, pool.weight.shape).astype(np.float32)
    elif kind == "special":
        pool.weight = rng.choice(np.array([0.0, -0.0, 1.0, 1e-40, -1.0, np.nan, np.inf, -np.inf, 3e38], dtype=np.float32),
                                 pool.weight.shape)
    pool.on_device()
    free = np.setdiff1d(np.arange(pool.n), pool.table.ravel())
    dst = rng.permutation(free)[:len(kv_len) * blocks].reshape(len(kv_len), blocks).astype(np.int32)
    kept = torch.full((len(kv_len), kv_heads, budget), -7, dtype=torch.int32, device="cuda")
    new_len = torch.full((len(kv_len),), -7, dtype=torch.int32, device="cuda")
    batch = tql.Exl3Kv8Batch(dev(pool.table), dev(np.array(kv_len, dtype=np.int32)))
    tql.exl3_kv8_evict(pool.cache, batch, dev(dst), budget, recent, kept, new_len)
    torch.cuda.synchronize()
    assert new_len.tolist() == [min(budget, x) for x in kv_len]
    want = [pool.codes[0].copy(), pool.codes[1].copy(), pool.scales[0].copy(), pool.scales[1].copy(), pool.weight.copy()]
    for s, length in enumerate(kv_len):
        for h in range(kv_heads):
            w = pool.weight[pool.table[s], h].ravel()
            keep = ref.evict_choice(w, length, budget, recent)
            assert kept[s, h].tolist() == keep + [-1] * (budget - len(keep))
            for b in range(-(-len(keep) // 64)):
                at = np.array(keep[64 * b:64 * b + 64])
                page, slot = pool.table[s][at // 64], at % 64
                for i in range(2):
                    top = pool.scales[i][page, h].max()
                    want[2 + i][dst[s, b], h] = top
                    x = ref.VALUES[pool.codes[i][page, h, slot]] * (pool.scales[i][page, h] / top).astype(np.float64)[:, None]
                    want[i][dst[s, b], h, :at.size] = ref.nearest_code(x)
                want[4][dst[s, b], h, :at.size] = pool.weight[page, h, slot]
    for i in range(5):
        got = pool.t[i].cpu().numpy()
        if i < 2:
            zero = (got & 0x7F == 0) & (want[i] & 0x7F == 0)
            got, want[i] = np.where(zero, 0, got), np.where(zero, 0, want[i])
        assert np.array_equal(got, want[i], equal_nan=i == 4)


# --------------------------------------------------------------------------- logits


@pytest.mark.parametrize("n,ld", [(1, 4), (31, 32), (1000, 1000), (8191, 8192), (20077, 20096), (248077, 248192)])
@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("rules", ["all", "penalties", "mask", "none"])
def test_logits_adjust(n, ld, M, rules):
    torch = torch_mod()
    rng = np.random.default_rng([n, M])
    logits = (3 * rng.standard_normal((M, ld))).astype(np.float32)
    logits[:, n:] = np.nan
    logits[0, rng.integers(0, n)] = -np.inf
    if n > 100:
        logits[M - 1, 5] = np.nan
    hist = [rng.integers(-2, n + 2, int(rng.integers(0, 400))) for _ in range(M)]
    if n > 30:
        hist[0] = np.concatenate([np.full(300, 7), np.arange(30), hist[0]])
    bias = [[(int(t), float(np.float32(rng.standard_normal()))) for t in rng.integers(-1, n + 1, 70)] for _ in range(M)]
    bias[0] += [(0, 1.0), (0, -0.25), (n - 1, float("-inf"))]
    gen = rng.integers(0, 200, M).astype(np.int32)
    rep, pres, freq = (rng.uniform(a, b, M).astype(np.float32) for a, b in ((0.8, 1.6), (-0.5, 1.0), (-0.1, 0.5)))
    allow = rng.random((M, n)) < 0.6
    if M > 1:
        allow[1] = False  # nothing is left of this row
    kw = {}
    if rules in ("all", "penalties"):
        kw |= dict(history=dev(np.concatenate(hist).astype(np.int32)),
                   history_start=dev(np.cumsum([0] + [len(h) for h in hist]).astype(np.int32)), generated_from=dev(gen),
                   repetition=dev(rep), presence=dev(pres), frequency=dev(freq))
    if rules == "all":
        kw |= dict(bias_id=dev(np.array([t for b in bias for t, _ in b], dtype=np.int32)),
                   bias_value=dev(np.array([v for b in bias for _, v in b], dtype=np.float32)),
                   bias_start=dev(np.cumsum([0] + [len(b) for b in bias]).astype(np.int32)))
    if rules in ("all", "mask"):
        words = np.zeros((M, -(-n // 32) * 32), dtype=bool)
        words[:, :n] = allow
        kw |= dict(allowed=dev(np.packbits(words, axis=1, bitorder="little").view(np.uint32).view(np.int32)))
    for in_place in (False, True):
        x = dev(logits)
        out = x if in_place else torch.full((M, ld), 9.0, device="cuda")
        am = torch.full((M,), -9, dtype=torch.int32, device="cuda")
        tql.exl3_logits_adjust(x, n, out, am, **kw)
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        assert np.array_equal(got[:, n:], logits[:, n:] if in_place else np.full((M, ld - n), 9.0), equal_nan=True)
        for m in range(M):
            full = rules in ("all", "penalties")
            args = (hist[m] if full else [], gen[m], rep[m] if full else 1, pres[m] if full else 0, freq[m] if full else 0,
                    bias[m] if rules == "all" else [], allow[m] if rules in ("all", "mask") else None)
            want, pick = ref.adjust(logits[m, :n], *args, np.float32)
            assert np.array_equal(got[m, :n], want, equal_nan=True)
            assert int(am[m]) == pick
            exact, _ = ref.adjust(logits[m, :n], *args, np.float64)
            fine = np.isfinite(exact)
            # seven roundings of intermediate results, none above |l| * rep + |pres| + |freq| c + the biases
            big = np.abs(np.where(fine, logits[m, :n], 0)) * 2 + 1 + 0.5 * len(hist[m]) + sum(abs(v) for _, v in bias[m] if np.isfinite(v))
            assert np.all(np.abs(want[fine] - exact[fine]) <= (80 * U * big)[fine])


def test_logits_adjust_ties_take_the_first():
    torch = torch_mod()
    x = torch.zeros((3, 50000), device="cuda")
    x[1, 41000:] = 2.0
    x[2, :] = -0.0
    am = torch.empty((3,), dtype=torch.int32, device="cuda")
    tql.exl3_logits_adjust(x, 50000, x, am)
    assert am.tolist() == [0, 41000, 0]


# --------------------------------------------------------------------------- device-side checks, empty calls


def test_bad_indexes_on_the_device_are_reported_and_skipped():
    torch = torch_mod()
    pool = Pool([100, 100], 1, 64, seed=1)
    cache = pool.on_device()
    q = rows_on_device(np.ones((2, 64), dtype=np.float16), 0)
    out = torch.zeros((2, 64), dtype=torch.float16, device="cuda")
    before = [t.clone() for t in pool.t]

    def calls(batch):
        ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
        yield lambda: tql.exl3_kv8_attention(cache, batch, q, 1, 1.0, out, ws)
        yield lambda: tql.exl3_kv8_append(cache, batch, q, q)
        yield lambda: tql.exl3_kv8_weigh(cache, batch, q, 1, 1.0, torch.zeros((2, 1), device="cuda"))

    for table, kv_len, start in (([[-1] * 3, [pool.n] * 3], [100, 100], [0, 1, 2]), (pool.table, [1000, -5], [0, 1, 2]),
                                 (pool.table, [100, 100], [0, 5, 2]), (pool.table, [100, 100], [-3, 0, 2])):
        batch = tql.Exl3Kv8Batch(dev(np.array(table, dtype=np.int32)), dev(np.array(kv_len, dtype=np.int32)),
                                 dev(np.array(start, dtype=np.int32)), 2, 1)
        for call in calls(batch):
            call()
            assert tql.exl3_get_device_status() == 10
            assert tql.exl3_get_device_status() == 0
    # the other sequence of the third and fourth batches was still served: only its tokens may have changed
    same = np.setdiff1d(np.arange(pool.n), pool.table.ravel())
    for t, b in zip(pool.t, before):
        assert torch.equal(t[same], b[same])


@pytest.mark.parametrize("table,kv_len,start", [([[-1] * 3, [1 << 30] * 3], [100, 100], [0, 20, 40]),
                                                (None, [1000, -5], [0, 20, 40]), (None, [100, 100], [0, 41, 40]),
                                                (None, [100, 100], [-3, 0, 40])])
def test_bad_indexes_on_the_device_with_many_rows(table, kv_len, start):
    torch = torch_mod()
    pool = Pool([100, 100], 1, 128, seed=1)
    cache = pool.on_device()
    q = rows_on_device(np.ones((40, 128), dtype=np.float16), 0)
    batch = tql.Exl3Kv8Batch(dev(np.array(pool.table if table is None else table, dtype=np.int32)), dev(np.array(kv_len, dtype=np.int32)),
                             dev(np.array(start, dtype=np.int32)), 40, 20)
    out = torch.zeros((40, 128), dtype=torch.float16, device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
    for call in (lambda: tql.exl3_kv8_attention(cache, batch, q, 1, 1.0, out, ws), lambda: tql.exl3_kv8_append(cache, batch, q, q),
                 lambda: tql.exl3_kv8_weigh(cache, batch, q, 1, 1.0, torch.zeros((40, 1), device="cuda"))):
        call()
        assert tql.exl3_get_device_status() == 10
        assert tql.exl3_get_device_status() == 0


def test_chunk_lengths_change_under_one_graph():
    """As above for the kernels of many rows: a captured chunk serves other lengths and rows."""
    torch = torch_mod()
    pool = Pool([500, 300], 2, 64, seed=22)
    cache = pool.on_device()
    batch = pool.batch([60, 40])
    q = pool.rng.standard_normal((100, 4, 64)).astype(np.float16)
    qd = rows_on_device(q.reshape(100, -1), 0)
    out = torch.zeros((100, 256), dtype=torch.float16, device="cuda")
    lse = torch.zeros((100, 4), device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, 4), dtype=torch.uint8, device="cuda")

    def call():
        tql.exl3_kv8_attention(cache, batch, qd, 4, 0.2, out, ws, lse=lse)
        tql.exl3_kv8_weigh(cache, batch, qd, 4, 0.2, lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for kv_len, counts in (([500, 300], [60, 40]), ([130, 60], [45, 55]), ([33, 7], [60, 40])):
        batch._keep[1].copy_(dev(np.array(kv_len, dtype=np.int32)))
        batch._keep[2].copy_(dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts,
                             q, 0.2, 0.0, True)
        check_attention(out.float().cpu().numpy().reshape(100, 4, 64), lse.cpu().numpy(), want, 64, 0.0, 500)


def test_empty_calls_are_no_ops():
    torch = torch_mod()
    pool = Pool([10], 1, 64, seed=1)
    cache = pool.on_device()
    before = [t.clone() for t in pool.t]
    none = tql.Exl3Kv8Batch(torch.zeros((0, 1), dtype=torch.int32, device="cuda").reshape(0, 1), torch.zeros((1,), dtype=torch.int32, device="cuda")[:0],
                            torch.zeros((1,), dtype=torch.int32, device="cuda"), 0, 0)
    some = pool.batch([0])
    q = torch.zeros((1, 64), dtype=torch.float16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for batch in (none, some):
        batch.page_table = batch.page_table or table.data_ptr()
        batch.kv_len = batch.kv_len or table.data_ptr()
        tql.exl3_kv8_attention(cache, batch, q, 1, 1.0, torch.zeros_like(q), ws)
        tql.exl3_kv8_append(cache, batch, q, q)
        tql.exl3_kv8_weigh(cache, batch, q, 1, 1.0, torch.zeros((1, 1), device="cuda"))
    none.page_table = none.kv_len = table.data_ptr()
    tql.exl3_kv8_evict(cache, none, table, 64, 0, table, table)
    at, rules = before[4].data_ptr(), ctypes.byref(tql._LogitsRules())
    assert tql.load().exl3_logits_adjust(at, 4, 0, 4, rules, at, 4, at, None) == 0
    torch.cuda.synchronize()
    for t, b in zip(pool.t, before):
        assert torch.equal(t, b)
