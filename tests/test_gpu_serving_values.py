"""The serving operators on values of unusual size: small and missing value blocks,
caps far above the scores, weights spread over many tokens, scales of either sign.

Tolerances as in test_gpu_serving.py, or stated at the test.
"""
import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import U, Pool, attend, check_attention, dev, gpu, rows_on_device  # noqa: F401 (gpu: fixture)
from test_gpu_serving_limits import check_weigh

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


@pytest.mark.parametrize("cap", [30.0, 1e3, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("counts", [[1, 3], [70, 49]])
def test_caps_far_above_the_scores(cap, counts):
    """cap * tanh(s / cap) to an error relative to s: 2^-19, which is less than the products' (D + 8) ulp that the
    tolerance without a cap has. Caps of 1e8 and more are no caps: the weights too."""
    kv_len, heads, dim = [300, 999], 4, 128
    pool = Pool(kv_len, 2, dim, seed=31)
    pool.on_device()
    R, scale = sum(counts), 0.25
    q = (2 * pool.rng.standard_normal((R, heads, dim))).astype(np.float16)
    got, lse = attend(pool, counts, q, heads, scale, cap, True)
    args = (pool.table, kv_len, counts, q)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], *args, scale, cap, True)
    check_attention(got, lse, want, dim, 0.0, max(kv_len))
    lse = want[1].astype(np.float32)
    tql.exl3_kv8_weigh(pool.cache, pool.batch(counts), rows_on_device(q.reshape(R, -1), 8), heads, scale, dev(lse), softcap=cap)
    got = pool.t[4].cpu().numpy()
    add, bound = ref.weigh(pool.codes[0], pool.scales[0], *args, lse, scale, cap, True, 64 * pool.max_pages)
    for s, length in enumerate(kv_len):
        for b in range(-(-length // 64)):
            page, a, e = pool.table[s][b], add[s, :, 64 * b:64 * b + 64], bound[s, :, 64 * b:64 * b + 64]
            w = pool.weight[page].astype(np.float64) + a
            tol = ((dim + 8) * U + 2.0 ** -20) * e + (max(counts) * heads + 2) * U * (a + w)
            assert np.all(np.abs(got[page] - w) <= tol)


@pytest.mark.parametrize("cap", [1e-3, 1.0, 30.0, 5e4])
@pytest.mark.parametrize("rows", [1, 50])
def test_capped_score_to_its_stated_error(cap, rows):
    """A sequence of one token: lse is its capped score, to 2^-19 of it and two more roundings."""
    torch = torch_mod()
    seqs, heads, dim = 500, 2, 64
    codes = [torch.zeros((1, 1, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes[0][0, 0, 0, 0] = 7 << 3  # 1.0
    cache = tql.Exl3Kv8Cache(*codes, *[torch.ones((1, 1), device="cuda") for _ in range(2)])
    batch = tql.Exl3Kv8Batch(torch.zeros((seqs, 1), dtype=torch.int32, device="cuda"), torch.ones(seqs, dtype=torch.int32, device="cuda"),
                             torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * rows, seqs * rows, rows)
    rng = np.random.default_rng(int(cap * 1000) + rows)
    x = (rng.choice([-1.0, 1.0], (seqs * rows, heads)) * 2.0 ** rng.uniform(-12, 4, (seqs * rows, heads))).astype(np.float16)
    q = np.zeros((seqs * rows, heads, dim), dtype=np.float16)
    q[:, :, 0] = x
    qd = dev(q.reshape(seqs * rows, -1))
    out, lse = torch.empty_like(qd), torch.empty((seqs * rows, heads), device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, heads), dtype=torch.uint8, device="cuda")
    tql.exl3_kv8_attention(cache, batch, qd, heads, cap, out, ws, softcap=cap, causal=False, lse=lse)
    c = float(np.float32(cap))
    want = c * np.tanh(x.astype(np.float64))
    assert np.all(np.abs(lse.double().cpu().numpy() - want) <= (2.0 ** -19 + 4 * U) * np.abs(want) + 16 * U)


@pytest.mark.parametrize("rows,length,seqs,heads", [(1, 131072, 20, 8), (2, 65536, 40, 8), (60, 65536, 20, 8), (256, 40000, 20, 8)])
def test_weight_spread_over_many_tokens(rows, length, seqs, heads):
    """One token takes nearly all the weight and has no value; the others have 2^-25.25 of its weight each, and all the
    value. Each of their probabilities is rounded to 11 bits, the sums (an output is one of at most `length` / 16 steps in
    fp32, which the tensor cores cut off) and the fp16 result: 2^-10 + length / 16 * 2^-23 in all."""
    torch = torch_mod()
    dim, blocks = 64, length // 64
    small = 2.0 ** -25.25
    codes = [torch.zeros((2, heads, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    one = 7 << 3  # 1.0 in E4M3
    codes[0][0, :, 0, 0] = one
    codes[1][:] = one
    codes[1][0, :, 0] = 0
    cache = tql.Exl3Kv8Cache(*codes, *[torch.ones((2, heads), device="cuda") for _ in range(2)])
    table = torch.ones((seqs, blocks), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    batch = tql.Exl3Kv8Batch(table, torch.full((seqs,), length, dtype=torch.int32, device="cuda"),
                             torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * rows, seqs * rows, rows)
    q = torch.zeros((seqs * rows, heads * dim), dtype=torch.float16, device="cuda")
    q[:, ::dim] = 1.0
    out, lse = torch.empty_like(q), torch.empty((seqs * rows, heads), device="cuda")
    ws = torch.empty(tql.exl3_kv8_attention_workspace_bytes(cache, batch, heads), dtype=torch.uint8, device="cuda")
    tql.exl3_kv8_attention(cache, batch, q, heads, float(-np.log(small)), out, ws, causal=False, lse=lse)
    rest = (length - 1) * small
    want = rest / (1 + rest)
    assert np.abs(out.double().cpu().numpy() / want - 1).max() <= 2.0 ** -10 + length / 16 * 2.0 ** -23
    assert np.abs(lse.double().cpu().numpy() - (np.log1p(rest) - np.log(small))).max() <= 2.0 ** -16


@pytest.mark.parametrize("scale", [-0.125, 0.0])
@pytest.mark.parametrize("counts,cap", [([1, 2], 0.0), ([20, 9], 20.0), ([60, 130], 0.0), ([60, 130], 20.0)])
def test_scales_of_either_sign(scale, counts, cap):
    pool = Pool([300, 257], 2, 64, seed=41)
    pool.on_device()
    q = (2 * pool.rng.standard_normal((sum(counts), 4, 64))).astype(np.float16)
    got, lse = attend(pool, counts, q, 4, scale, cap, True)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, pool.kv_len, counts, q, scale, cap, True)
    check_attention(got, lse, want, 64, cap, 300)
    check_weigh(pool, counts, 4, q, want[1].astype(np.float32), scale, cap, True)


@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("counts", [[1], [60]])
def test_blocks_of_very_different_size(which, counts):
    """Scales from 2^-29 to 2^8. Single tokens have every block exactly. Many rows lose what is below 2^-25 of the largest
    block's largest value (448 scales), seen or not: that much of a key element or value, on top of the other tolerances."""
    pool = Pool([900], 1, 64, seed=43, spread=0)
    i = 0 if which == "keys" else 1
    for b in range(15):
        pool.scales[i][pool.table[0][b]] = 2.0 ** [8, -29, -16, -10, -18, 0, -25, -17, -7, -29, -24, -20, 4, -27, -12][(b + 4) % 15]
    pool.on_device()
    scale = 2.0 ** -14 if which == "keys" else 0.125
    q = pool.rng.standard_normal((sum(counts), 1, 64)).astype(np.float16)
    got, lse = attend(pool, counts, q, 1, scale, 0.0, True)
    out, wlse, mag, sabs = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, [900], counts, q, scale,
                                         0.0, True)
    lost = 0.0 if counts == [1] else 2.0 ** -25 * 448 * 2.0 ** 8
    s_lost = lost * scale * np.abs(q.astype(np.float64)).sum(2) if which == "keys" else 0 * wlse
    s_err = (64 + 8) * U * sabs + 2.0 ** -20 * (1 + np.abs(wlse) + sabs) + s_lost
    assert np.all(np.abs(lse - wlse) <= s_err)
    tol = 2.0 ** -11 * np.abs(out) + (2.0 ** -11 + 2 * s_err[:, :, None]) * mag + 2.0 ** -25 + (lost if which == "values" else 0.0)
    assert np.all(np.abs(got - out) <= tol)


@pytest.mark.parametrize("gain", [2.0 ** -22, 2.0 ** -6])
@pytest.mark.parametrize("rows", [1, 60])
def test_lse_of_few_tokens_with_small_scores(gain, rows):
    """As test_gpu_serving.py has it: 2^-21 of 1 + |lse|, besides the products' error."""
    rng = np.random.default_rng(rows)
    kv_len = rng.integers(1, 40, 300).tolist()
    counts = [rows] + rng.integers(0, rows + 1, 299).tolist()
    pool = Pool(kv_len, 1, 64, seed=51, spread=0, gain=gain)
    pool.on_device()
    q = rng.standard_normal((sum(counts), 1, 64)).astype(np.float16)
    got, lse = attend(pool, counts, q, 1, 0.125, 0.0, False)
    want = ref.attention(pool.codes[0], pool.scales[0], pool.codes[1], pool.scales[1], pool.table, kv_len, counts, q, 0.125, 0.0, False)
    assert np.all(np.abs(lse - want[1]) <= 2.0 ** -21 * (1 + np.abs(want[1]) + want[3]) + (64 + 8) * U * want[3])
